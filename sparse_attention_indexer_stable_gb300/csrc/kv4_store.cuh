// kv4_store.cuh -- writing tokens into the 4-bit cache and reading them back.
//
// One thread per block of 16 elements, of K and of V: a block's amax, scale and
// codes need nothing from other threads, its loads are 32 or 64 contiguous
// bytes and neighbouring threads take neighbouring blocks, so both sides are
// coalesced.  2.56 bytes move per 16-bit element.  8192 tokens of 8 heads x 128
// (86 MB in all) go in and come back in 21.5 us, 59% of the measured copy rate:
// each kernel is two or three waves of CTAs long, and the append issues 215
// instructions a warp and block besides.
#pragma once

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

struct StoreParams {
  Planes c;
  const void* in[2];  // K, V
  int64_t row_stride[2], head_stride[2];
  bool vec[2];  // 16-byte loads possible
  void* out[2];
  const int64_t* slots;
  int64_t N;
  int dtype;
  int blocks;  // per head: dim / 16
};

// A block of 16 elements as it lies in memory: 32 bytes, or 64 of fp32.
struct RawBlock {
  uint4 v[4];
};

__device__ __forceinline__ RawBlock load_block(const void* base, int64_t i, int dtype, bool vec) {
  RawBlock r;
  if (vec) {
    const uint4* p = dtype == DCP_F32
                         ? reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i)
                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    r.v[0] = __ldg(p);
    r.v[1] = __ldg(p + 1);
    if (dtype == DCP_F32) r.v[2] = __ldg(p + 2), r.v[3] = __ldg(p + 3);
    return r;
  }
  uint32_t* w = reinterpret_cast<uint32_t*>(r.v);
  if (dtype == DCP_F32) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = __float_as_uint(__ldg(static_cast<const float*>(base) + i + e));
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = __ldg(p + 2 * e) | ((uint32_t)__ldg(p + 2 * e + 1) << 16);
  }
  return r;
}

// Its values in fp32 and their largest magnitude, NaN if any element is NaN.
__device__ __forceinline__ float unpack_block(const RawBlock& r, int dtype, float (&x)[16]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
  if (dtype == DCP_F32) {
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = __uint_as_float(w[e]);
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(x[e])));
    }
    return amax;
  }
  // pairs of 16-bit elements: magnitudes compared two at a time
  uint32_t top = 0u;
  if (dtype == DCP_BF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[e] & 0x7FFF7FFFu));
    }
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(top << 16));
    return __uint_as_float(top & 0xFFFF0000u);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + e));
    x[2 * e] = f.x, x[2 * e + 1] = f.y;
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(w[e] & 0x7FFF7FFFu));
  }
  asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(top << 16));
  return __half2float(__ushort_as_half((unsigned short)(top >> 16)));
}

// The scale of a block whose largest magnitude is amax units.  The division
// is correctly rounded, and no quotient rounds onto a midpoint of the 8-bit
// grid that the exact quotient misses (6 times a midpoint is an fp32 number of
// at most 7 significant bits, and a neighbouring fp32 dividend is more than
// half a unit of the quotient's last place away), so the scale is the exact
// quotient rounded once.
__device__ __forceinline__ float encode_scale(float amax, uint8_t& bits) {
  uint16_t pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(pair)
      : "f"(0.0f), "f"(fminf(__fdiv_rn(amax, 6.0f), 448.0f)));
  bits = (uint8_t)pair;
  return __half2float(__ushort_as_half((unsigned short)scales_to_half(pair & 0xFFu)));
}

__device__ __forceinline__ uint32_t encode_pair(float lo, float hi) {
  uint32_t b;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}"
      : "=r"(b)
      : "f"(hi), "f"(lo));
  return b;
}

// Codes (8 bytes) and scale of a block; each code is the exact quotient
// rounded once.
//  - With fp32 inputs by correctly rounded divisions, which meet a midpoint of
//    the 4-bit grid only where the exact quotient does (as for the scale).
//  - With 16-bit inputs (at most 11 significant bits) by the scale's
//    reciprocal: a quotient that is no midpoint is at least 2^-13 away from
//    it, one that is errs by less than 2^-19, so rounding to multiples of
//    2^-16 first (by adding and subtracting 192) puts every tie back on its
//    midpoint and moves nothing else across.  16 divisions a block made the
//    pair of kernels 26 us long instead of 22.
__device__ __forceinline__ uint2 encode_block(const float (&x)[16], float amax, float inv_unit,
                                              bool narrow, uint8_t& scale) {
  if (amax != amax) {  // NaN: the others' largest
    amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
    narrow = false;
  }
  const float s = encode_scale(amax * inv_unit, scale);  // unit is a power of two
  uint32_t w[2] = {0u, 0u};
  if (!(s > 0.0f)) return make_uint2(0u, 0u);
  const float inv = __fdiv_rn(inv_unit, s);
  if (narrow && s < 448.0f && inv > 1e-30f && inv < 1e30f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float lo = __fadd_rn(__fmaf_rn(x[2 * e], inv, 192.0f), -192.0f);
      const float hi = __fadd_rn(__fmaf_rn(x[2 * e + 1], inv, 192.0f), -192.0f);
      w[e >> 2] |= encode_pair(lo, hi) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // NaN becomes 0 (the conversion would give the largest value)
    const float lo = x[2 * e] == x[2 * e] ? __fdiv_rn(x[2 * e] * inv_unit, s) : 0.0f;
    const float hi =
        x[2 * e + 1] == x[2 * e + 1] ? __fdiv_rn(x[2 * e + 1] * inv_unit, s) : 0.0f;
    w[e >> 2] |= encode_pair(lo, hi) << (8 * (e & 3));
  }
  return make_uint2(w[0], w[1]);
}

// This thread's block: its token and its place in the token; false beyond the
// last.  In 32 bits where the blocks can be counted so (a 64-bit division
// costs as much as the rest of the kernel).
__device__ __forceinline__ bool find_block(const StoreParams& p, int64_t& n, int& r) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const uint32_t per_token = (uint32_t)(p.c.heads * p.blocks);
  const int64_t all = p.N * per_token;
  if (i >= all) return false;
  if (all <= 0xffffffffll) {
    const uint32_t t = (uint32_t)i / per_token;
    n = t;
    r = (int)((uint32_t)i - t * per_token);
  } else {
    n = i / per_token;
    r = (int)(i - n * per_token);
  }
  return true;
}

__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ StoreParams p) {
  grid_dependency_wait();
  int64_t n;
  int r;
  if (!find_block(p, n, r)) return;
  const int h = r / p.blocks, b = r - h * p.blocks;
  const int64_t slot = __ldg(p.slots + n);
  RawBlock raw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)  // K, V
    raw[i] = load_block(p.in[i], n * p.row_stride[i] + h * p.head_stride[i] + b * kBlock, p.dtype,
                        p.vec[i]);
  if ((uint64_t)slot >= p.c.num_slots()) return;
  const int64_t at = slot * (p.c.heads * p.blocks) + r;  // block's index in the plane
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[16];
    const float amax = unpack_block(raw[i], p.dtype, x);
    uint8_t scale;
    const uint2 codes = encode_block(x, amax, 1.0f / (i ? p.c.v_unit : p.c.k_unit),
                                     p.dtype != DCP_F32, scale);
    reinterpret_cast<uint2*>(i ? p.c.v_codes : p.c.k_codes)[at] = codes;
    (i ? p.c.v_scales : p.c.k_scales)[at] = scale;
  }
}

// The values of a block in fp32.
__device__ __forceinline__ void decode_block(uint2 codes, uint32_t scale, float unit,
                                             float2 (&f)[8]) {
  const uint32_t s2 = scales_to_half(scale | (scale << 8));
  uint32_t d[8], w[4];
  codes_to_half(codes.x, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = hmul2(w[e], s2);
  codes_to_half(codes.y, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[4 + e] = hmul2(w[e], s2);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = __half22float2(*reinterpret_cast<const __half2*>(d + e));
    f[e].x *= unit, f[e].y *= unit;
  }
}

__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ StoreParams p) {
  grid_dependency_wait();
  int64_t n;
  int r;
  if (!find_block(p, n, r)) return;
  const int64_t per_token = (int64_t)p.c.heads * p.blocks, i = n * per_token + r;
  const int64_t slot = __ldg(p.slots + n);
  uint2 codes[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};  // K, V
  uint32_t scale[2] = {0u, 0u};
  if ((uint64_t)slot < p.c.num_slots()) {
    const int64_t at = slot * per_token + r;
    codes[0] = __ldg(reinterpret_cast<const uint2*>(p.c.k_codes) + at);
    codes[1] = __ldg(reinterpret_cast<const uint2*>(p.c.v_codes) + at);
    scale[0] = __ldg(p.c.k_scales + at);
    scale[1] = __ldg(p.c.v_scales + at);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 f[8];
    decode_block(codes[k], scale[k], k ? p.c.v_unit : p.c.k_unit, f);
    if (p.dtype == DCP_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out[k]) + i * kBlock);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = make_float4(f[2 * e].x, f[2 * e].y, f[2 * e + 1].x, f[2 * e + 1].y);
    } else {
      uint32_t u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = pack_pair(f[e].x, f[e].y, p.dtype);
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[k]) + i * kBlock);
      o[0] = make_uint4(u[0], u[1], u[2], u[3]);
      o[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }
}

}  // namespace kv4
}  // namespace dcp
