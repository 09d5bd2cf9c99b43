// kv4_store.cuh -- writing tokens into the 4-bit cache and reading them back.
//
// One thread per block of 16 elements: a block's amax, scale and codes need
// nothing from other threads, its loads are 32 or 64 contiguous bytes and
// neighbouring threads take neighbouring blocks, so both sides are coalesced.
// Bound by memory: 2.56 bytes move per 16-bit element.
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

// The 16 elements at p (in elements of dtype) in fp32.
__device__ __forceinline__ void load_block(const void* base, int64_t i, int dtype, bool vec,
                                           float (&x)[16]) {
  if (dtype == DCP_F32) {
    const float* p = static_cast<const float*>(base) + i;
    if (vec) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p) + e);
        x[4 * e] = v.x, x[4 * e + 1] = v.y, x[4 * e + 2] = v.z, x[4 * e + 3] = v.w;
      }
      return;
    }
  } else if (vec) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint4 v[2] = {__ldg(p), __ldg(p + 1)};
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (dtype == DCP_BF16) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + e));
        x[2 * e] = f.x, x[2 * e + 1] = f.y;
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = load_element(base, i + e, dtype);
}

// Codes (8 bytes) and scale of a block.  The two divisions are correctly
// rounded, and no quotient rounds onto a midpoint of the 4- or 8-bit grid
// that the exact quotient misses (the midpoints times 6, and times any scale,
// are fp32 numbers of at most 7 significant bits; a neighbouring fp32
// dividend is more than half a unit of the quotient's last place away), so
// each code and scale is the exact quotient rounded once.
__device__ __forceinline__ uint2 encode_block(float (&x)[16], float inv_unit, uint8_t& scale) {
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    x[e] *= inv_unit;                  // a power of two
    amax = fmaxf(amax, fabsf(x[e]));   // NaN is ignored
  }
  uint16_t pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(pair)
      : "f"(0.0f), "f"(fminf(__fdiv_rn(amax, 6.0f), 448.0f)));
  scale = (uint8_t)pair;
  const uint32_t h = scales_to_half(pair & 0xFFu);
  const float s = __half2float(__ushort_as_half((unsigned short)h));
  uint32_t w[2] = {0u, 0u};
  if (s > 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // NaN becomes 0 (the conversion would give the largest value)
      const float lo = x[2 * e] == x[2 * e] ? __fdiv_rn(x[2 * e], s) : 0.0f;
      const float hi = x[2 * e + 1] == x[2 * e + 1] ? __fdiv_rn(x[2 * e + 1], s) : 0.0f;
      uint32_t b;
      asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}"
          : "=r"(b)
          : "f"(hi), "f"(lo));
      w[e >> 2] |= b << (8 * (e & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ StoreParams p) {
  grid_dependency_wait();
  const int which = blockIdx.y;  // 0: K, 1: V
  const int64_t per_token = (int64_t)p.c.heads * p.blocks;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.N * per_token) return;
  const int64_t n = i / per_token;
  const int r = (int)(i - n * per_token);
  const int h = r / p.blocks, b = r - h * p.blocks;
  const int64_t slot = __ldg(p.slots + n);
  if ((uint64_t)slot >= p.c.num_slots()) return;
  float x[16];
  load_block(p.in[which], n * p.row_stride[which] + h * p.head_stride[which] + b * kBlock, p.dtype,
             p.vec[which], x);
  uint8_t scale;
  const uint2 codes = encode_block(x, 1.0f / (which ? p.c.v_unit : p.c.k_unit), scale);
  const int64_t at = slot * per_token + r;  // block's index in the plane
  reinterpret_cast<uint2*>(which ? p.c.v_codes : p.c.k_codes)[at] = codes;
  (which ? p.c.v_scales : p.c.k_scales)[at] = scale;
}

__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ StoreParams p) {
  grid_dependency_wait();
  const int which = blockIdx.y;
  const int64_t per_token = (int64_t)p.c.heads * p.blocks;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.N * per_token) return;
  const int64_t n = i / per_token;
  const int64_t slot = __ldg(p.slots + n);
  uint2 codes = make_uint2(0u, 0u);
  uint32_t scale = 0u;
  if ((uint64_t)slot < p.c.num_slots()) {
    const int64_t at = slot * per_token + (i - n * per_token);
    codes = __ldg(reinterpret_cast<const uint2*>(which ? p.c.v_codes : p.c.k_codes) + at);
    scale = __ldg((which ? p.c.v_scales : p.c.k_scales) + at);
  }
  const float unit = which ? p.c.v_unit : p.c.k_unit;
  const uint32_t s2 = scales_to_half(scale | (scale << 8));
  uint32_t d[8], w[4];
  codes_to_half(codes.x, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = hmul2(w[e], s2);
  codes_to_half(codes.y, w);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[4 + e] = hmul2(w[e], s2);
  float2 f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = __half22float2(*reinterpret_cast<const __half2*>(d + e));
    f[e].x *= unit, f[e].y *= unit;
  }
  if (p.dtype == DCP_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out[which]) + i * kBlock);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = make_float4(f[2 * e].x, f[2 * e].y, f[2 * e + 1].x, f[2 * e + 1].y);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = pack_pair(f[e].x, f[e].y, p.dtype);
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[which]) + i * kBlock);
    o[0] = make_uint4(u[0], u[1], u[2], u[3]);
    o[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

}  // namespace kv4
}  // namespace dcp
