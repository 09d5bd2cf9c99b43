// prompt_rows.cuh -- attention over whole prompts, one row and head to a warp,
// on the plain arithmetic units: for rows that the tensor cores cannot do (see
// prompt_tiles.cuh), at about a 200th of their speed (2048 rows, 64 heads of 128
// over 8, all of them: 17.4 ms, 4 TFLOP/s), and which rows those are.
//
// With x_j = s_j / ln 2 and a reference r that is a running maximum,
//   l = sum 2^(x_j - r),  out = sum 2^(x_j - r) v_j / l,  lse = ln 2 * (r + log2 l);
// when r grows by d, l and the sum so far are multiplied by 2^-d.  A lane takes
// a key's score, then each lane its 32nd of the value.  Only what a row sees is
// read.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcp_prompt.h"
#include "kv4_common.cuh"

namespace dcp {
namespace prompt {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const void *q, *k, *v;
  int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
  const int32_t* starts;
  void* out;
  float* lse;
  int rows, num_seqs, q_heads, kv_heads, group;
  int dtype, causal, window;
  int capped;
  float mult;  // brings products to powers of two, or to units of the cap
  float cap;   // in powers of two
};

// Sequence bounds as given, cut to the rows that there are.
__device__ __forceinline__ int start_of(const Params& p, int b) {
  return min(max(p.starts[b], 0), p.rows);
}

// A score in powers of two, from q . k.
__device__ __forceinline__ float score_of(const Params& p, float dot) {
  const float s = dot * p.mult;
  return p.capped ? p.cap * kv4::tanh_score(s) : s;
}

template <bool kHalf>
__device__ __forceinline__ float2 pair_of(uint32_t x) {
  if constexpr (kHalf) return __half22float2(reinterpret_cast<const __half2&>(x));
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// As many elements as a lane takes of a row of D: 4, 8 or 16 bytes.
template <int D>
struct alignas(D / 16) Words {
  uint32_t x[D / 64];
};

// Row t (row i of the sequence that starts at row `first` and has n rows), head
// h, by one warp.  It counts `beats` (see Patience), since a row of many keys takes
// longer than those that wait for it would: one every 256 keys, which take some
// 40 us.  A chain of loads and sums bounds it (eight loads are under way at a time;
// with sixteen, and the values' first ones before the scores, 2 to 10% less).
template <int D, bool kHalf>
__device__ __forceinline__ void attend_row(const Params& p, int first, int n, int i, int h,
                                           int* beats) {
  constexpr int kWords = D / 64;  // of two elements, a lane's part of a row
  const int lane = threadIdx.x & 31;
  const int64_t t = first + i;
  const int kv = h / p.group;
  const int from = p.window ? max(0, i - p.window + 1) : 0, to = p.causal ? i + 1 : n;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                  t * p.q_row_stride + h * p.q_head_stride);
  const uint16_t* keys = static_cast<const uint16_t*>(p.k) + first * p.k_row_stride +
                         kv * p.k_head_stride;
  const uint16_t* values = static_cast<const uint16_t*>(p.v) + first * p.v_row_stride +
                           kv * p.v_head_stride + 2 * kWords * lane;
  __syncwarp();  // after what other lanes have written to this row
  float acc[2 * kWords], r = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < 2 * kWords; ++e) acc[e] = 0.0f;
  for (int base = from; base < to; base += 32) {
    if ((base - from) % 256 == 0 && lane == 0) atomicAdd(beats, 1);
    const bool sees = base + lane < to;
    float x = -INFINITY;
    if (sees) {
      const uint4* key = reinterpret_cast<const uint4*>(keys + (base + lane) * p.k_row_stride);
      float dot[4] = {};
#pragma unroll 1
      for (int c = 0; c < D / 8; c += 8) {
        uint4 k[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) k[e] = key[c + e];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 u = q[c + e];
          const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {k[e].x, k[e].y, k[e].z, k[e].w};
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const float2 y = pair_of<kHalf>(a[f]), z = pair_of<kHalf>(b[f]);
            dot[f] = fmaf(y.y, z.y, fmaf(y.x, z.x, dot[f]));
          }
        }
      }
      x = score_of(p, (dot[0] + dot[1]) + (dot[2] + dot[3]));
    }
    float top = x;
#pragma unroll
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float next = fmaxf(r, top);
    const float ref = next == -INFINITY ? 0.0f : next;
    const float shrink = exp2f(r - ref);  // 0 at first
    const float w = exp2f(x - ref);
    float sum = sees ? w : 0.0f;
#pragma unroll
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    l = l * shrink + sum;
    r = next;
#pragma unroll
    for (int e = 0; e < 2 * kWords; ++e) acc[e] *= shrink;
    const int count = min(32, to - base);
#pragma unroll 1
    for (int j = 0; j < count; j += 8) {
      Words<D> v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = {};
        if (j + e < count)
          v[e] = *reinterpret_cast<const Words<D>*>(values + (base + j + e) * p.v_row_stride);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float we = __shfl_sync(~0u, w, j + e);  // 0 where there is no key
#pragma unroll
        for (int f = 0; f < kWords; ++f) {
          const float2 y = pair_of<kHalf>(v[e].x[f]);
          acc[2 * f] = fmaf(we, y.x, acc[2 * f]);
          acc[2 * f + 1] = fmaf(we, y.y, acc[2 * f + 1]);
        }
      }
    }
  }
  const int64_t out_row = t * p.q_heads + h;
  const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
  Words<D> y;
#pragma unroll
  for (int f = 0; f < kWords; ++f)
    y.x[f] = kv4::pack_pair(acc[2 * f] * inverse, acc[2 * f + 1] * inverse,
                            kHalf ? DCP_F16 : DCP_BF16);
  *reinterpret_cast<Words<D>*>(static_cast<uint16_t*>(p.out) + out_row * D + 2 * kWords * lane) = y;
  if (lane == 0) p.lse[out_row] = l == 0.0f ? -INFINITY : kLn2 * (r + log2f(l));
}

// What eight values hold that is not finite: bits of the NaN, of the infinities
// (from bit 8 on) and of the negative ones (from bit 16 on).
__device__ __forceinline__ uint32_t marks_of(const uint4& x, uint32_t infinity) {
  const uint32_t words[4] = {x.x, x.y, x.z, x.w};
  uint32_t marks = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t bits = words[e / 2] >> (e % 2 * 16) & 0xFFFF, size = bits & 0x7FFF;
    if (size > infinity) marks |= 1u << e;
    if (size == infinity) marks |= 1u << (e + (bits >> 15 ? 16 : 8));
  }
  return marks;
}
// Whether there are any: the exponent's bits carry into the sign's.
__device__ __forceinline__ bool marked(const uint4& x, uint32_t infinity) {
  const uint32_t add = (0x8000 - infinity) * 0x10001u, size = 0x7FFF7FFFu;
  return (((x.x & size) + add) | ((x.y & size) + add) | ((x.z & size) + add) |
          ((x.w & size) + add)) & 0x80008000u;
}
// The marks that a sum has where its terms have these: NaN by a NaN or by both
// infinities, an infinity by that one.
__device__ __forceinline__ uint32_t explained_by(uint32_t marks) {
  return marks | (marks >> 8 & marks >> 16 & 0xFF);
}

// Which of `rows` (lanes of the warp with row i and head h of the sequence, whose
// output has something that is not finite) have to be computed again, after a
// product over `keys` keys of the sequence from `from` on.  Not those that have only what the values that they see make of them: no value that they
// do not see is infinite or NaN, and all that is not finite in them is explained
// by keys that all the rows see.  (An infinity in the first value of a prompt of
// 2048 rows, 64 heads of 128: 180 us, as all are finite 75; all rows again: 17 ms.)
//
// The warp looks at 4 or more values at a time, 16 bytes to a lane, first at
// those that some row does not see, a few hundred, then at the others until all
// is explained.
template <int D>
__device__ __forceinline__ unsigned unexplained(const Params& p, int first, int n, int from,
                                                int keys, int i, int h, unsigned rows, int* beats) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kLoads = 4;
  const int lane = threadIdx.x & 31, chunk = lane % kLanes, which = lane / kLanes;
  const uint32_t infinity = p.dtype == DCP_BF16 ? 0x7F80u : 0x7C00u;
  const bool mine = rows >> lane & 1;
  const int kv = __shfl_sync(~0u, h, __ffs(rows) - 1) / p.group;
  const int64_t out_row = (int64_t)(first + i) * p.q_heads + h;
  first += from;
  const int lo = p.window ? max(0, i - p.window + 1) - from : 0;  // seen, counted from there
  const int hi = (p.causal ? i + 1 : n) - from;
  keys = min(keys, start_of(p, p.num_seqs) - first);  // those behind are zeros
  const int all_lo = min(__reduce_max_sync(~0u, mine ? lo : 0), keys);
  const int all_hi = max(min(__reduce_min_sync(~0u, mine ? hi : INT32_MAX), keys), all_lo);
  const uint16_t* values = static_cast<const uint16_t*>(p.v) + (int64_t)first * p.v_row_stride +
                           kv * p.v_head_stride + 8 * chunk;
  const uint16_t* out = static_cast<const uint16_t*>(p.out) + 8 * chunk;
  auto load = [&](int j, int end) {
    return j < end ? *reinterpret_cast<const uint4*>(values + j * p.v_row_stride)
                   : make_uint4(0, 0, 0, 0);
  };
  auto out_marks = [&](int r) {  // of a row's output, by other lanes or a copy: not cached here
    const int64_t at = __shfl_sync(~0u, out_row, r) * D;
    return marks_of(__ldcg(reinterpret_cast<const uint4*>(out + at)), infinity);
  };

  bool hidden = false;
  for (int part = 0; part < 2; ++part) {
    const int end = part ? keys : all_lo;
    for (int j = part ? all_hi : 0; j < end; j += kAtOnce * kLoads) {
      uint4 x[kLoads];
#pragma unroll
      for (int e = 0; e < kLoads; ++e) x[e] = load(j + e * kAtOnce + which, end);
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const unsigned bad = __ballot_sync(~0u, marked(x[e], infinity));
        for (int g = 0; bad && g < kAtOnce; ++g) {
          const int key = j + e * kAtOnce + g;
          if (bad >> (g * kLanes) & ((1ull << kLanes) - 1)) hidden |= key < lo || key >= hi;
        }
      }
    }
  }
  unsigned again = __ballot_sync(~0u, mine && hidden);
  unsigned open = rows & ~again;
  uint32_t wanted = 0, marks = 0;
  for (unsigned left = open; left; left &= left - 1) wanted |= out_marks(__ffs(left) - 1);
  for (int j = all_lo; j < all_hi; j += kAtOnce * kLoads) {
    if ((j - all_lo) % 2048 == 0) {
      if (lane == 0) atomicAdd(beats, 1);
      if (!__any_sync(~0u, wanted & ~explained_by(marks))) break;
    }
    uint4 x[kLoads];
#pragma unroll
    for (int e = 0; e < kLoads; ++e) x[e] = load(j + e * kAtOnce + which, all_hi);
    bool some = false;
#pragma unroll
    for (int e = 0; e < kLoads; ++e) some |= marked(x[e], infinity);
    if (!__any_sync(~0u, some)) continue;
    uint32_t found = 0;
#pragma unroll
    for (int e = 0; e < kLoads; ++e) found |= marks_of(x[e], infinity);
#pragma unroll
    for (int d = kLanes; d < 32; d *= 2) found |= __shfl_xor_sync(~0u, found, d);
    marks |= found;
    if (!__any_sync(~0u, wanted & ~explained_by(marks))) break;
  }
  for (; open; open &= open - 1) {
    const int r = __ffs(open) - 1;
    if (__any_sync(~0u, out_marks(r) & ~explained_by(marks))) again |= 1u << r;
  }
  return again;
}

// Computes again what has to be of the warp's rows: all of `anyway`, and those of
// `rows` that unexplained() names.
template <int D, bool kHalf>
__device__ __noinline__ void attend_again(const Params& p, int first, int n, int from, int keys,
                                          int i, int h, unsigned rows, unsigned anyway,
                                          int* beats) {
  if (rows) anyway |= unexplained<D>(p, first, n, from, keys, i, h, rows, beats);
  for (; anyway; anyway &= anyway - 1) {
    const int r = __ffs(anyway) - 1;
    attend_row<D, kHalf>(p, first, n, __shfl_sync(~0u, i, r), __shfl_sync(~0u, h, r), beats);
  }
}

}  // namespace prompt
}  // namespace dcp
