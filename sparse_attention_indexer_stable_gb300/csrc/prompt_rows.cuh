// prompt_rows.cuh -- attention over whole prompts, one row and head to a warp,
// on the plain arithmetic units: for rows that the tensor cores cannot do (see
// prompt_tiles.cuh), about a thousandth of their speed.
//
// With x_j = s_j / ln 2 and a reference r that is a running maximum,
//   l = sum 2^(x_j - r),  out = sum 2^(x_j - r) v_j / l,  lse = ln 2 * (r + log2 l);
// when r grows by d, l and the sum so far are multiplied by 2^-d.  A lane takes
// a key's score, then all lanes take every 32nd element of its value.  Only
// what a row sees is read.
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

// Row t (row i of the sequence that starts at row `first` and has n rows), head
// h, by one warp.  It counts `beats` (see Patience), since a row of many keys takes
// longer than those that wait for it would: one every 256 keys, which take some
// 100 us.
template <int D>
__device__ __forceinline__ void attend_row(const Params& p, int first, int n, int i, int h,
                                           int* beats) {
  const int lane = threadIdx.x & 31;
  const int64_t t = first + i;
  const int kv = h / p.group;
  const int from = p.window ? max(0, i - p.window + 1) : 0, to = p.causal ? i + 1 : n;
  const int64_t q_at = t * p.q_row_stride + h * p.q_head_stride;
  __syncwarp();  // after what other lanes have written to this row
  float acc[D / 32], r = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
  for (int base = from; base < to; base += 32) {
    if ((base - from) % 256 == 0 && lane == 0) atomicAdd(beats, 1);
    const int64_t key = (int64_t)first + base + lane;
    const bool sees = base + lane < to;
    float x = -INFINITY;
    if (sees) {
      float dot = 0.0f;
      const int64_t at = key * p.k_row_stride + kv * p.k_head_stride;
#pragma unroll 16
      for (int e = 0; e < D; ++e)
        dot = fmaf(kv4::load_element(p.q, q_at + e, p.dtype),
                   kv4::load_element(p.k, at + e, p.dtype), dot);
      x = score_of(p, dot);
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
    for (int e = 0; e < D / 32; ++e) acc[e] *= shrink;
    const int count = min(32, to - base);
    for (int j = 0; j < count; ++j) {
      const float wj = __shfl_sync(~0u, w, j);
      const int64_t at = ((int64_t)first + base + j) * p.v_row_stride + kv * p.v_head_stride;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        acc[e] = fmaf(wj, kv4::load_element(p.v, at + lane + 32 * e, p.dtype), acc[e]);
    }
  }
  const int64_t out_row = t * p.q_heads + h;
  const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    const float y = acc[e] * inverse;
    const int64_t at = out_row * D + lane + 32 * e;
    if (p.dtype == DCP_BF16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(y);
  }
  if (lane == 0) p.lse[out_row] = l == 0.0f ? -INFINITY : kLn2 * (r + log2f(l));
}

}  // namespace prompt
}  // namespace dcp
