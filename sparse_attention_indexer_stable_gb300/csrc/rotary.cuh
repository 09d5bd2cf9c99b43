// rotary.cuh -- rotary positions of queries and keys.
//
// Pair i of a head turns by position * frequency_i.  The frequency is a 64-bit
// fraction of a turn, so position * frequency mod 2^64 is the exact fraction of
// the turn that is left, whatever the position: no 64-bit floating point, no
// reduction of large arguments.  Its nearest quarter is taken off as an
// integer, and the rest, at most an eighth of a turn, keeps a relative 2^-24
// when it becomes a float.
//
// A CTA takes a few tokens and all heads (up to 2^15 pieces of them): cosines and
// sines, once for all heads, into shared memory, then 16-byte pieces, or pairs of
// them, each read and written once.  Memory bounds it, by what is on its way:
// threads with few registers, all 2048 of an SM, do better than threads that load
// ahead.  16384 tokens of 72 heads x 128, bf16: 90 us, 99% of the copy rate; 124
// with a pair, 152 with two pairs loaded before the cosines.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dcp_prompt.h"
#include "kv4_common.cuh"

namespace dcp {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryPairs = 512;  // of a token, at most (dim 1024)

struct RotaryParams {
  const void* in[2];  // q, k
  void* out[2];
  int64_t row_stride[2], head_stride[2], out_row_stride[2], out_head_stride[2];
  const int32_t* positions;
  const uint64_t* turns;
  int64_t tokens;
  int q_heads, heads;  // of q; of q and k
  int pairs, dim;
  int tokens_per_cta, heads_per_cta;
  int turn_items, items;  // pieces of a head: turned, all
  int per_token;          // pieces of a token
  uint32_t by_token, by_head, by_pairs;  // what divides by per_token, items, pairs
  float magnitude;
};

// cos and sin of 2 pi phase / 2^64, times m.
__device__ __forceinline__ float2 turned_by(uint64_t phase, float m) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -x * m : x * m, quarter >= 2 ? -y * m : y * m);
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T x[V];
};

// x / d for x < 2^16 and `by` = ceil(2^32 / d): the product is too large by less
// than x / 2^32, less than the 1 / d that the quotient has left to the next one.
__host__ __device__ constexpr uint32_t division_by(uint32_t d) {
  return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d);
}
__device__ __forceinline__ int divide(int x, uint32_t by) {
  return by ? (int)__umulhi((uint32_t)x, by) : x;
}

// V elements a piece (16 bytes, or one where an address, a stride or a size
// does not allow that).
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 rotary_smem[];  // [tokens_per_cta][V][turn_items]
  using P = Piece<T, V>;
  kv4::grid_dependency_wait();
  const int64_t first = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int here = (int)min((int64_t)p.tokens_per_cta, p.tokens - first);
  for (int i = threadIdx.x; i < here * p.pairs; i += kRotaryThreads) {
    const int t = divide(i, p.by_pairs);
    const uint64_t position = (uint64_t)(int64_t)p.positions[first + t];
    const int pair = i - t * p.pairs;
    rotary_smem[t * p.pairs + pair % V * p.turn_items + pair / V] =
        turned_by(position * p.turns[pair], p.magnitude);
  }
  __syncthreads();
  const int total = here * p.per_token;
  for (int i = threadIdx.x; i < total; i += kRotaryThreads) {
    const int t = divide(i, p.by_token), in_token = i - t * p.per_token;
    const int in_cta = divide(in_token, p.by_head), item = in_token - in_cta * p.items;
    const int h = blockIdx.y * p.heads_per_cta + in_cta;
    if (h >= p.heads) continue;
    const bool key = h >= p.q_heads;
    const int head = key ? h - p.q_heads : h;
    const T* x = static_cast<const T*>(p.in[key]) + (first + t) * p.row_stride[key] +
                 head * p.head_stride[key];
    T* y = static_cast<T*>(p.out[key]) + (first + t) * p.out_row_stride[key] +
           head * p.out_head_stride[key];
    if (item >= p.turn_items) {  // not turned
      const int at = 2 * p.pairs + (item - p.turn_items) * V;
      *reinterpret_cast<P*>(y + at) = *reinterpret_cast<const P*>(x + at);
      continue;
    }
    const float2* cs = rotary_smem + t * p.pairs + item;
    const int at = item * V * (kInterleaved ? 2 : 1);
    const int other = at + (kInterleaved ? V : p.pairs);
    const P a = *reinterpret_cast<const P*>(x + at);
    const P b = *reinterpret_cast<const P*>(x + other);
    P c, d;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // elements 2e and 2e + 1 of the two pieces, or e of each
      constexpr bool kI = kInterleaved;
      const float x0 = to_float(kI ? (2 * e < V ? a.x[2 * e % V] : b.x[2 * e % V]) : a.x[e]);
      const float x1 = to_float(
          kI ? (2 * e + 1 < V ? a.x[(2 * e + 1) % V] : b.x[(2 * e + 1) % V]) : b.x[e]);
      const float2 r = cs[e * p.turn_items];
      const T y0 = from_float<T>(x0 * r.x - x1 * r.y);
      const T y1 = from_float<T>(x1 * r.x + x0 * r.y);
      if constexpr (kI) {
        if (2 * e < V) c.x[2 * e % V] = y0; else d.x[2 * e % V] = y0;
        if (2 * e + 1 < V) c.x[(2 * e + 1) % V] = y1; else d.x[(2 * e + 1) % V] = y1;
      } else {
        c.x[e] = y0;
        d.x[e] = y1;
      }
    }
    *reinterpret_cast<P*>(y + at) = c;
    *reinterpret_cast<P*>(y + other) = d;
  }
}

}  // namespace dcp
