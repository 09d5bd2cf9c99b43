// kv4_evict.cuh -- choosing the tokens that a sequence keeps, and copying them.
//
// Choice: the budget - sinks - recent largest weights of the middle, ties to
// the lowest position, as a set in position order, so nothing is sorted.  A
// cluster of CTAs takes a sequence, each CTA a slice of the middle: three
// digit histograms (11, 11, 10 bits) of order-preserving 32-bit keys, added
// over the cluster through distributed shared memory, give the smallest kept
// key and how many of its ties stay; counts per warp and CTA then give every
// kept token its place.  Bound by the latency of its passes over weights that
// sit in L2 after the first.
//
// Copy: a warp per four kept tokens, their loads together.  Bound by memory.
#pragma once

#include <cooperative_groups.h>

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 16;     // weights of a thread at a time
constexpr int kSelMostCtas = 8;  // of a cluster

struct EvictParams {
  Planes c;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const float* weights;
  int64_t weights_stride;
  const int32_t* out_table;
  int64_t out_table_stride;
  int32_t* kept;
  int32_t* out_lens;
  float* out_weights;
  int num_seqs, limit, budget, sinks, recent;
  int row_codes;   // bytes of a slot in a code plane
  int row_scales;  // and in a scale plane
};

// Order-preserving map of a weight to 32 bits: -0 equals +0, NaN lies below
// everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t bits = __float_as_uint(w + 0.0f);
  return bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u);
}

struct SelectState {
  uint32_t hist[3][kSelBins];  // one per pass: a CTA may still read one while the next fills
  uint32_t warp_sum[kSelWarps];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t digit, above;
  uint32_t cta_gt, cta_eq;
};

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  return v;  // inclusive
}

__global__ void __launch_bounds__(kSelThreads, 1)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  __shared__ SelectState s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ctas;
  for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&s.hist[0][0])[i] = 0u;

  grid_dependency_wait();
  const int n = max(0, min(__ldg(p.lens + b), p.limit));
  const float* w = p.weights + (int64_t)b * p.weights_stride;
  int32_t* kept = p.kept + (int64_t)b * p.budget;
  float* out_w = p.out_weights + (int64_t)b * p.budget;
  if (rank == 0 && tid == 0) p.out_lens[b] = min(n, p.budget);
  const int all = rank * kSelThreads + tid, stride = ctas * kSelThreads;
  if (n <= p.budget) {  // the whole cluster: n is the sequence's
    for (int j = all; j < p.budget; j += stride) {
      kept[j] = j < n ? j : -1;
      out_w[j] = j < n ? w[j] : 0.0f;
    }
    return;
  }
  for (int j = all; j < p.sinks; j += stride) kept[j] = j, out_w[j] = w[j];
  for (int j = all; j < p.recent; j += stride) {
    kept[p.budget - p.recent + j] = n - p.recent + j;
    out_w[p.budget - p.recent + j] = w[n - p.recent + j];
  }
  const int need = p.budget - p.sinks - p.recent;  // fewer than the middle has
  if (need == 0) return;

  // This CTA's slice of the middle, and this warp's of that: groups of 16
  // weights a lane, 32 apart, loaded together.  A slice of one group per warp
  // stays in registers, a longer one is read again in each pass (it is in L2).
  const int lo = p.sinks, hi = n - p.recent;
  constexpr int kGroup = kSelKeys * 32, kRound = kGroup * kSelWarps;
  const int rounds = ((hi - lo + ctas - 1) / ctas + kRound - 1) / kRound;
  const int64_t warp0 = lo + ((int64_t)rank * kSelWarps + warp) * rounds * kGroup;
  float v[kSelKeys];
  auto load = [&](int round) {
    const int64_t at = warp0 + (int64_t)round * kGroup + lane;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i)
      v[i] = at + 32 * i < hi ? __ldg(w + at + 32 * i) : 0.0f;
  };
  auto in = [&](int round, int i) {
    return warp0 + (int64_t)round * kGroup + 32 * i + lane < hi;
  };
  load(0);
  __syncthreads();  // hist is zero

  uint32_t prefix = 0u, left = (uint32_t)need;
  // digits from the top: bits [21, 32), [10, 21), [0, 10)
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        const uint32_t key = weight_key(v[i]);
        // key >> 32 would be undefined: the first pass takes everything
        const bool take = in(round, i) &&
                          (pass == 0 || (key >> (shift + bits)) == (prefix >> (shift + bits)));
        if (!__any_sync(0xffffffffu, take)) continue;
        // lanes of one bin add up first: accumulated weights tie a lot
        const uint32_t bin = take ? (key >> shift) & ((1u << bits) - 1u) : 0xffffffffu;
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        if (take && lane == __ffs(same) - 1)
          atomicAdd(&s.hist[pass][bin], (uint32_t)__popc(same));
      }
    }
    cluster.sync();
    // bins in descending order, two per thread, added over the cluster
    const int b0 = kSelBins - 2 - 2 * tid;  // and b0 + 1 before it
    uint2 h = make_uint2(0u, 0u);
#pragma unroll
    for (int c = 0; c < kSelMostCtas; ++c)
      if (c < ctas) {
        const uint2 x =
            *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&s.hist[pass][b0], c));
        h.x += x.x, h.y += x.y;
      }
    const uint32_t incl = warp_scan(h.x + h.y, lane);
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    const uint32_t sums = warp_scan(s.warp_sum[lane], lane);
    const uint32_t before_warp = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
    const uint32_t before = (warp ? before_warp : 0u) + incl - (h.x + h.y);
    if (before < left && left <= before + h.y) s.digit = (uint32_t)b0 + 1u, s.above = before;
    if (before + h.y < left && left <= before + h.y + h.x)
      s.digit = (uint32_t)b0, s.above = before + h.y;
    __syncthreads();
    prefix |= s.digit << shift;
    left -= s.above;
    __syncthreads();  // digit and warp_sum have been read
  }
  // `prefix` is the smallest kept key, `left` how many of its ties are kept

  uint32_t gt = 0u, eq = 0u;
  for (int round = 0; round < rounds; ++round) {
    if (rounds > 1) load(round);
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const uint32_t key = weight_key(v[i]);
      gt += __popc(__ballot_sync(0xffffffffu, in(round, i) && key > prefix));
      eq += __popc(__ballot_sync(0xffffffffu, in(round, i) && key == prefix));
    }
  }
  if (lane == 0) s.warp_gt[warp] = gt, s.warp_eq[warp] = eq;
  __syncthreads();
  // this warp's counts of the warps before it, and the CTA's
  const uint32_t gt_to = warp_scan(s.warp_gt[lane], lane), eq_to = warp_scan(s.warp_eq[lane], lane);
  if (warp == 0 && lane == 31) s.cta_gt = gt_to, s.cta_eq = eq_to;
  cluster.sync();
  gt = __shfl_sync(0xffffffffu, gt_to, (warp + 31) & 31);
  eq = __shfl_sync(0xffffffffu, eq_to, (warp + 31) & 31);
  if (warp == 0) gt = eq = 0u;
  uint32_t cta_gt = 0u, cta_eq = 0u;
#pragma unroll
  for (int c = 0; c < kSelMostCtas; ++c)
    if (c < rank) {
      cta_gt += *cluster.map_shared_rank(&s.cta_gt, c);
      cta_eq += *cluster.map_shared_rank(&s.cta_eq, c);
    }
  gt += cta_gt, eq += cta_eq;
  for (int round = 0; round < rounds; ++round) {
    if (rounds > 1) load(round);
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const uint32_t key = weight_key(v[i]);
      const bool here = in(round, i);
      const unsigned is_gt = __ballot_sync(0xffffffffu, here && key > prefix);
      const unsigned is_eq = __ballot_sync(0xffffffffu, here && key == prefix);
      const unsigned below = (1u << lane) - 1u;
      const uint32_t my_eq = eq + __popc(is_eq & below);
      if (here && (key > prefix || (key == prefix && my_eq < left))) {
        const uint32_t at = p.sinks + gt + __popc(is_gt & below) + min(my_eq, left);
        kept[at] = (int32_t)(warp0 + (int64_t)round * kGroup + 32 * i + lane);
        out_w[at] = v[i];
      }
      gt += __popc(is_gt);
      eq += __popc(is_eq);
    }
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

constexpr int kCopy = 4;  // tokens of a warp

// Rows of one plane (those that are live), all loads before the stores.
template <typename Piece>
__device__ __forceinline__ void copy_rows(uint8_t* plane, const uint64_t (&dst)[kCopy],
                                          const uint64_t (&src)[kCopy], unsigned live, int bytes,
                                          int lane) {
  for (int i = lane; i < bytes / (int)sizeof(Piece); i += 32) {
    Piece x[kCopy];
#pragma unroll
    for (int k = 0; k < kCopy; ++k)
      if ((live >> k) & 1u)
        x[k] = reinterpret_cast<const Piece*>(plane + src[k] * (uint64_t)bytes)[i];
#pragma unroll
    for (int k = 0; k < kCopy; ++k)
      if ((live >> k) & 1u) reinterpret_cast<Piece*>(plane + dst[k] * (uint64_t)bytes)[i] = x[k];
  }
}

__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)p.num_seqs * p.budget;
  const int64_t item0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kCopy;
  grid_dependency_wait();
  // the first lanes look a token up each
  uint64_t from = 0, to = 0;
  bool ok = false;
  if (lane < kCopy && item0 + lane < items) {
    const int64_t item = item0 + lane;
    const int pos = p.kept[item];
    if (pos >= 0) {
      const int b = (int)(item / p.budget), j = (int)(item - (int64_t)b * p.budget);
      const int shift = p.c.page_shift, low = (1 << shift) - 1;
      const uint32_t page = (uint32_t)__ldg(p.table + (int64_t)b * p.table_stride + (pos >> shift));
      const uint32_t out = (uint32_t)__ldg(p.out_table + (int64_t)b * p.out_table_stride +
                                           (j >> shift));
      ok = page < p.c.num_pages && out < p.c.num_pages;  // else a hole
      from = ((uint64_t)page << shift) | (uint32_t)(pos & low);
      to = ((uint64_t)out << shift) | (uint32_t)(j & low);
    }
  }
  const unsigned live = __ballot_sync(0xffffffffu, ok);
  if (!live) return;
  uint64_t src[kCopy], dst[kCopy];
#pragma unroll
  for (int k = 0; k < kCopy; ++k) {
    src[k] = __shfl_sync(0xffffffffu, from, k);
    dst[k] = __shfl_sync(0xffffffffu, to, k);
  }
  copy_rows<uint4>(p.c.k_codes, dst, src, live, p.row_codes, lane);
  copy_rows<uint4>(p.c.v_codes, dst, src, live, p.row_codes, lane);
  copy_rows<uint32_t>(p.c.k_scales, dst, src, live, p.row_scales, lane);
  copy_rows<uint32_t>(p.c.v_scales, dst, src, live, p.row_scales, lane);
}

}  // namespace kv4
}  // namespace dcp
