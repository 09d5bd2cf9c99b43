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
// Copy: a warp per kept token, its codes and scales in 16-byte pieces.  Bound
// by memory.
#pragma once

#include <cooperative_groups.h>

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;

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

  // this CTA's slice of the middle, and this warp's of that, in whole warps
  const int lo = p.sinks, hi = n - p.recent;
  const int per_cta = ((hi - lo + ctas - 1) / ctas + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int64_t cta0 = lo + (int64_t)rank * per_cta;
  const int per_warp = per_cta / kSelWarps;
  const int64_t warp0 = cta0 + (int64_t)warp * per_warp;
  const int w0 = (int)min((int64_t)hi, warp0), w1 = (int)min((int64_t)hi, warp0 + per_warp);
  __syncthreads();  // hist is zero

  uint32_t prefix = 0u, left = (uint32_t)need;
  // digits from the top: bits [21, 32), [10, 21), [0, 10)
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t key = weight_key(__ldg(w + i));
      // key >> 32 would be undefined: the first pass takes everything
      const bool in = pass == 0 || (key >> (shift + bits)) == (prefix >> (shift + bits));
      const unsigned active = __activemask();
      const uint32_t bin = in ? (key >> shift) & ((1u << bits) - 1u) : 0xffffffffu;
      const unsigned same = __match_any_sync(active, bin);
      if (in && lane == __ffs(same) - 1) atomicAdd(&s.hist[pass][bin], (uint32_t)__popc(same));
    }
    cluster.sync();
    // bins in descending order, two per thread, added over the cluster
    const int b0 = kSelBins - 1 - 2 * tid;
    uint32_t h0 = 0u, h1 = 0u;
    for (int c = 0; c < ctas; ++c) {
      const uint32_t* other = cluster.map_shared_rank(&s.hist[pass][0], c);
      h0 += other[b0], h1 += other[b0 - 1];
    }
    const uint32_t incl = warp_scan(h0 + h1, lane);
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = 0u;
    for (int v = 0; v < warp; ++v) before += s.warp_sum[v];
    before += incl - (h0 + h1);
    if (before < left && left <= before + h0) s.digit = (uint32_t)b0, s.above = before;
    if (before + h0 < left && left <= before + h0 + h1)
      s.digit = (uint32_t)(b0 - 1), s.above = before + h0;
    __syncthreads();
    prefix |= s.digit << shift;
    left -= s.above;
    __syncthreads();  // digit and warp_sum have been read
  }
  // `prefix` is the smallest kept key, `left` how many of its ties are kept

  uint32_t gt = 0u, eq = 0u;
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t key = in ? weight_key(__ldg(w + i + lane)) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, in && key > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
  }
  if (lane == 0) s.warp_gt[warp] = gt, s.warp_eq[warp] = eq;
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0u, e = 0u;
    for (int v = 0; v < kSelWarps; ++v) a += s.warp_gt[v], e += s.warp_eq[v];
    s.cta_gt = a, s.cta_eq = e;
  }
  cluster.sync();
  gt = eq = 0u;
  for (int c = 0; c < rank; ++c) {
    gt += *cluster.map_shared_rank(&s.cta_gt, c);
    eq += *cluster.map_shared_rank(&s.cta_eq, c);
  }
  for (int v = 0; v < warp; ++v) gt += s.warp_gt[v], eq += s.warp_eq[v];
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const float v = in ? __ldg(w + i + lane) : 0.0f;
    const uint32_t key = weight_key(v);
    const unsigned is_gt = __ballot_sync(0xffffffffu, in && key > prefix);
    const unsigned is_eq = __ballot_sync(0xffffffffu, in && key == prefix);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t my_eq = eq + __popc(is_eq & below);
    if (in && (key > prefix || (key == prefix && my_eq < left))) {
      const uint32_t at = p.sinks + gt + __popc(is_gt & below) + min(my_eq, left);
      kept[at] = i + lane;
      out_w[at] = v;
    }
    gt += __popc(is_gt);
    eq += __popc(is_eq);
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

template <typename Piece>
__device__ __forceinline__ void copy_row(uint8_t* plane, uint64_t dst, uint64_t src, int bytes,
                                         int lane) {
  Piece* d = reinterpret_cast<Piece*>(plane + dst * (uint64_t)bytes);
  const Piece* s = reinterpret_cast<const Piece*>(plane + src * (uint64_t)bytes);
  for (int i = lane; i < bytes / (int)sizeof(Piece); i += 32) d[i] = s[i];
}

__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (item >= (int64_t)p.num_seqs * p.budget) return;
  const int b = (int)(item / p.budget), j = (int)(item - (int64_t)b * p.budget);
  const int pos = p.kept[item];
  if (pos < 0) return;
  const int shift = p.c.page_shift, low = (1 << shift) - 1;
  const uint32_t from = (uint32_t)__ldg(p.table + (int64_t)b * p.table_stride + (pos >> shift));
  const uint32_t to = (uint32_t)__ldg(p.out_table + (int64_t)b * p.out_table_stride + (j >> shift));
  if (from >= p.c.num_pages || to >= p.c.num_pages) return;  // holes
  const uint64_t src = ((uint64_t)from << shift) | (uint32_t)(pos & low);
  const uint64_t dst = ((uint64_t)to << shift) | (uint32_t)(j & low);
  copy_row<uint4>(p.c.k_codes, dst, src, p.row_codes, lane);
  copy_row<uint4>(p.c.v_codes, dst, src, p.row_codes, lane);
  copy_row<uint32_t>(p.c.k_scales, dst, src, p.row_scales, lane);
  copy_row<uint32_t>(p.c.v_scales, dst, src, p.row_scales, lane);
}

}  // namespace kv4
}  // namespace dcp
