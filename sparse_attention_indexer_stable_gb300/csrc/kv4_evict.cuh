// kv4_evict.cuh -- choosing the tokens that a sequence keeps, and copying them.
//
// Choice: the budget - sinks - recent largest weights of the middle, ties to
// the lowest position, as a set in position order, so nothing is sorted.  A
// cluster of CTAs takes a sequence, each CTA a slice of it and each thread 16
// weights in a row.  Four digit histograms (8 bits) of order-preserving 32-bit
// keys, added over the cluster through distributed shared memory, give the
// smallest kept key and how many of its ties stay; counts per thread then give
// every kept token its place.  Bound by the latency of its passes: with 32
// copies of a histogram, one for each lane, no two lanes of a warp meet (equal
// weights are common, and shared-memory atomics on one address follow one
// another); 2048 bins in one copy took twice as long, and grouping equal lanes
// first (__match_any_sync) longer still.
//
// Copy: a warp per four kept tokens, their loads together.  Bound by memory.
//
// Measured (8 heads x 128): 131072 tokens to 8192 25 us, of which the choice
// takes 18: four passes of about 5000 cycles, of which 1100 are the cluster's
// barrier and 1000 the loads from the other CTAs.  32 sequences of 3000 to
// 16384 tokens to 4096 66 us, of which the copy takes 45 at 6.7 TB/s.
#pragma once

#include <cooperative_groups.h>

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 256;
constexpr int kSelKeys = 16;     // weights of a thread at a time
constexpr int kSelMostCtas = 8;  // of a cluster
constexpr int kSelRound = kSelThreads * kSelKeys;

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
  union {
    uint32_t hist[kSelBins][32];  // a copy for each lane
    uint16_t list[kSelRound];     // a round's kept weights, by their place in the round
  };
  uint32_t sums[4][kSelBins];    // the CTA's histogram, one per pass: others may still read one
  uint32_t warp_sum[kSelWarps], warp_eq[kSelWarps];
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

// Keys of the weights [at, at + 16) of a row; beyond [lo, hi) none (bit i of
// the result: key i counts).
__device__ __forceinline__ uint32_t load_keys(const float* w, int64_t at, int lo, int hi, bool vec,
                                              uint32_t (&key)[kSelKeys]) {
  if (vec && at >= lo && at + kSelKeys <= hi) {
    float4 x[kSelKeys / 4];
#pragma unroll
    for (int i = 0; i < kSelKeys / 4; ++i)
      x[i] = __ldg(reinterpret_cast<const float4*>(w + at) + i);
#pragma unroll
    for (int i = 0; i < kSelKeys / 4; ++i) {
      key[4 * i] = weight_key(x[i].x), key[4 * i + 1] = weight_key(x[i].y);
      key[4 * i + 2] = weight_key(x[i].z), key[4 * i + 3] = weight_key(x[i].w);
    }
    return 0xffffu;
  }
  uint32_t in = 0u;
#pragma unroll
  for (int i = 0; i < kSelKeys; ++i) {
    const bool here = at + i >= lo && at + i < hi;
    key[i] = here ? weight_key(__ldg(w + at + i)) : 0u;
    in |= (uint32_t)here << i;
  }
  return in;
}

__global__ void __launch_bounds__(kSelThreads, 1)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  __shared__ SelectState s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ctas;

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

  // The middle [lo, hi): an equal slice for each CTA, whole pieces of 16, in
  // rounds of 16 weights a thread.  One round stays in registers, more are read
  // again in each pass (they are in L2).
  const int lo = p.sinks, hi = n - p.recent;
  const int need = p.budget - p.sinks - p.recent;  // fewer than the middle has
  const int first = lo & ~(kSelKeys - 1);
  const int64_t slice =
      ((int64_t)(hi - first) + (int64_t)ctas * kSelKeys - 1) / ((int64_t)ctas * kSelKeys) * kSelKeys;
  const int rounds = (int)((slice + kSelRound - 1) / kSelRound);
  const int64_t begin = first + rank * slice;
  const int end = (int)min((int64_t)hi, begin + slice);  // of this CTA
  const int64_t mine = begin + (int64_t)tid * kSelKeys;
  const bool vec = ((uintptr_t)w & 15u) == 0;
  uint32_t key[kSelKeys];
  uint32_t in = 0u;
  auto load = [&](int round) {
    in = load_keys(w, mine + (int64_t)round * kSelRound, lo, end, vec, key);
  };
  if (need > 0) load(0);

  uint32_t prefix = 0u, left = (uint32_t)need;
#pragma unroll 1
  for (int pass = 0; pass < 4 && need > 0; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < kSelBins * 32 / 4; i += kSelThreads)
      reinterpret_cast<uint4*>(&s.hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
      if (!__any_sync(0xffffffffu, in != 0u)) continue;
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        // the digits before this one agree (none before the first)
        const bool take = ((in >> i) & 1u) && (((key[i] ^ prefix) >> shift) >> 8) == 0u;
        if (take) atomicAdd(&s.hist[(key[i] >> shift) & 255u][lane], 1u);
      }
    }
    __syncthreads();
    // the 32 copies: a warp per bin
#pragma unroll
    for (int i = 0; i < kSelBins / kSelWarps; ++i) {
      const int bin = i * kSelWarps + warp;
      const uint32_t sum = __reduce_add_sync(0xffffffffu, s.hist[bin][lane]);
      if (lane == 0) s.sums[pass][bin] = sum;
    }
    cluster.sync();
    // over the cluster, a thread per bin in descending order; the first warps
    uint32_t h = 0u, incl = 0u;
    if (tid < kSelBins) {
#pragma unroll
      for (int c = 0; c < kSelMostCtas; ++c)
        if (c < ctas) h += *cluster.map_shared_rank(&s.sums[pass][kSelBins - 1 - tid], c);
      incl = warp_scan(h, lane);
      if (lane == 31) s.warp_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < kSelBins) {
      uint32_t before = incl - h;
      for (int v = 0; v < warp; ++v) before += s.warp_sum[v];
      if (before < left && left <= before + h)
        s.digit = (uint32_t)(kSelBins - 1 - tid), s.above = before;
    }
    __syncthreads();
    prefix |= s.digit << shift;
    left -= s.above;
  }
  // `prefix` is the smallest kept key, `left` how many of its ties are kept

  if (need > 0) {
    // how many above it and how many ties: this thread's, the CTA's
    auto count = [&](uint32_t& gt, uint32_t& eq) {
      gt = eq = 0u;
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        gt += ((in >> i) & 1u) && key[i] > prefix;
        eq += ((in >> i) & 1u) && key[i] == prefix;
      }
    };
    uint32_t gt, eq, sum_gt = 0u, sum_eq = 0u;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round);
      count(gt, eq);
      sum_gt += gt, sum_eq += eq;
    }
    sum_gt = __reduce_add_sync(0xffffffffu, sum_gt);
    sum_eq = __reduce_add_sync(0xffffffffu, sum_eq);
    __syncthreads();  // warp_sum has been read
    if (lane == 0) s.warp_sum[warp] = sum_gt, s.warp_eq[warp] = sum_eq;
    __syncthreads();
    if (warp == 0) {
      sum_gt = __reduce_add_sync(0xffffffffu, s.warp_sum[lane]);
      sum_eq = __reduce_add_sync(0xffffffffu, s.warp_eq[lane]);
      if (lane == 0) s.cta_gt = sum_gt, s.cta_eq = sum_eq;
    }
    cluster.sync();
    uint32_t base_gt = 0u, base_eq = 0u;  // before this CTA, then before this round
#pragma unroll
    for (int c = 0; c < kSelMostCtas; ++c)
      if (c < rank) {
        base_gt += *cluster.map_shared_rank(&s.cta_gt, c);
        base_eq += *cluster.map_shared_rank(&s.cta_eq, c);
      }
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) {
        load(round);
        count(gt, eq);
      }
      const uint32_t incl_gt = warp_scan(gt, lane), incl_eq = warp_scan(eq, lane);
      __syncthreads();  // the last round's sums have been read
      if (lane == 31) s.warp_sum[warp] = incl_gt, s.warp_eq[warp] = incl_eq;
      __syncthreads();
      const uint32_t warps_gt = warp_scan(s.warp_sum[lane], lane);
      const uint32_t warps_eq = warp_scan(s.warp_eq[lane], lane);
      uint32_t at_gt = base_gt + incl_gt - gt, at_eq = base_eq + incl_eq - eq;
      const uint32_t before_gt = __shfl_sync(0xffffffffu, warps_gt, (warp + 31) & 31);
      const uint32_t before_eq = __shfl_sync(0xffffffffu, warps_eq, (warp + 31) & 31);
      if (warp > 0) at_gt += before_gt, at_eq += before_eq;
      // The round's kept ones into a list, and from there to the outputs: side
      // by side, where the threads' own places would scatter.
      const uint32_t base = base_gt + min(base_eq, left);
      base_gt += __shfl_sync(0xffffffffu, warps_gt, 31);
      base_eq += __shfl_sync(0xffffffffu, warps_eq, 31);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) {
        const bool above = ((in >> i) & 1u) && key[i] > prefix;
        const bool tie = ((in >> i) & 1u) && key[i] == prefix;
        if (above || (tie && at_eq < left))
          s.list[at_gt + min(at_eq, left) - base] = (uint16_t)(tid * kSelKeys + i);
        at_gt += above;
        at_eq += tie;
      }
      __syncthreads();
      const int count_kept = (int)(base_gt + min(base_eq, left) - base);
      const int64_t from = begin + (int64_t)round * kSelRound;
      for (int j = tid; j < count_kept; j += kSelThreads) {
        const int64_t pos = from + s.list[j];
        kept[p.sinks + base + j] = (int32_t)pos;
        out_w[p.sinks + base + j] = __ldg(w + pos);
      }
    }
  }
  for (int j = all; j < p.sinks; j += stride) kept[j] = j, out_w[j] = w[j];
  for (int j = all; j < p.recent; j += stride) {
    kept[p.budget - p.recent + j] = n - p.recent + j;
    out_w[p.budget - p.recent + j] = w[n - p.recent + j];
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

constexpr int kCopy = 4;  // tokens of a warp

// Rows of the K and V planes of one kind (those that are live; zeros for a
// source that is not there), all loads before the stores.
template <typename Piece>
__device__ __forceinline__ void copy_rows(uint8_t* k_plane, uint8_t* v_plane,
                                          const uint64_t (&dst)[kCopy],
                                          const uint64_t (&src)[kCopy], unsigned live,
                                          unsigned there, int bytes, int lane) {
  for (int i = lane; i < bytes / (int)sizeof(Piece); i += 32) {
    Piece x[kCopy] = {}, y[kCopy] = {};
#pragma unroll
    for (int k = 0; k < kCopy; ++k)
      if ((there >> k) & 1u) {
        x[k] = reinterpret_cast<const Piece*>(k_plane + src[k] * (uint64_t)bytes)[i];
        y[k] = reinterpret_cast<const Piece*>(v_plane + src[k] * (uint64_t)bytes)[i];
      }
#pragma unroll
    for (int k = 0; k < kCopy; ++k)
      if ((live >> k) & 1u) {
        reinterpret_cast<Piece*>(k_plane + dst[k] * (uint64_t)bytes)[i] = x[k];
        reinterpret_cast<Piece*>(v_plane + dst[k] * (uint64_t)bytes)[i] = y[k];
      }
  }
}

__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)p.num_seqs * p.budget;
  const int64_t item0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kCopy;
  grid_dependency_wait();
  // the first lanes look a token up each
  uint64_t from = 0, to = 0;
  bool ok = false, found = false;
  if (lane < kCopy && item0 + lane < items) {
    const int64_t item = item0 + lane;
    const int pos = p.kept[item];
    if (pos >= 0) {
      const int b = (int)(item / p.budget), j = (int)(item - (int64_t)b * p.budget);
      const int shift = p.c.page_shift, low = (1 << shift) - 1;
      const uint32_t page = (uint32_t)__ldg(p.table + (int64_t)b * p.table_stride + (pos >> shift));
      const uint32_t out = (uint32_t)__ldg(p.out_table + (int64_t)b * p.out_table_stride +
                                           (j >> shift));
      ok = out < p.c.num_pages;  // else a hole
      found = ok && page < p.c.num_pages;  // a hole's token reads as zeros
      from = ((uint64_t)page << shift) | (uint32_t)(pos & low);
      to = ((uint64_t)out << shift) | (uint32_t)(j & low);
    }
  }
  const unsigned live = __ballot_sync(0xffffffffu, ok);
  const unsigned there = __ballot_sync(0xffffffffu, found);
  if (!live) return;
  uint64_t src[kCopy], dst[kCopy];
#pragma unroll
  for (int k = 0; k < kCopy; ++k) {
    src[k] = __shfl_sync(0xffffffffu, from, k);
    dst[k] = __shfl_sync(0xffffffffu, to, k);
  }
  copy_rows<uint32_t>(p.c.k_scales, p.c.v_scales, dst, src, live, there, p.row_scales,
                      lane);
  copy_rows<uint4>(p.c.k_codes, p.c.v_codes, dst, src, live, there, p.row_codes, lane);
}

}  // namespace kv4
}  // namespace dcp
