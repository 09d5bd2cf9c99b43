// kv4_slices.cuh -- attention of short rows: a cluster of 1, 2, 4 or 8 CTAs per
// row and key/value head, each a slice of the row's tiles dealt to its 8 warps,
// joined through distributed shared memory.  One launch, and no workspace but the
// scores where weights are wanted.  Bound by latency: a row of 2048 tokens is one tile per warp and slice, 7 us with 8
// heads x 128 (with slices joined by a second kernel through a workspace 7 us
// too, but 3 us more on the host).  16 rows x 2048 ids take 18 us in teams of
// two heads (kv4_team.cuh) and 24 with a ring per warp: then an SM's L1 takes in
// lines for 16000 cycles (16 warps, 4 tiles of 128 lines, 2 cycles a line), 8 us,
// and in teams for half of that.
#pragma once

#include "kv4_team.cuh"

namespace dcp {
namespace kv4 {

constexpr int kSliceWarps = 8;
constexpr int kSliceThreads = 32 * kSliceWarps;

// A CTA's 8 warps work on one head, or (kTeam) in teams on neighbouring heads.
//
// The join, in the rings' place: each warp's outputs (padded rows), references
// and sums, and behind them the CTA's own for the cluster (16 bytes per output
// pair).
template <int D, int NT, bool kTeam>
struct SliceShape {
  static constexpr int kMembers = kTeam ? TeamStage<D>::kTeam : 1;  // heads
  static constexpr int kRings = kTeam ? kSliceWarps / kMembers * TeamShape<D, NT>::kBytes
                                      : kSliceWarps * RingShape<D, NT>::kBytes;
  static constexpr int kStride = D + 4;
  static constexpr int kWarpBytes = (kSliceWarps * 8 * NT * (kStride + 2) * 4 + 15) & ~15;
  static constexpr int kJoin = kWarpBytes + kMembers * 8 * NT * D / 2 * 16;
  static constexpr int kSmem = kRings > kJoin ? kRings : kJoin;
  static constexpr int kPerSm = RingShape<D, NT>::kWarpsPerSm / kSliceWarps;  // CTAs
  static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Leaves a warp's sums in shared memory (all warps of the CTA: barriers).
template <int D, int NT>
__device__ __forceinline__ void leave_sums(const Heads<D, NT>& hd, uint8_t* smem) {
  using Join = SliceShape<D, NT, false>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  __syncthreads();  // every warp has read its ring
  float* join_o = reinterpret_cast<float*>(smem);
  float* join_m = join_o + kSliceWarps * 8 * NT * Join::kStride;
  float* join_l = join_m + kSliceWarps * 8 * NT;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = hd.l[n][c];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int col = warp * 8 * NT + 8 * n + 2 * tq + c;
      if (g == 0) join_m[col] = hd.m[n][c], join_l[col] = sum;
      float* dst = join_o + col * Join::kStride + g * (D / 8);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(hd.o[n][i][c], hd.o[n][i][c + 2]);
    }
  __syncthreads();
}

// What leave_sums left, added over the warps first, first + step, ...:
// reference, sum and two outputs of `head` at element d.
template <int D, int NT, int kStep>
__device__ __forceinline__ Joined join_warps(const uint8_t* smem, int first, int head, int d) {
  using Join = SliceShape<D, NT, false>;
  const float* join_o = reinterpret_cast<const float*>(smem);
  const float* join_m = join_o + kSliceWarps * 8 * NT * Join::kStride;
  const float* join_l = join_m + kSliceWarps * 8 * NT;
  Joined j{kNoScore, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kSliceWarps; w += kStep)
    j.top = fmaxf(j.top, join_m[(first + w) * 8 * NT + head]);
#pragma unroll
  for (int w = 0; w < kSliceWarps; w += kStep) {
    const int col = (first + w) * 8 * NT + head;
    const float f = exp2_approx(join_m[col] - j.top);
    const float2 v = *reinterpret_cast<const float2*>(join_o + col * Join::kStride + d);
    j.sum += f * join_l[col];
    j.x += f * v.x;
    j.y += f * v.y;
  }
  return j;
}

// blockIdx.x = ((row * head_tiles + head tile) * groups + group) * slices +
// slice; a group is a head, or a team's heads.
template <int D, int NT, bool kIds, bool kTeam>
__global__ void __launch_bounds__(kSliceThreads, SliceShape<D, NT, kTeam>::kPerSm)
    attention_slices_kernel(const __grid_constant__ AttentionParams p) {
  namespace cg = cooperative_groups;
  using Shape = SliceShape<D, NT, kTeam>;
  constexpr int kMembers = Shape::kMembers;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int slices = (int)cluster.num_blocks(), slice = (int)cluster.block_rank();
  const unsigned unit = blockIdx.x / (unsigned)slices;
  const unsigned groups = (unsigned)p.c.heads / kMembers;  // teams: the host divides evenly
  const int h0 = (int)(unit % groups) * kMembers;
  const unsigned rest = unit / groups;
  const int ht = (int)(rest % (unsigned)p.head_tiles);
  const int t = (int)(rest / (unsigned)p.head_tiles);
  const int heads = min(8 * NT, p.group - ht * 8 * NT);  // query heads of each
  const int warp = threadIdx.x >> 5, member = warp % kMembers;
  const int head0 = (h0 + member) * p.group + ht * 8 * NT;  // first query head of this warp

  grid_dependency_wait();
  const RowSpan r = row_span<kIds>(p, t);
  const int tiles = (int)(((int64_t)r.n + kTile - 1) / kTile);
  const int per = (tiles + slices - 1) / slices;
  const int tile0 = min(tiles, slice * per), tile1 = min(tiles, tile0 + per);
  Heads<D, NT> hd;
  if constexpr (kTeam)
    attend_team<D, NT, kIds>(p, r, t, h0, kMembers, member, true, head0, heads, tile0, tile1,
                             warp / kMembers, kSliceWarps / kMembers, smem, hd);
  else
    attend_tiles<D, NT, kIds>(p, r, t, h0, head0, heads, tile0, tile1, warp, kSliceWarps, smem,
                              hd);
  leave_sums<D, NT>(hd, smem);

  // output pairs of the CTA: member, query head, element
  const int pairs = kMembers * heads * (D / 2);
  auto join_pair = [&](int i) {
    const int q = i / (D / 2);
    return join_warps<D, NT, kMembers>(smem, kMembers == 1 ? 0 : q / heads, q % heads,
                                       2 * (i % (D / 2)));
  };
  auto write_pair = [&](int i, const Joined& j) {
    const int q = i / (D / 2);
    const int64_t at = (int64_t)t * p.q_heads + (h0 + q / heads) * p.group + ht * 8 * NT;
    write_out<D>(p, at + q % heads, 2 * (i % (D / 2)), j);
  };
  if (slices == 1) {
    for (int i = threadIdx.x; i < pairs; i += kSliceThreads) write_pair(i, join_pair(i));
    return;
  }
  // The CTA's own join goes behind the warps' (each thread its own values),
  // then every CTA adds its part of the outputs over the cluster.
  Joined* mine = reinterpret_cast<Joined*>(smem + Shape::kWarpBytes);
  for (int i = threadIdx.x; i < pairs; i += kSliceThreads) mine[i] = join_pair(i);
  cluster.sync();
  for (int i = slice * kSliceThreads + threadIdx.x; i < pairs; i += slices * kSliceThreads) {
    Joined j{kNoScore, 0.0f, 0.0f, 0.0f};
    Joined other[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < slices) {
        other[c] = *cluster.map_shared_rank(mine + i, c);
        j.top = fmaxf(j.top, other[c].top);
      }
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < slices) {
        const float f = exp2_approx(other[c].top - j.top);
        j.sum += f * other[c].sum;
        j.x += f * other[c].x;
        j.y += f * other[c].y;
      }
    write_pair(i, j);
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

}  // namespace kv4
}  // namespace dcp
