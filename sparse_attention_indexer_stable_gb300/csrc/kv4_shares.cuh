// kv4_shares.cuh -- attention of long rows and of rows of different lengths: the
// tiles of all rows in one line, cut into an equal share for each CTA that fits
// on the GPU.  A share's first and last row may be pieces of a row: those go to
// the workspace, and a second kernel joins them.
//
// The key/value heads of a row are walked together, up to 8 at a time, by
// 8 / together warps each: a token's rows of neighbouring heads are neighbours
// in memory, and DRAM serves 128 bytes at a time.  Walked one after the other,
// 131072 tokens of 8 heads with 64-byte rows read 2.2 times their bytes.
//
// Measured and not taken: one producer warp that copies a token's rows of all
// heads in bulk (cp.async.bulk, 4 a token): about 60 cycles a copy, 983 us
// against 271 us for 256 rows of up to 8192 tokens.
#pragma once

#include "kv4_ring.cuh"

namespace dcp {
namespace kv4 {

// The line of tiles: rows in order, in a row its units (groups of `together`
// key/value heads, times head tiles), in a unit its tiles; a row that sees
// nothing has one (empty) tile per unit, so that its outputs are written.
// Share c is tiles [c * per, (c + 1) * per).
//
// Record of a share, for the join: its last piece, if that is the first of a
// unit that later shares go on with: x = row, y = unit, z = the last of those
// shares (0: no such piece).
struct Share {
  int t, unit, tile0;  // where it begins
  int left, per;       // its tiles, and those of a full share (host-checked: they fit)
};

__device__ __forceinline__ int tiles_of(const RowSpan& r) {
  return max(1, (int)(((int64_t)r.n + kTile - 1) / kTile));
}

// This CTA's share, by prefix sums of the rows' tiles, each thread a run of
// rows.  Barriers: the whole CTA takes part.
template <bool kIds>
__device__ __forceinline__ Share find_share(const AttentionParams& p, int units, int of) {
  __shared__ long long warp_sum[kWarps];
  __shared__ Share share;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = (p.rows + kThreads - 1) / kThreads;
  const int row0 = min(p.rows, (int)threadIdx.x * run), row1 = min(p.rows, row0 + run);
  long long own = 0;
  for (int t = row0; t < row1; ++t) own += tiles_of(row_span<kIds>(p, t));
  long long incl = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - own, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= units;
  // at least a tile for each of a head's warps
  const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)of);
  const long long x0 = min(total, blockIdx.x * per), x1 = min(total, x0 + per);
  if (x0 == x1 && threadIdx.x == 0) share = Share{0, 0, 0, 0, (int)per};
  if (x0 < x1 && before * units <= x0 && x0 < (before + own) * units) {
    for (int t = row0;; ++t) {
      const int n = tiles_of(row_span<kIds>(p, t));
      if (x0 < (before + n) * units) {
        const int unit = (int)((x0 - before * units) / n);
        share = Share{t, unit, (int)(x0 - before * units - (long long)unit * n), (int)(x1 - x0),
                      (int)per};
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  return share;
}

template <int D, int NT, bool kIds>
__global__ void __launch_bounds__(kThreads, RingShape<D, NT>::kCtasPerSm)
    attention_shares_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kMTiles = D / 16;
  // a warp's sums on their way to another: outputs, references, sums
  constexpr int kStateWords = NT * (kMTiles * 4 + 4);
  static_assert(kWarps / 2 * kStateWords * 32 * 4 <= RingShape<D, NT>::kSmem, "fits the ring");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int groups = (p.c.heads + p.together - 1) / p.together;
  const int of = kWarps / p.together;           // warps of a head
  const int head = warp / of, sub = warp % of;  // this warp's head of the group, its turn
  grid_dependency_wait();
  Share s = find_share<kIds>(p, groups * p.head_tiles, of);

  int4 record = make_int4(0, 0, 0, 0);
  while (s.left > 0) {
    const RowSpan r = row_span<kIds>(p, s.t);
    const int tiles = tiles_of(r), tile0 = s.tile0, tile1 = min(tiles - tile0, s.left) + tile0;
    const int h = s.unit % groups * p.together + head, ht = s.unit / groups;
    const bool active = h < p.c.heads;
    const int heads = active ? min(8 * NT, p.group - ht * 8 * NT) : 0;  // query heads
    const int head0 = h * p.group + ht * 8 * NT;
    Heads<D, NT> hd;
    attend_tiles<D, NT, kIds>(p, r, s.t, active ? h : 0, head0, heads, tile0,
                              active ? tile1 : tile0, sub, of, smem, hd);

    // the warps of a head add up in halves, in the ring's place
    float* state = reinterpret_cast<float*>(smem);
    if (of > 1) __syncthreads();  // every warp has read its ring
    for (int step = of >> 1; step > 0; step >>= 1) {
      float* slot = state + (head * step + sub % step) * kStateWords * 32 + lane;
      if (sub >= step && sub < 2 * step) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* w = slot + n * (kMTiles * 4 + 4) * 32;
#pragma unroll
          for (int c = 0; c < 2; ++c) w[c * 32] = hd.m[n][c], w[(2 + c) * 32] = hd.l[n][c];
#pragma unroll
          for (int i = 0; i < kMTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[(4 + 4 * i + e) * 32] = hd.o[n][i][e];
        }
      }
      __syncthreads();
      if (sub < step) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float* w = slot + n * (kMTiles * 4 + 4) * 32;
          float mine[2], theirs[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float other = w[c * 32];
            const float top = fmaxf(hd.m[n][c], other);
            mine[c] = exp2_approx(hd.m[n][c] - top);
            theirs[c] = exp2_approx(other - top);
            hd.m[n][c] = top;
            hd.l[n][c] = hd.l[n][c] * mine[c] + w[(2 + c) * 32] * theirs[c];
          }
#pragma unroll
          for (int i = 0; i < kMTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              hd.o[n][i][e] =
                  hd.o[n][i][e] * mine[e & 1] + w[(4 + 4 * i + e) * 32] * theirs[e & 1];
        }
      }
      __syncthreads();
    }

    const bool whole = tile0 == 0 && tile1 == tiles;
    if (!whole && tile0 == 0)
      record = make_int4(s.t, s.unit, (int)blockIdx.x + (tiles - tile1 + s.per - 1) / s.per, 0);
    if (sub == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = hd.l[n][c];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int q = 8 * n + 2 * tq + c;
          if (q >= heads) continue;
          // D/8 contiguous elements of head q, from g * D/8 on
          if (whole) {
            const int64_t at = (int64_t)s.t * p.q_heads + head0 + q;
            const float inv = write_sum(p, at, hd.m[n][c], sum, g == 0);
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out) + (at * D + g * (D / 8)) / 2;
#pragma unroll
            for (int i = 0; i < kMTiles; i += 4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_pair(hd.o[n][i + e][c] * inv, hd.o[n][i + e][c + 2] * inv, p.dtype);
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            const int64_t at =
                (((int64_t)blockIdx.x * 2 + (tile0 == 0)) * p.together + head) * 8 * NT + q;
            if (g == 0) p.part_ml[at] = make_float2(hd.m[n][c], sum);
            float* dst = p.part_out + at * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < kMTiles; i += 2)
              *reinterpret_cast<float4*>(dst + 2 * i) =
                  make_float4(hd.o[n][i][c], hd.o[n][i][c + 2], hd.o[n][i + 1][c],
                              hd.o[n][i + 1][c + 2]);
          }
        }
    }
    s.left -= tile1 - tile0;
    s.tile0 = 0;
    if (++s.unit == groups * p.head_tiles) s.unit = 0, ++s.t;
  }
  if (threadIdx.x == 0) p.shares[blockIdx.x] = record;
}

// Joins the pieces of a unit that shares cut.  kByUnit: a CTA per unit and
// query head (few units of many pieces), its warps dealt the pieces; the
// unit's first share is found among the records.  Otherwise a CTA per share
// (for the unit whose first piece is the share's last) and 8 query heads, a
// warp each.  A lane holds D / 32 contiguous elements.
constexpr int kJoinWarps = 8;

template <int D, int NT, bool kByUnit>
__global__ void __launch_bounds__(32 * kJoinWarps)
    join_shares_kernel(const __grid_constant__ AttentionParams p, int shares) {
  constexpr int kPer = D / 32;
  constexpr int kWays = kByUnit ? kJoinWarps : 1;
  __shared__ float red[kByUnit ? kJoinWarps : 1][D];
  __shared__ float red_l[kJoinWarps];
  __shared__ int s_share;
  __shared__ int4 s_record;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.c.heads + p.together - 1) / p.together;
  grid_dependency_wait();
  int c = blockIdx.x;
  if constexpr (kByUnit) {
    const int units = groups * p.head_tiles;
    if (threadIdx.x == 0) s_share = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < shares; i += 32 * kJoinWarps) {
      const int4 x = p.shares[i];
      if (x.z && x.x == (int)blockIdx.x / units && x.y == (int)blockIdx.x % units) {
        s_share = i;
        s_record = x;
      }
    }
    __syncthreads();
    c = s_share;
    if (c < 0) return;  // one share walked the whole unit
  }
  const int4 record = kByUnit ? s_record : p.shares[c];
  if (!record.z) return;
  const int q = kByUnit ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
  const int kv = q / (8 * NT), head = q % (8 * NT);
  const int h = record.y % groups * p.together + kv, ht = record.y / groups;
  // the whole CTA with kByUnit, else this warp (no barrier follows)
  if (ht * 8 * NT + head >= p.group || h >= p.c.heads) return;
  const int last = record.z;
  auto piece = [&](int i) {
    return (((int64_t)2 * i + (i == c)) * p.together + kv) * 8 * NT + head;
  };
  Joined j{kNoScore, 0.0f, 0.0f, 0.0f};
  for (int i = c + lane; i <= last; i += 32) j.top = fmaxf(j.top, p.part_ml[piece(i)].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) j.top = fmaxf(j.top, __shfl_xor_sync(0xffffffffu, j.top, x));
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.0f;
#pragma unroll 8
  for (int i = c + (kByUnit ? warp : 0); i <= last; i += kWays) {
    const int64_t at = piece(i);
    const float2 v = p.part_ml[at];
    const float f = exp2_approx(v.x - j.top);
    const float* src = p.part_out + at * D + lane * kPer;
    j.sum += f * v.y;
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float2 w = *reinterpret_cast<const float2*>(src + e);
      acc[e] += f * w.x;
      acc[e + 1] += f * w.y;
    }
  }
  const int64_t at = (int64_t)record.x * p.q_heads + h * p.group + ht * 8 * NT + head;
  if constexpr (kByUnit) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) red[warp][lane * kPer + e] = acc[e];
    if (lane == 0) red_l[warp] = j.sum;
    __syncthreads();
    j.sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) j.sum += red_l[w];
    for (int d = 2 * threadIdx.x; d < D; d += 64 * kJoinWarps) {
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) j.x += red[w][d], j.y += red[w][d + 1];
      write_out<D>(p, at, d, j);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      j.x = acc[e], j.y = acc[e + 1];
      write_out<D>(p, at, lane * kPer + e, j);
    }
  }
}

}  // namespace kv4
}  // namespace dcp
