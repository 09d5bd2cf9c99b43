// kv4_shares.cuh -- attention of long rows and of rows of different lengths: the
// tiles of all rows in one line, cut into an equal share for each CTA that fits
// on the GPU.  A share's first and last row may be pieces of a row: those go to
// the workspace, and a second kernel joins them.
//
// The key/value heads of a row are walked together, up to 8 at a time, by
// kWarps / together warps each: a token's rows of neighbouring heads are neighbours
// in memory, and DRAM serves 128 bytes at a time.  Walked one after the other,
// 131072 tokens of 8 heads with 64-byte rows read 2.2 times their bytes.
//
// Measured (8 heads x 128, 8 query heads each): 256 rows of 64 to 8192 tokens
// 213 us, 5.8 TB/s, 85% of the measured copy rate (see kv4_pages.cuh).  16 rows
// of 1 to 16384 tokens 39 us, two of 100003 and 131072 58 us: there 7 go by before
// the first tile has landed, 3 to 5 between the median CTA's end and the last one's,
// 4 to 6 in the join.
//
// Measured and not taken: one producer warp that copies a token's rows of all
// heads in bulk (cp.async.bulk, 4 a token): about 60 cycles a copy, 983 us
// against 271 us for 256 rows of up to 8192 tokens.
#pragma once

#include <type_traits>

#include "kv4_pages.cuh"

namespace dcp {
namespace kv4 {

// 8 warps to a CTA.  One CTA of 16 warps per SM halves the number of pieces,
// but nothing then runs while it drains: 259 us against 237 for 256 rows of up
// to 8192 tokens.
template <int D, int NT>
struct ShareShape {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = RingShape<D, NT>::kWarpsPerSm / kWarps;
  static constexpr int kTeam = TeamStage<D>::kTeam;
  static constexpr int kRings = kWarps * RingShape<D, NT>::kBytes;
  static constexpr int kTeams = kWarps / kTeam * TeamShape<D, NT>::kBytes;
  static constexpr int kSmem = D < 256 && kTeams > kRings ? kTeams : kRings;
  // a warp's sums on their way to another: outputs, references, sums
  static constexpr int kStateWords = NT * (D / 16 * 4 + 4);
  static constexpr int kExchange = kWarps / 2 * kStateWords * 32 * 4;
  static_assert(kExchange <= kSmem && kExchange <= PageStage<D, 4>::kRings,
                "in the ring's place");
};
constexpr int kMostTogether = 8;  // key/value heads

// The line of tiles: rows in order, in a row its units (groups of `together`
// key/value heads, times head tiles), in a unit its tiles; a row that sees
// nothing has one (empty) tile per unit, so that its outputs are written.
// A unit's tiles are preceded by kPieceTiles places without one, for what its
// beginning costs: its share is that much shorter.  Share c is the places
// [c * per, (c + 1) * per).
//
// For the join, of a share: its last piece, if that is the first of a unit that
// later shares go on with: x = row, y = unit, z = the last of those shares (0:
// no such piece).  And of a unit, where there are few: its first and last share
// (the same: nothing to join).
struct Share {
  int t, unit, at;  // where it begins
  int left, per;    // its places, and those of a full share (host-checked: they fit)
};
constexpr int kPieceTiles = 2;

// How a share walks its tiles: with a ring per warp, in teams, or in groups of
// kWalk >= kByPages warps, for caches of as many heads (kv4_pages.cuh).
constexpr int kByRing = 0, kByTeam = 1, kByPages = 2;

// A row as shares walk it: in groups from a multiple of 8 on.
template <bool kIds, int kWalk>
__device__ __forceinline__ RowSpan share_span(const AttentionParams& p, int t) {
  RowSpan r = row_span<kIds>(p, t);
  if constexpr (kWalk >= kByPages) {
    if (r.n > 0) r.skip = r.start & 7;
    r.start -= r.skip, r.n += r.skip;
  }
  return r;
}

__device__ __forceinline__ int places_of(const RowSpan& r) {
  return kPieceTiles + max(1, (int)(((int64_t)r.n + kTile - 1) / kTile));
}

// This CTA's share, by prefix sums of the rows' places, each thread a run of
// rows.  Barriers: the whole CTA takes part.
template <bool kIds, int kWalk, int kWarps>
__device__ __forceinline__ Share find_share(const AttentionParams& p, int units, int of) {
  __shared__ long long warp_sum[kWarps];
  __shared__ Share share;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kThreads = 32 * kWarps;
  const int run = (p.rows + kThreads - 1) / kThreads;
  const int row0 = min(p.rows, (int)threadIdx.x * run), row1 = min(p.rows, row0 + run);
  long long own = 0;
  for (int t = row0; t < row1; ++t) own += places_of(share_span<kIds, kWalk>(p, t));
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
  const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)(kPieceTiles + of));
  const long long x0 = min(total, blockIdx.x * per), x1 = min(total, x0 + per);
  if (x0 == x1 && threadIdx.x == 0) share = Share{0, 0, 0, 0, (int)per};
  if (x0 < x1 && before * units <= x0 && x0 < (before + own) * units) {
    for (int t = row0;; ++t) {
      const int n = places_of(share_span<kIds, kWalk>(p, t));
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

template <int D, int NT, bool kIds, int kWalk>
__global__ void __launch_bounds__(ShareShape<D, NT>::kThreads, ShareShape<D, NT>::kPerSm)
    attention_shares_kernel(const __grid_constant__ AttentionParams p) {
  using Shape = ShareShape<D, NT>;
  constexpr int kMTiles = D / 16, kStateWords = Shape::kStateWords;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int groups = (p.c.heads + p.together - 1) / p.together;
  const int of = Shape::kWarps / (kWalk >= kByPages ? kWalk : p.together);  // warps of a head
  // this warp's head of the group and its turn; the warps of a team have
  // neighbouring heads and the same turn
  constexpr int kMembers = kWalk == kByTeam ? Shape::kTeam : 1;
  const int rest = warp / kMembers;
  const int head = rest / of * kMembers + warp % kMembers, sub = rest % of;
  if constexpr (kWalk >= kByPages) begin_pages<D, kWalk>(smem);
  uint32_t walked = 0;  // kByPages: tiles of this warp's group
  grid_dependency_wait();
  Share s = find_share<kIds, kWalk, Shape::kWarps>(p, groups * p.head_tiles, of);

  int4 record = make_int4(0, 0, 0, 0);
  while (s.left > 0) {
    const RowSpan r = share_span<kIds, kWalk>(p, s.t);
    // this share's places of the unit: [s.at, to), tile i at kPieceTiles + i
    const int places = places_of(r), to = min(places - s.at, s.left) + s.at;
    const int tiles = places - kPieceTiles;
    const int tile0 = max(0, s.at - kPieceTiles), tile1 = max(0, to - kPieceTiles);
    if (tile1 == tile0) break;  // the share's end, and not a tile of the unit
    const int h = s.unit % groups * p.together + head, ht = s.unit / groups;
    const bool active = h < p.c.heads;
    const int heads = active ? min(8 * NT, p.group - ht * 8 * NT) : 0;  // query heads
    const int head0 = h * p.group + ht * 8 * NT;
    Heads<D, NT> hd;
    if constexpr (kWalk >= kByPages)
      attend_pages<D, NT, kWalk>(p, r, s.t, head, head0, heads, tile0, tile1, sub, smem, walked,
                                 hd);
    else if constexpr (kWalk == kByTeam)
      attend_team<D, NT, kIds>(p, r, s.t, h - warp % kMembers,
                               min(kMembers, p.c.heads - (h - warp % kMembers)), warp % kMembers,
                               active, head0, heads, tile0, tile1, sub, of, smem, hd);
    else
      attend_tiles<D, NT, kIds>(p, r, s.t, active ? h : 0, head0, heads, tile0,
                                active ? tile1 : tile0, sub, of, smem, hd);

    // the warps of a head add up in halves, in the ring's place
    float* sums = reinterpret_cast<float*>(smem);
    if (of > 1) __syncthreads();  // every warp has read its ring
    for (int step = of >> 1; step > 0; step >>= 1) {
      float* slot = sums + (head * step + sub % step) * kStateWords * 32 + lane;
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
      // bulk copies come here next
      if constexpr (kWalk >= kByPages) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }

    const bool whole = tile0 == 0 && tile1 == tiles;
    if (tile0 == 0) {
      const int last = (int)blockIdx.x + (places - to + s.per - 1) / s.per;
      if (!whole) record = make_int4(s.t, s.unit, last, 0);
      if (p.cuts && threadIdx.x == 0)
        p.cuts[(int64_t)s.t * groups * p.head_tiles + s.unit] = make_int2((int)blockIdx.x, last);
    }
    if (sub == 0) {
      // what the CTA gave up on; late copies may have hit the warps' sums, too
      bool lost = false;
      if constexpr (kWalk >= kByPages) lost = *gave_up<D, kWalk>(smem);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = lost ? __int_as_float(0x7fffffff) : hd.l[n][c];
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
    s.left -= to - s.at;
    s.at = 0;
    if (++s.unit == groups * p.head_tiles) s.unit = 0, ++s.t;
  }
  if (threadIdx.x == 0) p.shares[blockIdx.x] = record;
  if constexpr (kWalk >= kByPages) end_pages<D, kWalk>(smem);
}

// Joins the pieces of a unit that shares cut.  kByUnit: a CTA per unit and
// query head (few units of many pieces), its warps dealt the pieces.  Otherwise
// a CTA per share (for the unit whose first piece is the share's last) and 8
// query heads, a warp each.  A lane holds D / 32 contiguous elements; a piece's
// outputs are loaded together with its reference, a batch of pieces at a time.
constexpr int kJoinWarps = 8;
constexpr int kLeastJoinWarps = 4, kMostJoinWarps = 32;  // of a CTA, kByUnit

template <int D, int NT, bool kByUnit>
__global__ void __launch_bounds__(32 * (kByUnit ? kMostJoinWarps : kJoinWarps))
    join_shares_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kPer = D / 32;
  __shared__ float red[kByUnit ? kMostJoinWarps : 1][D];
  __shared__ float2 red_ml[kByUnit ? kMostJoinWarps : 1];
  const int ways = kByUnit ? blockDim.x / 32 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.c.heads + p.together - 1) / p.together;
  const int units = groups * p.head_tiles;
  const int q = kByUnit ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
  const int kv = q / (8 * NT), head = q % (8 * NT);
  grid_dependency_wait();
  int t, unit, c, last;
  if constexpr (kByUnit) {
    const int2 cut = p.cuts[blockIdx.x];
    t = blockIdx.x / units, unit = blockIdx.x % units;
    c = cut.x, last = cut.y;
  } else {
    const int4 record = p.shares[blockIdx.x];
    t = record.x, unit = record.y;
    c = blockIdx.x, last = max(c, record.z);
  }
  if (last == c) return;  // one share walked the whole unit
  const int h = unit % groups * p.together + kv, ht = unit / groups;
  // the whole CTA with kByUnit, else this warp (no barrier follows)
  if (ht * 8 * NT + head >= p.group || h >= p.c.heads) return;
  auto piece = [&](int i) {
    return (((int64_t)2 * i + (i == c)) * p.together + kv) * 8 * NT + head;
  };
  // this warp's pieces, the references of up to 32 at a time in its lanes
  Joined j{kNoScore, 0.0f, 0.0f, 0.0f};
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.0f;
  constexpr int kBatch = kByUnit && D < 256 ? 4 : 2;  // pieces
  using Row = typename std::conditional<kPer == 2, float2, float4>::type;
  constexpr int kRows = kPer * 4 / (int)sizeof(Row);
  for (int i0 = c + (kByUnit ? warp : 0); i0 <= last; i0 += 32 * ways) {
    const int count = min(32, (last - i0) / ways + 1);
    const int mine = i0 + lane * ways;
    Row w[kBatch][kRows];
    auto load = [&](int k0) {  // beyond the last piece: that once more, times 0
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + min(k0 + k, count - 1) * ways;
        const float* src = p.part_out + piece(i) * D + lane * kPer;
#pragma unroll
        for (int e = 0; e < kRows; ++e) w[k][e] = reinterpret_cast<const Row*>(src)[e];
      }
    };
    load(0);
    const float2 ml = mine <= last ? p.part_ml[piece(mine)] : make_float2(kNoScore, 0.0f);
    float top = ml.x;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, j.top);
    const float scale = exp2_approx(j.top - top);
    const float f = mine <= last ? exp2_approx(ml.x - top) : 0.0f;
    j.top = top;
    j.sum = j.sum * scale + f * ml.y;  // of this lane's pieces
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= scale;
    for (int k0 = 0;;) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k0 + k);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          acc[e] += fk * reinterpret_cast<const float*>(w[k])[e];
      }
      k0 += kBatch;
      if (k0 >= count) break;
      load(k0);
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) j.sum += __shfl_xor_sync(0xffffffffu, j.sum, x);
  const int64_t at = (int64_t)t * p.q_heads + h * p.group + ht * 8 * NT + head;
  if constexpr (kByUnit) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) red[warp][lane * kPer + e] = acc[e];
    if (lane == 0) red_ml[warp] = make_float2(j.top, j.sum);
    __syncthreads();
    j = Joined{kNoScore, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < ways; ++w) j.top = fmaxf(j.top, red_ml[w].x);
    for (int d = 2 * threadIdx.x; d < D; d += 2 * blockDim.x) {
      j.sum = j.x = j.y = 0.0f;
#pragma unroll 4
      for (int w = 0; w < ways; ++w) {
        const float f = exp2_approx(red_ml[w].x - j.top);
        j.sum += f * red_ml[w].y;
        j.x += f * red[w][d];
        j.y += f * red[w][d + 1];
      }
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
