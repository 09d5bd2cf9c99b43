// kv4_team.cuh -- how a team of warps, each on its own key/value head, brings
// tiles in together.
//
// L1 takes in about one line of a copy every two cycles, whatever part of the
// line is wanted.  A head's row is 32 bytes of codes at dim 64, 64 at dim 128,
// and 4 or 8 of scales: fetched by a warp for its own head, a tile of 32 tokens
// at dim 128 is 128 lines.  The rows of neighbouring heads lie side by side: 4
// or 2 warps whose heads' codes fill a line share a ring, each copying a part
// of the tile's tokens for all of them, 64 lines a warp.  One barrier of the
// team a tile says both that a tile has landed and that the one before it has
// been read.
#pragma once

#include "kv4_ring.cuh"

namespace dcp {
namespace kv4 {

// A stage: 32 rows of 128 bytes of codes of the team's heads and 16 bytes of
// scales, for K and for V.
template <int D>
struct TeamStage {
  static constexpr int kTeam = 256 / D;           // warps, heads
  static constexpr int kTokens = kTile / kTeam;   // that a warp copies
  static constexpr int kChunks = 8 / kTeam;       // 16-byte pieces of a head's row
  static constexpr int kRow = 128, kScale = 16;
  static constexpr int kV = kTile * kRow;
  static constexpr int kKS = 2 * kTile * kRow;
  static constexpr int kVS = kKS + kTile * kScale;
  static constexpr int kMask = kVS + kTile * kScale;
  static constexpr int kBytes = kMask + 16;

  // Where chunk c of row r lies: the lanes that are served at a time touch all
  // banks.  Reading K these are half of the rows r and r + 2 (at dim 64 a
  // quarter of r .. r + 3), reading V^T a quarter of r, r + 1, r + 4, r + 5.
  static __device__ __forceinline__ uint32_t k_at(int r, int c) {
    const int b0 = r & 1, b1 = (r >> 1) & 1;
    return (uint32_t)(r * kRow + (c ^ ((b1 << 2) | (D == 64 ? b0 << 1 : 0))) * 16);
  }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) {
    const int b0 = r & 1, b2 = (r >> 2) & 1;
    return (uint32_t)(r * kRow + (c ^ ((b2 << 2) | (b0 << 1))) * 16);
  }
};

// A thread's operands in a stage (see attend_tile); `head`: of the team's.
template <int D>
struct TeamAt {
  using S = TeamStage<D>;
  const uint8_t *k0, *v0, *ks0, *vs0;
  static constexpr int kSubStep = 16, kHalfStep = 8;  // tokens
  static constexpr bool kRaw = false;
  __device__ void k_read() const {}
  __device__ void v_wait() const {}

  static __device__ __forceinline__ constexpr int token(int i) { return RingAt<D>::token(i); }
  __device__ TeamAt(const uint8_t* stage, int head, int g, int tq) {
    const int c = head * S::kChunks;
    k0 = stage + (D == 64 ? S::k_at(token(g), c + (tq >> 1)) + (tq & 1) * 8
                          : S::k_at(token(g), c + tq));
    v0 = stage + S::kV + S::v_at(token(2 * tq), c + g * (D / 16) / 16) + (g * (D / 16)) % 16;
    ks0 = stage + S::kKS + token(g) * S::kScale + head * (D / 16) + (D == 64 ? tq : 2 * tq);
    vs0 = stage + S::kVS + token(2 * tq) * S::kScale + head * (D / 16) + (D == 64 ? g >> 1 : g);
  }
  __device__ const uint8_t* k(int u, int i) const { return k0 + (16 * u + 8 * i) * S::kRow; }
  __device__ const uint8_t* k_second(int, int) const { return nullptr; }  // dim 256 has no team
  __device__ const uint8_t* k_scale(int u, int i) const {
    return ks0 + (16 * u + 8 * i) * S::kScale;
  }
  __device__ const uint8_t* v(int u, int i) const {
    return v0 + ((i & 1) * 2 + 16 * u + 8 * (i >> 1)) * S::kRow;
  }
  __device__ const uint8_t* v_scale(int u, int i) const {
    return vs0 + ((i & 1) * 2 + 16 * u + 8 * (i >> 1)) * S::kScale;
  }
};

template <int D, int NT>
struct TeamShape {
  static constexpr int kStages = 3;
  static constexpr int kQueue = kStages * TeamStage<D>::kBytes;  // then the warps' ids
  static constexpr int kBytes = kQueue + TeamStage<D>::kTeam * kIdQueue * 32 * 4;  // per team
};

template <int D>
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TeamStage<D>::kTeam) : "memory");
}

// attend_tiles for the warps of a team: key/value heads h0 .. h0 + heads_kv - 1
// (some, or all, may be missing at the end of a row), this warp's being the
// `member`-th; `active`: it is there.
template <int D, int NT, bool kIds>
__device__ __forceinline__ void attend_team(const AttentionParams& p, const RowSpan& r, int t,
                                            int h0, int heads_kv, int member, bool active,
                                            int head0, int heads, int tile0, int tile1, int sub,
                                            int of, uint8_t* smem, Heads<D, NT>& hd) {
  using S = TeamStage<D>;
  using Shape = TeamShape<D, NT>;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int team = (int)(threadIdx.x >> 5) / S::kTeam;
  const int mine = heads_kv > 0 && tile1 - tile0 > sub
                       ? (int)((unsigned)(tile1 - tile0 - sub + of - 1) / (unsigned)of)
                       : 0;
  uint8_t* ring = smem + team * Shape::kBytes;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  const int token0 = member * S::kTokens, my_token = token0 + lane % S::kTokens;
  hd.fetch(p, t, head0, heads);
  Lookup<kIds> look(p, r, t, tile0 + sub, of, my_token,
                    ring + Shape::kQueue + member * kIdQueue * 32 * 4);

  // Copies: chunk lane % 8 of the tokens token0 + lane / 8 + 4i.
  const int chunk = lane & 7, row0 = token0 + (lane >> 3);
  const bool there = chunk < heads_kv * S::kChunks;
  const uint32_t code_stride = (uint32_t)p.c.heads * (D / 2);
  const uint32_t scale_stride = (uint32_t)p.c.heads * (D / 16);
  const uint32_t k_to = S::k_at(row0, chunk), v_to = S::kV + S::v_at(row0, chunk);
  const uint8_t* k_src = p.c.k_codes + (int64_t)h0 * (D / 2) + chunk * 16;
  const uint8_t* v_src = p.c.v_codes + (int64_t)h0 * (D / 2) + chunk * 16;
  // Scales: a lane a token and plane, in one piece where rows of scales are
  // whole 16-byte pieces, else word by word.
  const bool of_v = lane / S::kTokens == 1, scale_lane = lane < 2 * S::kTokens;
  const uint8_t* s_src = (of_v ? p.c.v_scales : p.c.k_scales) + (int64_t)h0 * (D / 16);
  const uint32_t s_to = (of_v ? S::kVS : S::kKS) + my_token * S::kScale;
  const int scale_bytes = heads_kv * (D / 16);
  const bool whole_scales = p.c.heads * (D / 16) % 16 == 0;

  auto issue = [&](int k, uint32_t stage) {
    if (k < mine) {
      const uint32_t st = ring_addr + stage * S::kBytes;
      uint32_t slot;
      const bool ok = look.slot(slot);
      const uint32_t mask = __ballot_sync(0xffffffffu, ok);
#pragma unroll
      for (int i = 0; i < S::kTokens / 4; ++i) {
        const uint32_t row = __shfl_sync(0xffffffffu, slot, 4 * i + (lane >> 3));
        // rows 4i on: one bit of the place in V flips with i
        const uint32_t k_dst = st + k_to + i * 4 * S::kRow;
        const uint32_t v_dst = st + (i & 1 ? v_to ^ 64u : v_to) + i * 4 * S::kRow;
        if (mask == 0xffffffffu && heads_kv == S::kTeam) {
          cp_async_all<16>(k_dst, row_at(k_src, row, code_stride));
          cp_async_all<16>(v_dst, row_at(v_src, row, code_stride));
        } else {  // absent tokens' rows are zeros, absent heads' are not read by anyone
          const bool here = there && ((mask >> (4 * i + (lane >> 3))) & 1u);
          cp_async<16>(k_dst, row_at(k_src, row, code_stride), here);
          cp_async<16>(v_dst, row_at(v_src, row, code_stride), here);
        }
      }
      if (scale_lane) {
        const uint8_t* src = row_at(s_src, slot, scale_stride);
        if (whole_scales)
          cp_async_some(st + s_to, src, ok ? scale_bytes : 0);
        else
          for (int b = 0; b < scale_bytes; b += 4) cp_async<4>(st + s_to + b, src + b, ok);
      }
      // this warp's bits of the tile's mask
      if (lane == 0) {
        uint8_t* to = ring + stage * S::kBytes + S::kMask + member * (S::kTokens / 8);
        if constexpr (S::kTokens == 16)
          *reinterpret_cast<uint16_t*>(to) = (uint16_t)mask;
        else
          *to = (uint8_t)mask;
      }
      look.advance(k);
    }
    cp_async_commit();
  };

  team_sync<D>(team);  // the ring of the piece before has been read
#pragma unroll
  for (int k = 0; k < Shape::kStages - 1; ++k) issue(k, k);
  hd.begin(p, t, head0, heads, tile0 == 0 && sub == 0);

  uint32_t stage = 0, refill = Shape::kStages - 1;
  for (int k = 0; k < mine; ++k) {
    cp_async_wait<Shape::kStages - 2>();  // tile k of this warp's copies
    team_sync<D>(team);                   // and of the others'; tile k - 1 has been read
    issue(k + Shape::kStages - 1, refill);
    const uint8_t* st = ring + stage * S::kBytes;
    refill = stage;
    stage = stage + 1 == Shape::kStages ? 0 : stage + 1;
    const uint32_t mask = *reinterpret_cast<const uint32_t*>(st + S::kMask);
    if (active)
      attend_tile<D, NT>(p, r, t, head0, heads, TeamAt<D>(st, member, g, tq), mask,
                         (int64_t)kTile * (tile0 + sub + (int64_t)of * k), hd);
  }
  hd.end();
  cp_async_wait<0>();
}

}  // namespace kv4
}  // namespace dcp
