// kv4_ring.cuh -- how a warp walks tiles of 32 tokens and brings them in by
// itself: cp.async into a ring of its own, so that warps need no barrier
// between them.
#pragma once

#include "kv4_attention.cuh"

namespace dcp {
namespace kv4 {

// Shared memory of one warp's stage: the tile's K and V code rows, its K and
// V scales, the mask of present tokens.
template <int D>
struct Stage {
  static constexpr int kRow = D / 2;      // bytes of a code row
  static constexpr int kScale = D / 16;   // bytes of a scale row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kV = kTile * kRow;
  static constexpr int kKS = 2 * kTile * kRow;
  static constexpr int kVS = kKS + kTile * kScale;
  static constexpr int kMask = kVS + kTile * kScale;
  static constexpr int kBytes = kMask + 16;

  // Where chunk c (16 bytes) of row r lies: the lanes that are served at a
  // time touch all banks.  Reading K these are whole rows r and r + 2 (at dim
  // 256 half of each); reading V^T neighbouring chunks of the rows r, r + 1,
  // r + 4, r + 5.
  static __device__ __forceinline__ uint32_t k_at(int r, int c) {
    const int b1 = (r >> 1) & 1;
    return (uint32_t)(r * kRow + (D == 256 ? c ^ (b1 << 2) : c) * 16);
  }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) {
    const int b0 = r & 1, b1 = (r >> 1) & 1, b2 = (r >> 2) & 1, high = r & ~7;
    if constexpr (D == 64)  // four rows to 128 bytes
      return (uint32_t)((high | (b1 << 2) | (b2 << 1) | b0) * kRow + c * 16);
    else if constexpr (D == 128)  // two rows to 128 bytes
      return (uint32_t)(r * kRow + (c ^ (b2 << 1)) * 16);
    else
      return (uint32_t)(r * kRow + (c ^ ((b2 << 2) | (b0 << 1))) * 16);
  }
};

// A thread's operands in a stage (see attend_tile).
template <int D>
struct RingAt {
  using S = Stage<D>;
  const uint8_t *k0, *k1, *v0, *ks0, *vs0;
  static constexpr int kSubStep = 16, kHalfStep = 8;  // tokens
  static constexpr bool kRaw = false;
  __device__ void k_read() const {}
  __device__ void v_wait() const {}

  // The token (of 8) of the accumulator's row i: bits 0 and 1 swapped, so that
  // the rows that a warp reads at once lie in different banks.
  static __device__ __forceinline__ constexpr int token(int i) {
    return (i & 4) | ((i & 1) << 1) | ((i >> 1) & 1);
  }
  __device__ RingAt(const uint8_t* stage, int g, int tq) {
    const uint32_t k = S::k_at(token(g), D == 64 ? 0 : tq) + (D == 64 ? tq * 8 : 0);
    k0 = stage + k;
    k1 = stage + (k ^ 64u);
    v0 = stage + S::kV + S::v_at(token(2 * tq), g * S::kChunks / 8) + (g * (D / 16)) % 16;
    ks0 = stage + S::kKS + token(g) * S::kScale + (D == 64 ? tq : 2 * tq);
    vs0 = stage + S::kVS + token(2 * tq) * S::kScale +
          (D == 256 ? 2 * g : D == 128 ? g : g >> 1);
  }
  __device__ const uint8_t* k(int u, int i) const { return k0 + (16 * u + 8 * i) * S::kRow; }
  __device__ const uint8_t* k_second(int u, int i) const {
    return k1 + (16 * u + 8 * i) * S::kRow;
  }
  __device__ const uint8_t* k_scale(int u, int i) const {
    return ks0 + (16 * u + 8 * i) * S::kScale;
  }
  // the rows 2tq and 2tq + 1 stand for tokens two apart
  __device__ const uint8_t* v(int u, int i) const {
    return v0 + ((i & 1) * (D == 64 ? 4 : 2) + 16 * u + 8 * (i >> 1)) * S::kRow;
  }
  __device__ const uint8_t* v_scale(int u, int i) const {
    return vs0 + ((i & 1) * 2 + 16 * u + 8 * (i >> 1)) * S::kScale;
  }
};

// D * NT >= 256 takes up to 255 registers a thread, the others 128: 8 or 16
// warps fit on an SM.
template <int D, int NT>
struct RingShape {
  static constexpr int kWarpsPerSm = D * NT >= 256 ? 8 : 16;
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kQueue = kStages * Stage<D>::kBytes;  // ids on their way
  static constexpr int kBytes = kQueue + kIdQueue * 32 * 4;  // per warp
};

// One warp's tiles: every `of`-th of [tile0, tile1) of row t, from the
// `sub`-th on, for the query heads [head0, head0 + heads) of key/value head h;
// what they sum up to is in hd.
template <int D, int NT, bool kIds>
__device__ __forceinline__ void attend_tiles(const AttentionParams& p, const RowSpan& r, int t,
                                             int h, int head0, int heads, int tile0, int tile1,
                                             int sub, int of, uint8_t* smem, Heads<D, NT>& hd) {
  using S = Stage<D>;
  using Shape = RingShape<D, NT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int mine =
      tile1 - tile0 > sub ? (int)((unsigned)(tile1 - tile0 - sub + of - 1) / (unsigned)of) : 0;
  uint8_t* ring = smem + warp * Shape::kBytes;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  hd.fetch(p, t, head0, heads);
  Lookup<kIds> look(p, r, t, tile0 + sub, of, lane, ring + Shape::kQueue);

  // Copies: chunk `chunk` of the rows row0 + i * kStep; the i-th row's
  // destination lies at a constant distance (at dim 256 with a flipped chunk).
  constexpr int kStep = 32 / S::kChunks;
  const int chunk = lane % S::kChunks, row0 = lane / S::kChunks;
  const uint32_t code_stride = (uint32_t)p.c.heads * S::kRow;
  const uint32_t scale_stride = (uint32_t)p.c.heads * S::kScale;
  const uint32_t k_to = S::k_at(row0, chunk), v_to = S::kV + S::v_at(row0, chunk);
  auto row_to = [](uint32_t to, int i, bool v) {
    return (D == 256 && v && (i & 1) ? to ^ 64u : to) + (uint32_t)(i * kStep * S::kRow);
  };
  const uint8_t* k_src = p.c.k_codes + (int64_t)h * S::kRow + chunk * 16;
  const uint8_t* v_src = p.c.v_codes + (int64_t)h * S::kRow + chunk * 16;
  const uint8_t* ks_src = p.c.k_scales + (int64_t)h * S::kScale;
  const uint8_t* vs_src = p.c.v_scales + (int64_t)h * S::kScale;

  auto issue = [&](int k, uint32_t stage) {
    if (k < mine) {
      const uint32_t st = ring_addr + stage * S::kBytes;
      uint32_t slot;
      const bool ok = look.slot(slot);
      const uint32_t mask = __ballot_sync(0xffffffffu, ok);
      if (mask == 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
          const uint32_t row = __shfl_sync(0xffffffffu, slot, row0 + i * kStep);
          cp_async_all<16>(st + row_to(k_to, i, false), row_at(k_src, row, code_stride));
          cp_async_all<16>(st + row_to(v_to, i, true), row_at(v_src, row, code_stride));
        }
        cp_async_all<S::kScale>(st + S::kKS + lane * S::kScale,
                                row_at(ks_src, slot, scale_stride));
        cp_async_all<S::kScale>(st + S::kVS + lane * S::kScale,
                                row_at(vs_src, slot, scale_stride));
      } else {  // absent tokens' rows are zeros
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
          const uint32_t row = __shfl_sync(0xffffffffu, slot, row0 + i * kStep);
          const bool there = (mask >> (row0 + i * kStep)) & 1u;
          cp_async<16>(st + row_to(k_to, i, false), row_at(k_src, row, code_stride), there);
          cp_async<16>(st + row_to(v_to, i, true), row_at(v_src, row, code_stride), there);
        }
        cp_async<S::kScale>(st + S::kKS + lane * S::kScale, row_at(ks_src, slot, scale_stride),
                            ok);
        cp_async<S::kScale>(st + S::kVS + lane * S::kScale, row_at(vs_src, slot, scale_stride),
                            ok);
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::kBytes + S::kMask) = mask;
      look.advance(k);
    }
    cp_async_commit();
  };

#pragma unroll
  for (int k = 0; k < Shape::kStages - 1; ++k) issue(k, k);
  hd.begin(p, t, head0, heads, tile0 == 0 && sub == 0);

  uint32_t stage = 0, refill = Shape::kStages - 1;
  for (int k = 0; k < mine; ++k) {
    __syncwarp();  // the stage that issue() refills has been read by every lane
    issue(k + Shape::kStages - 1, refill);
    cp_async_wait<Shape::kStages - 1>();
    __syncwarp();  // the other lanes' copies and the mask
    const uint8_t* st = ring + stage * S::kBytes;
    refill = stage;
    stage = stage + 1 == Shape::kStages ? 0 : stage + 1;
    const uint32_t mask = *reinterpret_cast<const uint32_t*>(st + S::kMask);
    attend_tile<D, NT>(p, r, t, head0, heads, RingAt<D>(st, g, tq), mask,
                       (int64_t)kTile * (tile0 + sub + (int64_t)of * k), hd);
  }
  hd.end();
  cp_async_wait<0>();
}

}  // namespace kv4
}  // namespace dcp
