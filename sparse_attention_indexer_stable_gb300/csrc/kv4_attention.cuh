// kv4_attention.cuh -- attention of single query rows over the 4-bit cache.
//
// For one row and one key/value head, with the group's query heads q_h and
// the visible tokens j:
//   x_hj = c(q_h . k_j) in units of log2,  out_h = sum_j 2^(x_hj - m_h) v_j / l_h
// with m_h a reference within 2^8 of the running maximum and l_h the running
// sum.  A token costs dim + dim/8 bytes and 4 * dim operations per query
// head, so with up to 16 heads to a group the cache's bytes bound it, closely
// followed by the conversions of its codes.
//
// A CTA of 8 warps takes one row, one key/value head, up to 8 * NT of its
// query heads and some tiles of 32 tokens; each warp walks its tiles on its
// own, so nothing but the final join synchronises the CTA.
//  - Tiles come in by cp.async, a ring per warp.  A lane looks one token of
//    the tile up (id, page, slot) two tiles before its copy, so a gather by
//    ids costs little more than a range.
//  - S^T = K Q^T and O^T = V^T P^T by mma m16n8k16 (tokens and then elements
//    of the head as rows, query heads as columns): up to 8 heads fill the
//    8 columns, where Q K^T would leave half of 16 rows empty.  tcgen05 wants
//    64 or 128 rows and operands in shared memory; here the converted values
//    go straight from registers into the product.
//  - The sum over dim may run in any order: thread tq of a row takes 16-byte
//    pieces, so its codes are wide loads.  In V^T thread g takes dim/8
//    contiguous elements of four tokens; nibbles of two tokens are paired
//    before the conversion, which then yields the operand's pairs.
//  - codes and scales multiply exactly in fp16 (at most 6 significant bits).
//  - P moves from the accumulator's layout to the operand's by one transpose
//    of 8x8 matrices per 8 tokens (movmatrix).
//  - The accumulator is rescaled only when a score passes the reference by
//    2^8 (fp16 holds P up to 65504), which after the first tiles is rare.
//
// Two ways to cut a call up:
//  - slices: a cluster of 1, 2, 4 or 8 CTAs per row and head, joined through
//    distributed shared memory: one launch, no workspace.  For short rows.
//  - even shares: the tiles of all rows and heads in one line, cut into equal
//    shares for as many CTAs as fit on the GPU.  A share's first and last row
//    may be pieces of a row: those go to the workspace, and a second kernel
//    joins them.  For long rows and rows of different lengths.
#pragma once

#include <cooperative_groups.h>

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

constexpr int kAttWarps = 8;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr float kNoScore = -3.0e38f;  // reference of a head that has seen no token
constexpr float kSlack = 8.0f;        // scores may pass the reference by 2^8
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttentionParams {
  Planes c;
  const void* q;
  int64_t q_row_stride, q_head_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* starts;
  const int32_t* owner;
  const int32_t* ids;
  int64_t ids_stride;
  const int32_t* row_starts;
  void* out;
  float* lse;
  int4* shares;       // even shares, [share]: see attention_shares_kernel
  float* part_out;    // [share][2][together][8 * NT][dim]: outputs of its first and last piece
  float2* part_ml;    // [share][2][together][8 * NT]: their references and sums
  // when weights are wanted:
  float* scores;      // [rows][width][q_heads]: score / row_mult in log2 units
  float* row_mult;    // [rows][q_heads]
  float2* row_ml;     // [rows][q_heads]: the whole row's reference and sum
  float* weights;
  int64_t weights_stride, weights_width;
  int dtype, rows, q_heads, group, head_tiles, num_seqs;
  int together;       // even shares: key/value heads that a CTA walks at the same time
  int limit;          // positions end here at the latest
  int num_ids;
  int width;          // tokens per row of `scores`
  bool q_vec;
  bool score_pairs;   // two heads' scores can be stored at once
  float scale;        // of q.k, the K unit folded in
  float softcap;      // 0: none
};

// The tokens a row sees: positions [start, end), or num_ids ids of which
// those inside count.
struct RowSpan {
  int seq, start, end, n;
};

template <bool kIds>
__device__ __forceinline__ RowSpan row_span(const AttentionParams& p, int t) {
  RowSpan r;
  r.seq = p.owner ? __ldg(p.owner + t) : t;
  r.start = p.starts ? max(0, __ldg(p.starts + t)) : 0;
  r.end = min(__ldg(p.lens + t), p.limit);
  if ((unsigned)r.seq >= (unsigned)p.num_seqs) r.seq = 0, r.end = 0;
  r.n = r.end > r.start ? (kIds ? p.num_ids : r.end - r.start) : 0;
  return r;
}

// Position of the row's j-th token; -1: absent.
template <bool kIds>
__device__ __forceinline__ int token_pos(const AttentionParams& p, const RowSpan& r, int t,
                                         int row_start, int j) {
  if constexpr (kIds) {
    const int id = __ldg(p.ids + (int64_t)t * p.ids_stride + j);
    // 64-bit: an id near the end of int32 minus a negative row start
    const long long pos = (long long)id - row_start;
    return id >= 0 && pos >= r.start && pos < r.end ? (int)pos : -1;
  } else {
    return r.start + j;
  }
}

constexpr int kTile = 32;  // tokens of a tile: one per lane to look up

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

// The token (of 8) of the accumulator's row i: bits 0 and 1 swapped, so that
// the rows that a warp reads at once lie in different banks.
__device__ __forceinline__ constexpr int token_row(int i) {
  return (i & 4) | ((i & 1) << 1) | ((i >> 1) & 1);
}

template <int D, int NT>
struct AttentionShape {
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kCtasPerSm = D * NT >= 256 ? 1 : 2;
  static constexpr int kRing = kStages * Stage<D>::kBytes;  // per warp
  // the join: each warp's outputs (padded rows), references and sums
  static constexpr int kOutStride = D + 4;
  static constexpr int kJoin = (kAttWarps * 8 * NT * (kOutStride + 2) * 4 + 15) & ~15;
  // and behind it the CTA's own join, for the cluster: 16 bytes per output pair
  static constexpr int kSmem = kAttWarps * kRing;
  static_assert(kJoin + 8 * NT * D / 2 * 16 <= kSmem, "the join reuses the ring");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int kWords>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[kWords]) {
  if constexpr (kWords == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// First element of thread tq's run e of 8 query values (the elements of one
// code word): its code bytes are the 16-byte chunk tq (and 4 + tq at dim 256;
// 8 bytes at dim 64).
template <int D>
__device__ __forceinline__ constexpr int word_element(int tq, int w) {
  return D == 256 ? 128 * (w >> 2) + 32 * tq + 8 * (w & 3) : tq * (D / 4) + 8 * w;
}

// Head g's query values of this thread as the B operand of S^T = K Q^T,
// with the scale's sign, scaled by a power of two so that the head's largest magnitude is in
// [2^14, 2^15): bf16's 8 and fp16's 11 bits then fit fp16 for all elements
// within 2^-28 of the largest.  Returns the power of two to undo.  Heads
// beyond the group are zeros.
template <int D>
__device__ __forceinline__ float load_query(const AttentionParams& p, int t, int head, bool ok,
                                            int tq, uint32_t (&qf)[D / 8]) {
  float f[D / 4];
  const int64_t at = (int64_t)t * p.q_row_stride + (int64_t)head * p.q_head_stride;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const int64_t from = at + word_element<D>(tq, w);
    if (!ok) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[8 * w + e] = 0.0f;
    } else if (p.q_vec) {
      const uint4 x =
          __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + from));
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.dtype == DCP_BF16) {
          f[8 * w + 2 * e] = __uint_as_float(u[e] << 16);
          f[8 * w + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        } else {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(u + e));
          f[8 * w + 2 * e] = h.x, f[8 * w + 2 * e + 1] = h.y;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[8 * w + e] = load_element(p.q, from + e, p.dtype);
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(f[e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // exponent field of the largest magnitude; zero, subnormal and infinite
  // heads stay as they are
  const int ex = (int)(__float_as_uint(amax) >> 23);
  const bool plain = ex == 0 || ex == 255;
  const int shift = plain ? 0 : 14 - (ex - 127);  // within [-113, 140]
  // in two factors, each a normal fp32 power of two
  const float up1 =
      copysignf(__uint_as_float((uint32_t)(127 + shift / 2) << 23), p.scale);
  const float up2 = __uint_as_float((uint32_t)(127 + shift - shift / 2) << 23);
#pragma unroll
  for (int e = 0; e < D / 8; ++e)
    qf[e] = pack_pair(f[2 * e] * up1 * up2, f[2 * e + 1] * up1 * up2, DCP_F16);
  return __uint_as_float((uint32_t)(127 - shift / 2) << 23) *
         __uint_as_float((uint32_t)(127 - (shift - shift / 2)) << 23);
}

// One warp's work on one piece: every `of`-th of the tiles [tile0, tile1) of
// row t, from the `sub`-th on, for the query heads [head0, head0 + heads) of
// key/value head h.  Leaves in shared memory its outputs, references and sums
// (all warps of the CTA take part: barriers).
template <int D, int NT, bool kIds>
__device__ __forceinline__ void attend_piece(const AttentionParams& p, const RowSpan& r, int t,
                                             int h, int head0, int heads, int tile0, int tile1,
                                             int sub, int of, uint8_t* smem) {
  using S = Stage<D>;
  using Shape = AttentionShape<D, NT>;
  constexpr int kMTiles = D / 16;
  constexpr int kSub = kTile / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int mine =
      heads > 0 && tile1 - tile0 > sub ? (int)((unsigned)(tile1 - tile0 - sub + of - 1) / of) : 0;
  const int first = tile0 + sub;
  const int row_start = kIds && p.row_starts ? __ldg(p.row_starts + t) : 0;
  const int32_t* table = p.table + (int64_t)r.seq * p.table_stride;

  uint8_t* ring = smem + warp * Shape::kRing;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);

  // This lane's tokens, tile after tile.
  uint32_t j_next = (uint32_t)kTile * (uint32_t)first + lane;  // n < 2^31: no overflow
  const uint32_t j_step = (uint32_t)kTile * (uint32_t)of;
  auto next_pos = [&]() {
    const int pos = j_next < (uint32_t)r.n ? token_pos<kIds>(p, r, t, row_start, (int)j_next) : -1;
    j_next += j_step;
    return pos;
  };
  auto page_of = [&](int pos) { return pos >= 0 ? __ldg(table + (pos >> p.c.page_shift)) : -1; };

  // The position and page of the next tile to fetch, and the position after
  // it: loaded one and two tiles ahead of the copies that need them.
  int pos0 = next_pos();
  int pos1 = next_pos();
  int page0 = page_of(pos0);

  // Copies: chunk `chunk` of the rows row0 + i * kStep.
  constexpr int kStep = 32 / S::kChunks;
  const int chunk = lane % S::kChunks, row0 = lane / S::kChunks;
  const uint32_t code_stride = (uint32_t)p.c.heads * S::kRow;
  const uint32_t scale_stride = (uint32_t)p.c.heads * S::kScale;
  // destinations in a stage; the i-th row's by a constant (and at dim 256 a
  // flip of its chunk)
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
      const bool ok = (uint32_t)page0 < p.c.num_pages;
      const uint32_t slot =
          ok ? ((uint32_t)page0 << p.c.page_shift) | (pos0 & ((1u << p.c.page_shift) - 1u)) : 0u;
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
      } else {
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
      pos0 = pos1;
      page0 = page_of(pos0);
      pos1 = next_pos();
    }
    cp_async_commit();
  };

#pragma unroll
  for (int k = 0; k < Shape::kStages - 1; ++k) issue(k, k);

  // Queries while the first tiles are under way.
  uint32_t qf[NT][D / 8];
  // What brings the products of the columns 2tq, 2tq+1 to log2 units (or to
  // units of the cap); positive, a negative scale's sign is in the queries.
  float mult[NT][2];
  const float unit = fabsf(p.softcap > 0.0f ? p.scale / p.softcap : p.scale * kLog2e);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float undo =
        load_query<D>(p, t, head0 + 8 * n + g, 8 * n + g < heads, tq, qf[n]) * unit;
    // above 0: -infinity times it stays -infinity
    mult[n][0] = fmaxf(__shfl_sync(0xffffffffu, undo, 8 * tq), 1e-37f);
    mult[n][1] = fmaxf(__shfl_sync(0xffffffffu, undo, 8 * tq + 4), 1e-37f);
  }
  const float cap = p.softcap * kLog2e;
  // Scores that are capped get their units at once, the others in the
  // exponent's multiply-add.
  const bool capped = p.softcap > 0.0f;
  float late[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      late[n][c] = capped ? 1.0f : mult[n][c];
      const int head = 8 * n + 2 * tq + c;
      if (p.row_mult && tile0 == 0 && sub == 0 && g == 0 && head < heads)
        p.row_mult[(int64_t)t * p.q_heads + head0 + head] = late[n][c];
    }

  float o[NT][kMTiles][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) m[n][c] = kNoScore, l[n][c] = 0.0f;
#pragma unroll
    for (int i = 0; i < kMTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
  }

  // Where this thread reads in a stage: the first of its K rows, V rows and
  // scales; the others lie at constant distances.
  constexpr int kVWords = D / 64;  // per thread and token
  const uint32_t k_from = S::k_at(token_row(g), D == 64 ? 0 : tq) + (D == 64 ? tq * 8 : 0);
  const uint32_t v_from = S::kV + S::v_at(token_row(2 * tq), g * S::kChunks / 8) +
                          (g * (D / 16)) % 16;
  constexpr uint32_t kVNext = (D == 64 ? 4 : 2) * S::kRow;  // from row r to row r + 2
  const uint32_t ks_from = S::kKS + token_row(g) * S::kScale + (D == 64 ? tq : 2 * tq);
  const uint32_t vs_from =
      S::kVS + token_row(2 * tq) * S::kScale + (D == 256 ? 2 * g : D == 128 ? g : g >> 1);

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

    // S^T: rows are tokens 16u + token_row(g) and + 8, columns the heads 2tq and 2tq + 1
    float s[NT][kSub][4];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      constexpr int kWords = D / 32;  // per thread and row
      uint32_t kw[2][kWords], ks[2][(kWords + 3) / 4];  // ks: two blocks' scales each
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* kp = st + k_from + (16 * u + 8 * i) * S::kRow;
        const uint8_t* sp = st + ks_from + (16 * u + 8 * i) * S::kScale;
        if constexpr (D == 256) {
          uint32_t lo[4], hi[4];
          load_words<4>(kp, lo);
          load_words<4>(st + (k_from ^ 64u) + (16 * u + 8 * i) * S::kRow, hi);
#pragma unroll
          for (int e = 0; e < 4; ++e) kw[i][e] = lo[e], kw[i][4 + e] = hi[e];
          ks[i][0] = scales_to_half(*reinterpret_cast<const uint16_t*>(sp));
          ks[i][1] = scales_to_half(*reinterpret_cast<const uint16_t*>(sp + 8));
        } else {
          load_words<kWords>(kp, kw[i]);
          if constexpr (D == 128)
            ks[i][0] = scales_to_half(*reinterpret_cast<const uint16_t*>(sp));
          else
            ks[i][0] = scales_to_half(sp[0]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][u][e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          codes_to_half(kw[i][w], a[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            a[i][e] = D != 64 && (w & 2) ? hmul2_high(a[i][e], ks[i][w >> 2])
                                         : hmul2_low(a[i][e], ks[i][w >> 2]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(s[n][u], a[0][0], a[1][0], a[0][1], a[1][1], qf[n][4 * w], qf[n][4 * w + 1]);
          mma_f16(s[n][u], a[0][2], a[1][2], a[0][3], a[1][3], qf[n][4 * w + 2],
                  qf[n][4 * w + 3]);
        }
      }
    }

    if (capped) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] = cap * tanhf(s[n][u][e] * mult[n][e & 1]);
    }
    if (mask != 0xffffffffu) {
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((mask >> (16 * u + token_row(g) + 8 * (e >> 1))) & 1u))
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][u][e] = -INFINITY;
    }
    if (p.scores) {
      const int64_t j = (int64_t)kTile * (first + (int64_t)of * k);
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t tok = j + 16 * u + token_row(g) + 8 * i;
          float* dst = p.scores + ((int64_t)t * p.width + tok) * p.q_heads + head0 + 2 * tq;
          if (tok < r.n)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int head = 8 * n + 2 * tq;
              if (p.score_pairs && head + 1 < heads) {
                *reinterpret_cast<float2*>(dst + 8 * n) =
                    make_float2(s[n][u][2 * i], s[n][u][2 * i + 1]);
              } else {
                if (head < heads) dst[8 * n] = s[n][u][2 * i];
                if (head + 1 < heads) dst[8 * n + 1] = s[n][u][2 * i + 1];
              }
            }
        }
    }
    bool past = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[n][c] = s[n][0][c];
#pragma unroll
        for (int e = c + 2; e < 4 * kSub; e += 2)
          top[n][c] = fmaxf(top[n][c], s[n][e >> 2][e & 3]);
        top[n][c] *= late[n][c];
        past |= top[n][c] > m[n][c] + kSlack;
      }
    if (__any_sync(0xffffffffu, past)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = top[n][c];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[n][c], x);
          const float corr = exp2_approx(m[n][c] - mn);
          m[n][c] = mn;
          l[n][c] *= corr;
#pragma unroll
          for (int i = 0; i < kMTiles; ++i) o[n][i][c] *= corr, o[n][i][c + 2] *= corr;
        }
    }
    uint32_t pf[NT][kSub][2];  // P^T: column head g, tokens of rows 2tq, 2tq + 1 and + 8
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][u][e] = exp2_approx(fmaf(s[n][u][e], late[n][e & 1], -m[n][e & 1]));
          l[n][e & 1] += s[n][u][e];
        }
        pf[n][u][0] = transpose8x8(pack_pair(s[n][u][0], s[n][u][1], DCP_F16));
        pf[n][u][1] = transpose8x8(pack_pair(s[n][u][2], s[n][u][3], DCP_F16));
      }

    // O^T: rows are elements g * D/8 + 2i and + 1 (tile i), columns heads
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      constexpr int kBlocks = D == 256 ? 2 : 1;
      uint32_t vw[4][kVWords];
      uint32_t vs[2][kBlocks];  // scales of the tokens' pairs, per block of the thread's elements
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load_words<kVWords>(
            st + v_from + (i & 1) * kVNext + (16 * u + 8 * (i >> 1)) * S::kRow, vw[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* sp = st + vs_from + (16 * u + 8 * i) * S::kScale;
        if constexpr (D == 256) {
          const uint32_t x = *reinterpret_cast<const uint16_t*>(sp);
          const uint32_t y = *reinterpret_cast<const uint16_t*>(sp + 2 * S::kScale);
          vs[i][0] = scales_to_half(__byte_perm(x, y, 0x0040));
          vs[i][1] = scales_to_half(__byte_perm(x, y, 0x0051));
        } else {
          vs[i][0] = scales_to_half((uint32_t)sp[0] + (uint32_t)sp[2 * S::kScale] * 256u);
        }
      }
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        uint32_t a[2][2][4];  // [token pair][even, odd element][byte]
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = vw[2 * i][w], y = vw[2 * i + 1][w];
          codes_to_half((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), a[i][0]);
          codes_to_half(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), a[i][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[i][0][e] = hmul2(a[i][0][e], vs[i][w >> 1]);
            a[i][1][e] = hmul2(a[i][1][e], vs[i][w >> 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_f16(o[n][4 * w + e], a[0][0][e], a[0][1][e], a[1][0][e], a[1][1][e], pf[n][u][0],
                    pf[n][u][1]);
      }
    }
  }

  cp_async_wait<0>();
  __syncthreads();  // every warp has read its ring
  float* join_o = reinterpret_cast<float*>(smem);
  float* join_m = join_o + kAttWarps * 8 * NT * Shape::kOutStride;
  float* join_l = join_m + kAttWarps * 8 * NT;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = l[n][c];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int col = warp * 8 * NT + 8 * n + 2 * tq + c;
      if (g == 0) join_m[col] = m[n][c], join_l[col] = sum;
      float* dst = join_o + col * Shape::kOutStride + g * (D / 8);
#pragma unroll
      for (int i = 0; i < kMTiles; ++i)
        *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[n][i][c], o[n][i][c + 2]);
    }
  __syncthreads();
}

// What attend_piece left, added over the warps [warp0, warp0 + of): reference,
// sum and two outputs of `head` at element d.
struct __align__(16) Joined {
  float top, sum, x, y;
};

template <int D, int NT>
__device__ __forceinline__ Joined join_warps(const uint8_t* smem, int warp0, int of, int head,
                                             int d) {
  using Shape = AttentionShape<D, NT>;
  const float* join_o = reinterpret_cast<const float*>(smem);
  const float* join_m = join_o + kAttWarps * 8 * NT * Shape::kOutStride;
  const float* join_l = join_m + kAttWarps * 8 * NT;
  Joined j{kNoScore, 0.0f, 0.0f, 0.0f};
  for (int w = warp0; w < warp0 + of; ++w) j.top = fmaxf(j.top, join_m[w * 8 * NT + head]);
#pragma unroll 8
  for (int w = warp0; w < warp0 + of; ++w) {
    const int col = w * 8 * NT + head;
    const float f = exp2_approx(join_m[col] - j.top);
    const float2 v = *reinterpret_cast<const float2*>(join_o + col * Shape::kOutStride + d);
    j.sum += f * join_l[col];
    j.x += f * v.x;
    j.y += f * v.y;
  }
  return j;
}

// A row's finished head: `at` = row * q_heads + head.
template <int D>
__device__ __forceinline__ void write_out(const AttentionParams& p, int64_t at, int d,
                                          const Joined& j) {
  // no token: 0; a NaN sum goes through
  const float inv = j.sum == 0.0f ? 0.0f : p.c.v_unit / j.sum;
  reinterpret_cast<uint32_t*>(p.out)[(at * D + d) >> 1] = pack_pair(j.x * inv, j.y * inv, p.dtype);
  if (d == 0) {
    p.lse[at] = j.sum == 0.0f ? -INFINITY : (j.top + log2f(j.sum)) * kLn2;
    if (p.row_ml) p.row_ml[at] = make_float2(j.top, j.sum);
  }
}

// Slices: cluster rank s takes the s-th part of the row's tiles.  blockIdx.x =
// ((row * head_tiles + head tile) * heads + head) * slices + slice.
template <int D, int NT, bool kIds>
__global__ void __launch_bounds__(kAttThreads, AttentionShape<D, NT>::kCtasPerSm)
    attention_slices_kernel(const __grid_constant__ AttentionParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int slices = (int)cluster.num_blocks(), slice = (int)cluster.block_rank();
  const unsigned unit = blockIdx.x / (unsigned)slices;
  const int h = (int)(unit % (unsigned)p.c.heads);
  const unsigned rest = unit / (unsigned)p.c.heads;
  const int ht = (int)(rest % (unsigned)p.head_tiles);
  const int t = (int)(rest / (unsigned)p.head_tiles);
  const int head0 = h * p.group + ht * 8 * NT;           // first query head of this CTA
  const int heads = min(8 * NT, p.group - ht * 8 * NT);  // and how many

  grid_dependency_wait();
  const RowSpan r = row_span<kIds>(p, t);
  const int tiles = (int)(((int64_t)r.n + kTile - 1) / kTile);
  const int per = (tiles + slices - 1) / slices;
  const int tile0 = min(tiles, slice * per), tile1 = min(tiles, tile0 + per);
  attend_piece<D, NT, kIds>(p, r, t, h, head0, heads, tile0, tile1, threadIdx.x >> 5, kAttWarps,
                            smem);

  const int64_t at = (int64_t)t * p.q_heads + head0;
  if (slices == 1) {
    for (int i = threadIdx.x; i < heads * (D / 2); i += kAttThreads) {
      const int head = i / (D / 2), d = 2 * (i % (D / 2));
      write_out<D>(p, at + head, d, join_warps<D, NT>(smem, 0, kAttWarps, head, d));
    }
    return;
  }
  // The CTA's own join goes behind the warps' (each thread its own values),
  // then every CTA adds its part of the outputs over the cluster.
  Joined* mine = reinterpret_cast<Joined*>(smem + AttentionShape<D, NT>::kJoin);
  for (int i = threadIdx.x; i < heads * (D / 2); i += kAttThreads)
    mine[i] = join_warps<D, NT>(smem, 0, kAttWarps, i / (D / 2), 2 * (i % (D / 2)));
  cluster.sync();
  for (int i = slice * kAttThreads + threadIdx.x; i < heads * (D / 2);
       i += slices * kAttThreads) {
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
    write_out<D>(p, at + i / (D / 2), 2 * (i % (D / 2)), j);
  }
  cluster.sync();  // no CTA leaves while others read its shared memory
}

// Even shares.  The line of tiles: rows in order, in a row its units (groups of
// `together` key/value heads, times head tiles), in a unit its tiles; a row
// that sees nothing has one (empty) tile per unit, so that its outputs are
// written.  Share c is tiles [c * per, (c + 1) * per).
//
// The heads of a group are walked at the same time, by 8 / together warps
// each: a token's rows of neighbouring heads are neighbours in memory, and
// DRAM serves 128 bytes at a time.  Walked one after the other, 131072 tokens
// of 8 heads of 64-byte rows read 2.2 times their bytes.
//
// Record of a share, for the join: its last piece, if that is the first of a
// unit that later shares go on with: x = row, y = unit, z = the last of those
// shares (0: no such piece).

template <int D, int NT, bool kIds>
__global__ void __launch_bounds__(kAttThreads, AttentionShape<D, NT>::kCtasPerSm)
    attention_shares_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long warp_sum[kAttWarps];
  __shared__ int s_row;
  __shared__ long long s_before;  // tiles of a head in the rows before s_row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.c.heads + p.together - 1) / p.together;
  const int units = groups * p.head_tiles;
  const int of = kAttWarps / p.together;  // warps of a head
  grid_dependency_wait();

  auto tiles_of = [&](const RowSpan& r) {
    return max(1, (int)(((int64_t)r.n + kTile - 1) / kTile));
  };
  // prefix sums of the rows' tiles: each thread a run of rows
  const int run = (p.rows + kAttThreads - 1) / kAttThreads;
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
  for (int w = 0; w < kAttWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= units;
  // at least a tile for each warp
  const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)of);
  const long long x0 = min(total, blockIdx.x * per), x1 = min(total, x0 + per);
  if (x0 < x1 && before * units <= x0 && x0 < (before + own) * units) {
    int t = row0;
    for (;; ++t) {
      const int n = tiles_of(row_span<kIds>(p, t));
      if (x0 < (before + n) * units) break;
      before += n;
    }
    s_row = t;
    s_before = before;
  }
  __syncthreads();

  int4 record = make_int4(0, 0, 0, 0);
  if (x0 < x1) {
    int t = s_row;
    long long base = s_before * units;  // where row t begins
    RowSpan r = row_span<kIds>(p, t);
    int tiles = tiles_of(r);
    for (long long x = x0; x < x1;) {
      const int unit = (int)((x - base) / tiles);
      const int tile0 = (int)((x - base) - (long long)unit * tiles);
      const int tile1 = (int)min((long long)tiles, tile0 + (x1 - x));
      const int h0 = unit % groups * p.together, ht = unit / groups;
      const int heads = min(8 * NT, p.group - ht * 8 * NT);  // query heads of each
      const int heads_kv = min(p.together, p.c.heads - h0);
      const int h = h0 + warp / of;  // this warp's; beyond the last: nothing to do
      attend_piece<D, NT, kIds>(p, r, t, h, h * p.group + ht * 8 * NT,
                                h < p.c.heads ? heads : 0, tile0, tile1, warp % of, of, smem);
      const bool whole = tile0 == 0 && tile1 == tiles;
      const int64_t at = (int64_t)t * p.q_heads + h0 * p.group + ht * 8 * NT;
      const int64_t part = ((int64_t)blockIdx.x * 2 + (tile0 == 0)) * p.together * 8 * NT;
      for (int i = threadIdx.x; i < heads_kv * heads * (D / 2); i += kAttThreads) {
        const int q = i / (D / 2), d = 2 * (i % (D / 2));
        const int kv = q / heads, head = q - kv * heads;
        const Joined j = join_warps<D, NT>(smem, kv * of, of, head, d);
        if (whole) {
          write_out<D>(p, at + kv * p.group + head, d, j);
        } else {
          const int64_t to = part + kv * 8 * NT + head;
          *reinterpret_cast<float2*>(p.part_out + to * D + d) = make_float2(j.x, j.y);
          if (d == 0) p.part_ml[to] = make_float2(j.top, j.sum);
        }
      }
      if (!whole && tile0 == 0) record = make_int4(t, unit, (int)((x + tiles - 1) / per), 0);
      __syncthreads();  // the join has been read before the next piece's copies
      x += tile1 - tile0;
      if (tile1 == tiles && unit == units - 1 && x < x1) {
        base += (long long)tiles * units;
        r = row_span<kIds>(p, ++t);
        tiles = tiles_of(r);
      }
    }
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

// weights[t][pos] += sum over the query heads of 2^(x - m) / l: 8 lanes per
// token, a CTA per 1024 tokens of a row.  From m and l rather than lse, whose
// rounding would be an error of the exponent; the exponent is the attention's
// own, bit for bit.
constexpr int kWeightTokens = 1024;

template <bool kIds>
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ float weight_heads[];  // [3][q_heads]: multiplier, reference, 1 / sum
  float* mult = weight_heads;
  float* ref = mult + p.q_heads;
  float* inv = ref + p.q_heads;
  const int tiles = (p.width + kWeightTokens - 1) / kWeightTokens;
  const int t = blockIdx.x / tiles;
  const int64_t j0 = (int64_t)(blockIdx.x % tiles) * kWeightTokens;
  grid_dependency_wait();
  const RowSpan r = row_span<kIds>(p, t);
  const int n = min(r.n, p.width);
  if (j0 >= n) return;
  for (int h = threadIdx.x; h < p.q_heads; h += 256) {
    const int64_t at = (int64_t)t * p.q_heads + h;
    const float2 v = p.row_ml[at];
    mult[h] = p.row_mult[at];
    ref[h] = v.x;
    inv[h] = v.y == 0.0f ? 0.0f : 1.0f / v.y;
  }
  __syncthreads();
  const int row_start = kIds && p.row_starts ? __ldg(p.row_starts + t) : 0;
  const int sub = threadIdx.x & 7;
  for (int i = threadIdx.x >> 3; i < kWeightTokens; i += 32) {
    const int64_t j = j0 + i;
    float sum = 0.0f;
    if (j < n) {
      const float* x = p.scores + ((int64_t)t * p.width + j) * p.q_heads;
      for (int h = sub; h < p.q_heads; h += 8) {
        // absent tokens: 2^-inf = 0
        sum += exp2_approx(fmaf(x[h], mult[h], -ref[h])) * inv[h];
      }
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    if (sub == 0 && j < n) {
      const int pos = token_pos<kIds>(p, r, t, row_start, (int)j);
      if (pos >= 0 && pos < p.weights_width) {
        float* w = p.weights + (int64_t)t * p.weights_stride + pos;
        if constexpr (kIds)
          atomicAdd(w, sum);  // an id may be listed twice
        else
          *w += sum;
      }
    }
  }
}

}  // namespace kv4
}  // namespace dcp
