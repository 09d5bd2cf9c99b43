// kv4_attention.cuh -- attention of single query rows over the 4-bit cache.
//
// For one row and one key/value head, with the group's query heads q_h and
// the visible tokens j:
//   x_hj = c(q_h . k_j) in units of log2,  out_h = sum_j 2^(x_hj - m_h) v_j / l_h
// with m_h a reference from 2^7 below the running maximum to 2^15 below it and
// l_h the running sum.  A token costs dim + dim/8 bytes and 4 * dim operations per query
// head, so with up to 16 heads to a group the cache's bytes bound it, closely
// followed by the conversions of its codes.
//
// What a warp does with a tile of 32 tokens (attend_tile):
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
//    2^15 (fp16 holds P up to 65504), which after the first tiles is rare: the
//    reference is set 2^7 below the maximum.  That also keeps light tokens: P
//    in fp16 steps by 2^-24 at the least, 2^-31 or less of the heaviest token's.
//    With the reference at the maximum, 2^17 tokens of 2^-25 each, a third of a
//    percent of a row together, fell out of the products and stayed in the sum.
//
// Two kernels cut a call up: kv4_slices.cuh for short rows, kv4_shares.cuh for
// long rows and rows of different lengths; kv4_ring.cuh brings the tiles in.
#pragma once

#include <cooperative_groups.h>

#include "kv4_common.cuh"

namespace dcp {
namespace kv4 {

constexpr float kNoScore = -3.0e38f;  // reference of a head that has seen no token
constexpr float kBelow = 7.0f;        // a reference is set 2^7 below the maximum
constexpr float kSlack = 15.0f;       // and scores may pass it by 2^15
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 32;  // tokens of a tile: one per lane to look up

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
  int4* shares;       // even shares, [share]: see kv4_shares.cuh
  int2* cuts;         // and [rows][units], where those are few: a unit's first and last share
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
  unsigned int* status;  // the device's status word
  bool q_vec;
  bool score_pairs;   // two heads' scores can be stored at once
  float scale;        // of q.k, the K unit folded in
  float softcap;      // 0: none
#ifdef DCP_DEBUG_POISON
  int withheld_share, withheld_tile;  // see dcp_kv4_selftest_withhold
#endif
};

// The tokens a row sees: positions [start, end), or num_ids ids of which
// those inside count.
struct RowSpan {
  int seq, start, end, n;
  int skip;  // of the n, the first that the row does not see
};

template <bool kIds>
__device__ __forceinline__ RowSpan row_span(const AttentionParams& p, int t) {
  RowSpan r;
  r.seq = p.owner ? __ldg(p.owner + t) : t;
  r.start = p.starts ? max(0, __ldg(p.starts + t)) : 0;
  r.end = min(__ldg(p.lens + t), p.limit);
  if ((unsigned)r.seq >= (unsigned)p.num_seqs) r.seq = 0, r.end = 0;
  r.n = r.end > r.start ? (kIds ? p.num_ids : r.end - r.start) : 0;
  r.skip = 0;
  return r;
}

// The position that the row's j-th token or id stands for, -1: none of the
// row's.  `given`: the id; without ids j itself.
template <bool kIds>
__device__ __forceinline__ int token_pos(const RowSpan& r, int row_start, int given) {
  if constexpr (kIds) {
    // 64-bit: an id near the end of int32 minus a negative row start
    const long long pos = (long long)given - row_start;
    return given >= 0 && pos >= r.start && pos < r.end ? (int)pos : -1;
  } else {
    return r.start + given;
  }
}

// Looks the tokens of a warp's tiles up, a lane a token: pages two tiles ahead
// of the copies that need them, ids, whose loads precede the pages', three
// tiles before that.  These go to shared memory by cp.async, a lane's own four
// at a time, in the groups of the tiles' copies: a load waits in line behind
// the copies sent before it, and with both loads in registers, an id and a page
// a tile ahead, 1024 rows x 2048 ids took 597 us (451 without the ids' loads).
constexpr int kIdQueue = 4;  // tiles

template <bool kIds>
struct Lookup {
  const AttentionParams& p;
  const RowSpan& r;
  const int32_t* table;
  const int32_t* ids;  // this lane's, ids only
  int32_t* queue;      // likewise; [kIdQueue][32]
  int row_start;
  uint32_t j, step;    // n < 2^31: no overflow
  int page0, page1;    // of the next tile to fetch and the one behind
  int pos0, pos1;      // ids only: their positions

  // tiles first, first + every, ... of row t; of each the token `token`
  __device__ Lookup(const AttentionParams& p_, const RowSpan& r_, int t, int first, int every,
                    int token, uint8_t* queue_)
      : p(p_), r(r_), table(p_.table + (int64_t)r_.seq * p_.table_stride) {
    j = (uint32_t)kTile * (uint32_t)first + token;
    step = (uint32_t)kTile * (uint32_t)every;
    if constexpr (kIds) {
      queue = reinterpret_cast<int32_t*>(queue_) + (threadIdx.x & 31);
      ids = p.ids + (int64_t)t * p.ids_stride;
      row_start = p.row_starts ? __ldg(p.row_starts + t) : 0;
      int given[5];  // tiles 0 to 4: their own number bounds the reads, not the row's length
#pragma unroll
      for (int i = 0; i < 5; ++i) given[i] = at(i) ? __ldg(ids + j + i * step) : -1;
#pragma unroll
      for (int i = 2; i < 5; ++i) queue[(i % kIdQueue) * 32] = given[i];
      pos0 = position(given[0]);
      pos1 = position(given[1]);
      page0 = page(pos0);
      page1 = page(pos1);
    } else {
      page0 = page(place(j));
      page1 = page(place(j + step));
    }
  }
  // Whether the ids reach to the i-th tile from here.
  __device__ bool at(int i) const { return j + (uint32_t)i * step < (uint32_t)p.num_ids; }
  __device__ int position(int given) const {
    return given < 0 ? -1 : token_pos<kIds>(r, row_start, given);
  }
  // A range's token at x, -1 beyond the last.
  __device__ int place(uint32_t x) const { return x < (uint32_t)r.n ? r.start + (int)x : -1; }
  __device__ int page(int pos) const {
    return pos >= 0 ? __ldg(table + (pos >> p.c.page_shift)) : -1;
  }
  // Whether this lane's token of the current tile is in the cache, and its slot.
  __device__ bool slot(uint32_t& to) const {
    const bool ok = (uint32_t)page0 < p.c.num_pages;
    const int pos = kIds ? pos0 : r.start + (int)j;
    to = ok ? ((uint32_t)page0 << p.c.page_shift) | (pos & ((1u << p.c.page_shift) - 1u)) : 0u;
    return ok;
  }
  // On to tile k + 1, after the copies of tile k and in their group.  The id
  // read here, of tile k + 2, came with the copies of tile k - 3, whose group is
  // complete: a ring has at most three stages.
  __device__ void advance(int k) {
    page0 = page1;
    if constexpr (kIds) {
      pos0 = pos1;
      pos1 = position(at(2) ? queue[((k + 2) % kIdQueue) * 32] : -1);
      page1 = page(pos1);
      if (at(5))
        cp_async_all<4>((uint32_t)__cvta_generic_to_shared(queue + ((k + 5) % kIdQueue) * 32),
                        ids + j + 5 * step);
      j += step;
    } else {
      j += step;
      page1 = page(place(j + step));
    }
  }
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

// Head g's query values of this thread, as they are (pairs of 16-bit
// elements); heads beyond the group are zeros.  Loaded before the first tokens
// are looked up, converted after their copies have been sent off.
template <int D>
__device__ __forceinline__ void fetch_query(const AttentionParams& p, int t, int head, bool ok,
                                            int tq, uint32_t (&qf)[D / 8]) {
  const int64_t at = (int64_t)t * p.q_row_stride + (int64_t)head * p.q_head_stride;
  const uint16_t* q = static_cast<const uint16_t*>(p.q);
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const int64_t from = at + word_element<D>(tq, w);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (ok && p.q_vec) {
      x = __ldg(reinterpret_cast<const uint4*>(q + from));
    } else if (ok) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = __ldg(q + from + 2 * e) | ((uint32_t)__ldg(q + from + 2 * e + 1) << 16);
      x = make_uint4(u[0], u[1], u[2], u[3]);
    }
    qf[4 * w] = x.x, qf[4 * w + 1] = x.y, qf[4 * w + 2] = x.z, qf[4 * w + 3] = x.w;
  }
}

// These as the B operand of S^T = K Q^T, with the scale's sign, scaled by a
// power of two so that the head's largest magnitude is in [2^14, 2^15): bf16's
// 8 and fp16's 11 bits then fit fp16 for all elements within 2^-28 of the
// largest.  Returns the power of two to undo.
template <int D>
__device__ __forceinline__ float convert_query(const AttentionParams& p, uint32_t (&qf)[D / 8]) {
  auto pair = [&](uint32_t u) {
    return p.dtype == DCP_BF16
               ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u))
               : __half22float2(*reinterpret_cast<const __half2*>(&u));
  };
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 8; ++e) {
    const float2 f = pair(qf[e]);
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
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
  for (int e = 0; e < D / 8; ++e) {
    const float2 f = pair(qf[e]);
    qf[e] = pack_pair(f.x * up1 * up2, f.y * up1 * up2, DCP_F16);
  }
  return __uint_as_float((uint32_t)(127 - shift / 2) << 23) *
         __uint_as_float((uint32_t)(127 - (shift - shift / 2)) << 23);
}

// A warp's query heads and what it has summed up of them: columns are the
// heads 8n + 2tq and + 1, O^T's rows the elements g * D/8 + 2i and + 1.
template <int D, int NT>
struct Heads {
  static constexpr int kMTiles = D / 16;
  uint32_t qf[NT][D / 8];
  // What brings the products to log2 units (or to units of the cap): positive,
  // a negative scale's sign is in the queries.
  float mult[NT][2];
  // Scores that are capped get their units at once, the others in the
  // exponent's multiply-add.
  float late[NT][2];
  float o[NT][kMTiles][4];
  float m[NT][2], l[NT][2];
  float over[NT][2];  // what l is too large by: see attend_tile

  __device__ void fetch(const AttentionParams& p, int t, int head0, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      fetch_query<D>(p, t, head0 + 8 * n + g, 8 * n + g < heads, tq, qf[n]);
  }

  // What fetch() has loaded, made ready; sums from zero.
  __device__ void begin(const AttentionParams& p, int t, int head0, int heads, bool write_mult) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
    const bool capped = p.softcap > 0.0f;
    const float unit = fabsf(capped ? p.scale / p.softcap : p.scale * kLog2e);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float undo = convert_query<D>(p, qf[n]) * unit;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // above 0: -infinity times it stays -infinity; finite: 0 times it stays 0
        mult[n][c] =
            fminf(fmaxf(__shfl_sync(0xffffffffu, undo, 8 * tq + 4 * c), 1e-37f), 3e38f);
        late[n][c] = capped ? 1.0f : mult[n][c];
        const int head = 8 * n + 2 * tq + c;
        if (write_mult && p.row_mult && g == 0 && head < heads)
          p.row_mult[(int64_t)t * p.q_heads + head0 + head] = late[n][c];
        m[n][c] = kNoScore;
        l[n][c] = over[n][c] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kMTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
    }
  }

  // After the last tile.
  __device__ void end() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) l[n][c] -= over[n][c];
  }
};

// All ones if the token of the V row (u, i) is there, else 0.
template <typename At>
__device__ __forceinline__ uint32_t present(const At& at, int u, int i, uint32_t mask) {
  return 0u - ((mask >> at.v_token(u, i)) & 1u);
}

// One tile.  `at` says where this thread's operands lie:
//   k(u, i), k_second(u, i): the codes of row i of sub-tile u (16 tokens), token
//     kSubStep u + kHalfStep i + token(g); 16 bytes (8 at dim 64), and at dim 256
//     16 more
//   k_scale(u, i): its scales, two bytes (one at dim 64), the second pair of
//     dim 256 8 bytes on
//   v(u, i): dim/16 bytes of the V rows of the tokens that rows 2tq, 2tq + 1,
//     2tq + 8, 2tq + 9 of the accumulator stand for
//   v_scale(u, i): their scales (two bytes at dim 256, else one)
//   k_read(), v_wait(): called when K has been read and before V is
//   kRaw: absent tokens' rows hold anything, so their V scales are taken as 0;
//     else they are zeros
// j0: the tile's first token among the row's.
template <int D, int NT, typename At>
__device__ __forceinline__ void attend_tile(const AttentionParams& p, const RowSpan& r, int t,
                                            int head0, int heads, const At& at, uint32_t mask,
                                            int64_t j0, Heads<D, NT>& hd) {
  constexpr int kMTiles = D / 16;
  constexpr int kSub = kTile / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  // S^T: rows are tokens (see k above), columns the heads 2tq and 2tq + 1
  float s[NT][kSub][4];
#pragma unroll
  for (int u = 0; u < kSub; ++u) {
    constexpr int kWords = D / 32;  // per thread and row
    uint32_t kw[2][kWords], ks[2][(kWords + 3) / 4];  // ks: two blocks' scales each
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* sp = at.k_scale(u, i);
      if constexpr (D == 256) {
        uint32_t lo[4], hi[4];
        load_words<4>(at.k(u, i), lo);
        load_words<4>(at.k_second(u, i), hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) kw[i][e] = lo[e], kw[i][4 + e] = hi[e];
        ks[i][0] = scales_to_half(*reinterpret_cast<const uint16_t*>(sp));
        ks[i][1] = scales_to_half(*reinterpret_cast<const uint16_t*>(sp + 8));
      } else {
        load_words<kWords>(at.k(u, i), kw[i]);
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
        mma_f16(s[n][u], a[0][0], a[1][0], a[0][1], a[1][1], hd.qf[n][4 * w], hd.qf[n][4 * w + 1]);
        mma_f16(s[n][u], a[0][2], a[1][2], a[0][3], a[1][3], hd.qf[n][4 * w + 2],
                hd.qf[n][4 * w + 3]);
      }
    }
  }

  at.k_read();

  if (p.softcap > 0.0f) {
    const float cap = p.softcap * kLog2e;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][u][e] = cap * tanh_score(s[n][u][e] * hd.mult[n][e & 1]);
  }
  if (mask != 0xffffffffu) {
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!((mask >> (At::kSubStep * u + At::token(g) + At::kHalfStep * (e >> 1))) & 1u))
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][u][e] = -INFINITY;
  }
  if (p.scores) {
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int64_t tok = j0 + At::kSubStep * u + At::token(g) + At::kHalfStep * i;
        if constexpr (At::kRaw) tok -= r.skip;
        float* dst = p.scores + ((int64_t)t * p.width + tok) * p.q_heads + head0 + 2 * tq;
        if (At::kRaw ? tok >= 0 && tok < r.n - r.skip : tok < r.n)
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
      top[n][c] *= hd.late[n][c];
      past |= top[n][c] - hd.m[n][c] > kSlack;  // as a difference: exact where both are large
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
        const float mn = fmaxf(hd.m[n][c], x - kBelow);
        const float corr = exp2_approx(hd.m[n][c] - mn);
        hd.m[n][c] = mn;
        hd.l[n][c] *= corr, hd.over[n][c] *= corr;
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) hd.o[n][i][c] *= corr, hd.o[n][i][c + 2] *= corr;
      }
  }
  float add[NT][2];           // to the running sums
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) add[n][c] = -hd.over[n][c];
  uint32_t pf[NT][kSub][2];  // P^T: column head g, tokens of rows 2tq, 2tq + 1 and + 8
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][u][e] = exp2_approx(fmaf(s[n][u][e], hd.late[n][e & 1], -hd.m[n][e & 1]));
        add[n][e & 1] += s[n][u][e];
      }
      pf[n][u][0] = transpose8x8(pack_pair(s[n][u][0], s[n][u][1], DCP_F16));
      pf[n][u][1] = transpose8x8(pack_pair(s[n][u][2], s[n][u][3], DCP_F16));
    }
  // The running sum, compensated: what its last addition rounded off comes along
  // with the tile's tokens.  Without that, tokens of 2^-25 vanish beside a heavy
  // one: 2^17 of them were missing from lse by 1e-4.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float sum = hd.l[n][c] + add[n][c];
      hd.over[n][c] = (sum - hd.l[n][c]) - add[n][c];
      hd.l[n][c] = sum;
    }

  at.v_wait();
  // O^T: rows are elements g * D/8 + 2i and + 1 (tile i), columns heads
#pragma unroll
  for (int u = 0; u < kSub; ++u) {
    constexpr int kWords = D / 64;  // per thread and token
    constexpr int kBlocks = D == 256 ? 2 : 1;
    uint32_t vw[4][kWords];
    uint32_t vs[2][kBlocks];  // scales of the tokens' pairs, per block of the thread's elements
#pragma unroll
    for (int i = 0; i < 4; ++i) load_words<kWords>(at.v(u, i), vw[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t* x = at.v_scale(u, 2 * i);
      const uint8_t* y = at.v_scale(u, 2 * i + 1);
      if constexpr (D == 256) {
        uint32_t a = *reinterpret_cast<const uint16_t*>(x);
        uint32_t b = *reinterpret_cast<const uint16_t*>(y);
        if constexpr (At::kRaw)
          if (mask != 0xffffffffu)
            a &= present(at, u, 2 * i, mask), b &= present(at, u, 2 * i + 1, mask);
        vs[i][0] = scales_to_half(__byte_perm(a, b, 0x0040));
        vs[i][1] = scales_to_half(__byte_perm(a, b, 0x0051));
      } else {
        uint32_t a = x[0], b = y[0];
        if constexpr (At::kRaw)
          if (mask != 0xffffffffu)
            a &= present(at, u, 2 * i, mask), b &= present(at, u, 2 * i + 1, mask);
        vs[i][0] = scales_to_half(a + b * 256u);
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
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
          mma_f16(hd.o[n][4 * w + e], a[0][0][e], a[0][1][e], a[1][0][e], a[1][1][e],
                  pf[n][u][0], pf[n][u][1]);
    }
  }
}

struct __align__(16) Joined {
  float top, sum, x, y;  // reference, sum and two outputs of a head
};

// A row's finished head (`at` = row * q_heads + head): writes its logarithm of
// the sum if `write`, returns what its outputs are multiplied by.
__device__ __forceinline__ float write_sum(const AttentionParams& p, int64_t at, float top,
                                           float sum, bool write) {
  if (write) {
    p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    if (p.row_ml) p.row_ml[at] = make_float2(top, sum);
  }
  // no token: 0; a NaN sum goes through
  return sum == 0.0f ? 0.0f : p.c.v_unit / sum;
}

template <int D>
__device__ __forceinline__ void write_out(const AttentionParams& p, int64_t at, int d,
                                          const Joined& j) {
  const float inv = write_sum(p, at, j.top, j.sum, d == 0);
  reinterpret_cast<uint32_t*>(p.out)[(at * D + d) >> 1] = pack_pair(j.x * inv, j.y * inv, p.dtype);
}

// weights[t][pos] += sum over the query heads of 2^(x - m) / l, from m and l
// rather than lse, whose rounding would be an error of the exponent; the
// exponent is the attention's own, bit for bit.  8 lanes a token, 4 heads to a
// lane's load where the rows allow it, 4 tokens of a lane in flight; a CTA per
// 128 tokens of a row.  8 rows of up to 16384 tokens x 64 heads: 9 us after the
// attention, whose score writes are another 25 MB.
constexpr int kWeightTokens = 128;
constexpr int kMostWeightHeads = 4096;  // 48 KB of shared memory

template <bool kIds>
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(16) float weight_heads[];  // [q_heads] each, rounded up to 4
  const int padded = (p.q_heads + 3) & ~3;
  float* mult = weight_heads;  // multiplier, reference, 1 / sum
  float* ref = mult + padded;
  float* inv = ref + padded;
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
  constexpr int kMine = kWeightTokens / 32;  // tokens of a lane
  const int64_t first = j0 + (threadIdx.x >> 3);
  float sum[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) sum[i] = 0.0f;
  // a token beyond the last reads the last
  const float* x[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    x[i] = p.scores + ((int64_t)t * p.width + min(first + 32 * i, (int64_t)n - 1)) * p.q_heads;
  // absent tokens: 2^-inf = 0
  if (p.q_heads % 4 == 0) {
    for (int h = 4 * sub; h < p.q_heads; h += 32) {
      const float4 a = *reinterpret_cast<const float4*>(mult + h);
      const float4 b = *reinterpret_cast<const float4*>(ref + h);
      const float4 c = *reinterpret_cast<const float4*>(inv + h);
      float4 v[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) v[i] = *reinterpret_cast<const float4*>(x[i] + h);
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        sum[i] += exp2_approx(fmaf(v[i].x, a.x, -b.x)) * c.x +
                  exp2_approx(fmaf(v[i].y, a.y, -b.y)) * c.y +
                  exp2_approx(fmaf(v[i].z, a.z, -b.z)) * c.z +
                  exp2_approx(fmaf(v[i].w, a.w, -b.w)) * c.w;
    }
  } else {
    for (int h = sub; h < p.q_heads; h += 8)
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        sum[i] += exp2_approx(fmaf(x[i][h], mult[h], -ref[h])) * inv[h];
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 4);
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int64_t j = first + 32 * i;
      if (j >= n) continue;
      const int given = kIds ? __ldg(p.ids + (int64_t)t * p.ids_stride + j) : (int)j;
      const int pos = token_pos<kIds>(r, row_start, given);
      if (pos >= 0 && pos < p.weights_width) {
        // a head whose sum is NaN made the absent tokens' shares NaN, too
        if (sum[i] != sum[i] &&
            (uint32_t)__ldg(p.table + (int64_t)r.seq * p.table_stride +
                            (pos >> p.c.page_shift)) >= p.c.num_pages)
          continue;
        float* w = p.weights + (int64_t)t * p.weights_stride + pos;
        if constexpr (kIds)
          atomicAdd(w, sum[i]);  // an id may be listed twice
        else
          *w += sum[i];
      }
    }
  }
}

}  // namespace kv4
}  // namespace dcp
