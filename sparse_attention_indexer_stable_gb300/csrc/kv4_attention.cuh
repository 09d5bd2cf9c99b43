// kv4_attention.cuh -- attention of single query rows over the 4-bit cache.
//
// For one row and one key/value head, with the group's query heads q_h and
// the visible tokens j:
//   x_hj = c(q_h . k_j) in units of log2,  out_h = sum_j 2^(x_hj - m_h) v_j / l_h
// with m_h a reference within 2^8 of the running maximum and l_h the running
// sum.  A token costs dim + dim/8 bytes and 4 * dim operations per query
// head, so with up to 16 heads to a group the cache's bytes bound it.
//
// A CTA of 8 warps takes one row, one key/value head, up to 8 * NT of its
// query heads and one slice of the tokens; each warp walks tiles of 16 tokens
// on its own, so nothing but the final join synchronises the CTA.
//  - Tiles come in by cp.async, a ring per warp: every thread fetches exactly
//    the bytes that it will convert, wherever the token's page lies, so a
//    gather by ids costs the same instructions as a range.
//  - S^T = K Q^T and O^T = V^T P^T by mma m16n8k16 (tokens and then elements
//    of the head as rows, query heads as columns): up to 8 heads fill the
//    8 columns, where P Q^T would leave half of 16 rows empty.  tcgen05 wants
//    64 or 128 rows and operands in shared memory; here the converted values
//    go straight from registers into the product.
//  - The sum over dim may run in any order: thread tq of a row takes dim/4
//    contiguous elements, so its codes are one wide load.  In V^T thread g
//    takes dim/8 contiguous elements of four tokens; nibbles of two tokens are
//    paired before the conversion, which then yields the operand's pairs.
//  - codes and scales multiply exactly in fp16 (at most 6 significant bits).
//  - P moves from the accumulator's layout to the operand's by one transpose
//    of 8x8 matrices per 8 tokens (movmatrix).
//  - The accumulator is rescaled only when a score passes the reference by
//    2^8 (fp16 holds P up to 65504), which after the first tiles is rare.
#pragma once

#include <cfloat>

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
  float* part_out;    // [rows][q_heads][splits][dim], when splits > 1
  float2* part_ml;    // [rows][q_heads][splits]: reference and sum
  float* scores;      // [rows][width][q_heads] in log2 units, when weights are wanted
  float2* row_ml;     // [rows][q_heads]: the whole row's reference and sum, likewise
  float* weights;
  int64_t weights_stride, weights_width;
  int dtype, rows, q_heads, group, head_tiles, num_seqs, splits;
  int limit;          // positions end here at the latest
  int num_ids;
  int width;          // tokens per row of `scores`
  bool q_vec;
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

// Shared memory of one warp's stage: the K words of rows g and g + 8, the V
// words of tokens 2tq, 2tq+1, 2tq+8, 2tq+9, each thread's own; the 16 tokens'
// K and V scales; the tile's mask of present tokens.
template <int D>
struct Stage {
  static constexpr int kKBytes = D / 8;   // per thread and row
  static constexpr int kVBytes = D / 16;  // per thread and token
  static constexpr int kSBytes = D / 16;  // per token
  static constexpr int kV = 2 * 32 * kKBytes;
  static constexpr int kS = kV + 4 * 32 * kVBytes;
  static constexpr int kMask = kS + 32 * kSBytes;
  static constexpr int kBytes = kMask + 16;
};

template <int D, int NT>
struct AttentionShape {
  static constexpr int kStages = D == 256 ? 3 : 4;
  static constexpr int kRing = kStages * Stage<D>::kBytes;  // per warp
  // the join: each warp's outputs (padded rows), references and sums
  static constexpr int kOutStride = D + 4;
  static constexpr int kJoin = kAttWarps * 8 * NT * (kOutStride + 2) * 4;
  static constexpr int kSmem = kAttWarps * kRing > kJoin ? kAttWarps * kRing : kJoin;
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

// The group's query heads of this tile as the B operand of S^T = K Q^T: head
// g, elements [tq * D/4, (tq+1) * D/4), scaled by a power of two so that the
// head's largest magnitude is in [2^14, 2^15): bf16's 8 and fp16's 11 bits
// then fit fp16 for all elements within 2^-28 of the largest.  Returns the
// power of two to undo.  Heads beyond the group are zeros.
template <int D>
__device__ __forceinline__ float load_query(const AttentionParams& p, int t, int head, bool ok,
                                            int tq, uint32_t (&qf)[D / 8]) {
  float f[D / 4];
  const int64_t at = (int64_t)t * p.q_row_stride + (int64_t)head * p.q_head_stride + tq * (D / 4);
  if (!ok) {
#pragma unroll
    for (int e = 0; e < D / 4; ++e) f[e] = 0.0f;
  } else if (p.q_vec) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at);
#pragma unroll
    for (int v = 0; v < D / 32; ++v) {
      const uint4 x = __ldg(src + v);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.dtype == DCP_BF16) {
          f[8 * v + 2 * e] = __uint_as_float(w[e] << 16);
          f[8 * v + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        } else {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(w + e));
          f[8 * v + 2 * e] = h.x, f[8 * v + 2 * e + 1] = h.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < D / 4; ++e) f[e] = load_element(p.q, at + e, p.dtype);
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
  const float up1 = __uint_as_float((uint32_t)(127 + shift / 2) << 23);
  const float up2 = __uint_as_float((uint32_t)(127 + shift - shift / 2) << 23);
#pragma unroll
  for (int e = 0; e < D / 8; ++e)
    qf[e] = pack_pair(f[2 * e] * up1 * up2, f[2 * e + 1] * up1 * up2, DCP_F16);
  return __uint_as_float((uint32_t)(127 - shift / 2) << 23) *
         __uint_as_float((uint32_t)(127 - (shift - shift / 2)) << 23);
}

template <int D, int NT, bool kIds>
__global__ void __launch_bounds__(kAttThreads, D * NT >= 256 ? 1 : 2)
    attention_kernel(const __grid_constant__ AttentionParams p) {
  using S = Stage<D>;
  using Shape = AttentionShape<D, NT>;
  constexpr int kMTiles = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;

  // blockIdx.x = ((row * splits + split) * head_tiles + head tile) * heads + head
  int64_t rest = blockIdx.x;
  const int h = (int)(rest % p.c.heads);
  rest /= p.c.heads;
  const int ht = (int)(rest % p.head_tiles);
  rest /= p.head_tiles;
  const int split = (int)(rest % p.splits);
  const int t = (int)(rest / p.splits);
  const int head0 = h * p.group + ht * 8 * NT;             // first query head of this CTA
  const int heads = min(8 * NT, p.group - ht * 8 * NT);    // and how many

  grid_dependency_wait();
  const RowSpan r = row_span<kIds>(p, t);
  // slices of whole tiles; 64-bit because n may be near 2^31
  const int64_t chunk = (((int64_t)r.n + p.splits - 1) / p.splits + 15) & ~(int64_t)15;
  const int c0 = (int)min((int64_t)r.n, split * chunk);
  const int c1 = (int)min((int64_t)r.n, (split + 1) * chunk);
  const int tiles = (c1 - c0 + 15) >> 4;
  const int mine = tiles > warp ? (tiles - warp + kAttWarps - 1) / kAttWarps : 0;
  const int row_start = kIds && p.row_starts ? __ldg(p.row_starts + t) : 0;
  const int32_t* table = p.table + (int64_t)r.seq * p.table_stride;

  uint8_t* ring = smem + warp * Shape::kRing;
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);

  // This lane's token of the warp's k-th tile: lane & 15.
  auto pos_of = [&](int k) {
    const int64_t j = c0 + 16 * ((int64_t)warp + (int64_t)kAttWarps * k) + (lane & 15);
    return k < mine && j < c1 ? token_pos<kIds>(p, r, t, row_start, (int)j) : -1;
  };
  auto page_of = [&](int pos) { return pos >= 0 ? __ldg(table + (pos >> p.c.page_shift)) : -1; };

  // The position and page of the next tile to fetch, and the position after
  // it: loaded one and two tiles ahead of the copies that need them.
  int pos0 = pos_of(0);
  int pos1 = pos_of(1);
  int page0 = page_of(pos0);

  auto issue = [&](int k) {
    if (k < mine) {
      const uint32_t st = ring_addr + (uint32_t)((k % Shape::kStages) * S::kBytes);
      const bool ok = (uint32_t)page0 < p.c.num_pages;
      const uint32_t slot =
          ok ? ((uint32_t)page0 << p.c.page_shift) | (pos0 & ((1u << p.c.page_shift) - 1u)) : 0u;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const uint32_t heads_kv = (uint32_t)p.c.heads;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = g + 8 * i;
        const uint64_t row =
            (uint64_t)__shfl_sync(0xffffffffu, slot, tok) * heads_kv + (uint32_t)h;
        const uint8_t* src = p.c.k_codes + row * (D / 2) + tq * S::kKBytes;
        const bool there = (mask >> tok) & 1u;
        if constexpr (S::kKBytes == 32) {
          cp_async<16>(st + (2 * i * 32 + lane) * 16, src, there);
          cp_async<16>(st + ((2 * i + 1) * 32 + lane) * 16, src + 16, there);
        } else {
          cp_async<S::kKBytes>(st + (i * 32 + lane) * S::kKBytes, src, there);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 2 * tq + (i & 1) + 8 * (i >> 1);
        const uint64_t row =
            (uint64_t)__shfl_sync(0xffffffffu, slot, tok) * heads_kv + (uint32_t)h;
        cp_async<S::kVBytes>(st + S::kV + (i * 32 + lane) * S::kVBytes,
                             p.c.v_codes + row * (D / 2) + g * S::kVBytes, (mask >> tok) & 1u);
      }
      {
        const uint64_t row = (uint64_t)slot * heads_kv + (uint32_t)h;
        cp_async<S::kSBytes>(st + S::kS + lane * S::kSBytes,
                             (lane < 16 ? p.c.k_scales : p.c.v_scales) + row * S::kSBytes, ok);
      }
      if (lane == 0)
        *reinterpret_cast<uint32_t*>(ring + (k % Shape::kStages) * S::kBytes + S::kMask) = mask;
      pos0 = pos1;
      page0 = page_of(pos0);
      pos1 = pos_of(k + 2);
    }
    cp_async_commit();
  };

  for (int k = 0; k < Shape::kStages - 1; ++k) issue(k);

  // Queries while the first tiles are under way.
  uint32_t qf[NT][D / 8];
  float mult[NT][2];  // of the columns 2tq, 2tq+1: to log2 units (or to units of the cap)
  const float unit = p.softcap > 0.0f ? p.scale / p.softcap : p.scale * kLog2e;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float undo =
        load_query<D>(p, t, head0 + 8 * n + g, 8 * n + g < heads, tq, qf[n]) * unit;
    mult[n][0] = __shfl_sync(0xffffffffu, undo, 8 * tq);
    mult[n][1] = __shfl_sync(0xffffffffu, undo, 8 * tq + 4);
  }
  const float cap = p.softcap * kLog2e;

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

  for (int k = 0; k < mine; ++k) {
    __syncwarp();  // the stage that issue() refills has been read by every lane
    issue(k + Shape::kStages - 1);
    cp_async_wait<Shape::kStages - 1>();
    __syncwarp();  // the other lanes' scales and the mask
    const uint8_t* st = ring + (k % Shape::kStages) * S::kBytes;
    const uint32_t mask = *reinterpret_cast<const uint32_t*>(st + S::kMask);

    // S^T: rows are tokens g and g + 8, columns the heads 2tq and 2tq + 1
    float s[NT][4];
    {
      constexpr int kWords = D / 32;  // per thread and row
      uint32_t kw[2][kWords], ks[2][D / 64];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (kWords == 8) {
          uint32_t lo[4], hi[4];
          load_words<4>(st + (2 * i * 32 + lane) * 16, lo);
          load_words<4>(st + ((2 * i + 1) * 32 + lane) * 16, hi);
#pragma unroll
          for (int e = 0; e < 4; ++e) kw[i][e] = lo[e], kw[i][4 + e] = hi[e];
        } else {
          load_words<kWords>(st + (i * 32 + lane) * S::kKBytes, kw[i]);
        }
        const uint8_t* sp = st + S::kS + (g + 8 * i) * S::kSBytes + tq * (D / 64);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) ks[i][b] = scales_to_half((uint32_t)sp[b] * 0x101u);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          codes_to_half(kw[i][w], a[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[i][e] = hmul2(a[i][e], ks[i][w >> 1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(s[n], a[0][0], a[1][0], a[0][1], a[1][1], qf[n][4 * w], qf[n][4 * w + 1]);
          mma_f16(s[n], a[0][2], a[1][2], a[0][3], a[1][3], qf[n][4 * w + 2], qf[n][4 * w + 3]);
        }
      }
    }

    const bool there[2] = {((mask >> g) & 1u) != 0u, ((mask >> (g + 8)) & 1u) != 0u};
    bool past = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[n][e] * mult[n][e & 1];
        if (p.softcap > 0.0f) x = cap * tanhf(x);
        x = there[e >> 1] ? x : -INFINITY;
        s[n][e] = x;
        past |= x > m[n][e & 1] + kSlack;
      }
    if (p.scores) {
      const int64_t j = c0 + 16 * ((int64_t)warp + (int64_t)kAttWarps * k);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t tok = j + g + 8 * (e >> 1);
          const int head = 8 * n + 2 * tq + (e & 1);
          if (tok < c1 && head < heads)
            p.scores[((int64_t)t * p.width + tok) * p.q_heads + head0 + head] = s[n][e];
        }
    }
    if (__any_sync(0xffffffffu, past)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(s[n][c], s[n][c + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float mn = fmaxf(m[n][c], top);
          const float corr = exp2_approx(m[n][c] - mn);
          m[n][c] = mn;
          l[n][c] *= corr;
#pragma unroll
          for (int i = 0; i < kMTiles; ++i) o[n][i][c] *= corr, o[n][i][c + 2] *= corr;
        }
    }
    uint32_t pf[NT][2];  // P^T: columns head g, tokens 2tq, 2tq+1 and 2tq+8, 2tq+9
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_approx(s[n][e] - m[n][e & 1]);
        l[n][e & 1] += s[n][e];
      }
      pf[n][0] = transpose8x8(pack_pair(s[n][0], s[n][1], DCP_F16));
      pf[n][1] = transpose8x8(pack_pair(s[n][2], s[n][3], DCP_F16));
    }

    // O^T: rows are elements g * D/8 + 2i and + 1 (tile i), columns heads
    {
      constexpr int kWords = D / 64;  // per thread and token
      uint32_t vw[4][kWords];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_words<kWords>(st + S::kV + (i * 32 + lane) * S::kVBytes, vw[i]);
      // scale pairs of tokens (2tq, 2tq+1) and (2tq+8, 2tq+9): one block of
      // the thread's elements per 16 (half a block at D = 64)
      constexpr int kBlocks = D / 128 > 0 ? D / 128 : 1;
      uint32_t vs[2][kBlocks];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint8_t* sp = st + S::kS + (16 + 2 * tq + 8 * i) * S::kSBytes +
                              (D >= 128 ? g * kBlocks + b : g >> 1);
          vs[i][b] = scales_to_half((uint32_t)sp[0] | ((uint32_t)sp[S::kSBytes] << 8));
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
            mma_f16(o[n][4 * w + e], a[0][0][e], a[0][1][e], a[1][0][e], a[1][1][e], pf[n][0],
                    pf[n][1]);
      }
    }
  }

  // Join of the warps: each leaves its reference, sum and outputs; then the
  // CTA adds them up under the largest reference.
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
  const float v_unit = p.c.v_unit;
  for (int i = threadIdx.x; i < heads * (D / 2); i += kAttThreads) {
    const int head = i / (D / 2), d = 2 * (i % (D / 2));
    float top = kNoScore;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, join_m[w * 8 * NT + head]);
    float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      const int col = w * 8 * NT + head;
      const float f = exp2_approx(join_m[col] - top);
      const float2 v = *reinterpret_cast<const float2*>(join_o + col * Shape::kOutStride + d);
      sum += f * join_l[col];
      x += f * v.x;
      y += f * v.y;
    }
    const int64_t at = (int64_t)t * p.q_heads + head0 + head;
    if (p.splits == 1) {
      // no token: 0; a NaN sum goes through
      const float inv = sum == 0.0f ? 0.0f : v_unit / sum;
      reinterpret_cast<uint32_t*>(p.out)[(at * D + d) >> 1] = pack_pair(x * inv, y * inv, p.dtype);
      if (d == 0) {
        p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        if (p.row_ml) p.row_ml[at] = make_float2(top, sum);
      }
    } else {
      *reinterpret_cast<float2*>(p.part_out + (at * p.splits + split) * D + d) = make_float2(x, y);
      if (d == 0) p.part_ml[at * p.splits + split] = make_float2(top, sum);
    }
  }
}

// Joins a row's slices: one CTA of 4 warps per row and query head, the slices
// dealt to the warps, a lane holding D / 32 contiguous elements.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kPer = D / 32;
  __shared__ float red[4][D];
  __shared__ float red_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t at = blockIdx.x;  // row * q_heads + head
  grid_dependency_wait();
  const float2* ml = p.part_ml + at * p.splits;
  float top = kNoScore;
  for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, ml[s].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  float acc[kPer], sum = 0.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.0f;
  for (int s = warp; s < p.splits; s += 4) {
    const float2 v = ml[s];
    if (v.y == 0.0f) continue;  // an empty slice
    const float f = exp2_approx(v.x - top);
    const float* src = p.part_out + (at * p.splits + s) * D + lane * kPer;
    sum += f * v.y;
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float2 w = *reinterpret_cast<const float2*>(src + e);
      acc[e] += f * w.x;
      acc[e + 1] += f * w.y;
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) red[warp][lane * kPer + e] = acc[e];
  if (lane == 0) red_l[warp] = sum;
  __syncthreads();
  sum = red_l[0] + red_l[1] + red_l[2] + red_l[3];
  const float inv = sum == 0.0f ? 0.0f : p.c.v_unit / sum;
  for (int d = 2 * threadIdx.x; d < D; d += 256) {
    const float x = red[0][d] + red[1][d] + red[2][d] + red[3][d];
    const float y = red[0][d + 1] + red[1][d + 1] + red[2][d + 1] + red[3][d + 1];
    reinterpret_cast<uint32_t*>(p.out)[(at * D + d) >> 1] = pack_pair(x * inv, y * inv, p.dtype);
  }
  if (threadIdx.x == 0) {
    p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    if (p.row_ml) p.row_ml[at] = make_float2(top, sum);
  }
}

// weights[t][pos] += sum over the query heads of 2^(x - m) / l: 8 lanes per
// token, a CTA per 1024 tokens of a row.  From m and l rather than lse, whose
// rounding would be an error of the exponent.
constexpr int kWeightTokens = 1024;

template <bool kIds>
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ float2 ml[];  // [q_heads]: reference, 1 / sum
  const int tiles = (p.width + kWeightTokens - 1) / kWeightTokens;
  const int t = blockIdx.x / tiles;
  const int64_t j0 = (int64_t)(blockIdx.x % tiles) * kWeightTokens;
  grid_dependency_wait();
  const RowSpan r = row_span<kIds>(p, t);
  const int n = min(r.n, p.width);
  if (j0 >= n) return;
  for (int h = threadIdx.x; h < p.q_heads; h += 256) {
    const float2 v = p.row_ml[(int64_t)t * p.q_heads + h];
    ml[h] = make_float2(v.x, v.y == 0.0f ? 0.0f : 1.0f / v.y);
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
        const float2 v = ml[h];
        sum += exp2_approx(x[h] - v.x) * v.y;  // absent tokens: 2^-inf = 0
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
