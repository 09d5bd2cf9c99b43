// prompt_tiles.cuh -- attention over whole prompts on the tensor cores.
//
// A CTA takes one or two tiles of 128 query rows of one key/value head and
// walks over the keys that they see, a step of keys at a time:
//
//   S = Q K^T        tensor cores, operands in shared memory, S in tensor memory
//   P = 2^(S mult - ref), l += sum P      four warps a tile, a row a thread
//   O += P V         tensor cores, P in tensor memory over S, O in tensor memory
//
// A tile's rows are p query heads that share the key/value head times 128 / p
// tokens, so that a short prompt still fills the tile and the diagonal cuts off
// little.  ref is a reference that follows the row's maximum: set 2^8 below it,
// and moved (O and l multiplied by the difference) only once the maximum has
// passed it by 2^15, so that O is rarely read before the end.  P stays below
// fp16's 65504, and fp16's smallest step, 2^-24, is 2^-32 of the largest P.
//
// Two tiles take turns: while one's rows are exponentiated, the tensor cores
// work on the other's.  One warp issues the products, one the tensor copies
// (K and V of a step in turn through a ring of stages).
//
// Masked scores are -infinity and their P is 0, but 0 times an infinite or NaN
// value is NaN: rows whose O is not finite although their sum is are computed
// again by attend_row, which reads only what a row sees.  Values behind the
// sequence's end, where there may be anything, become zeros before the product.
#pragma once

#include "prompt_rows.cuh"
#include "tensor_core.cuh"

namespace dcp {
namespace prompt {

constexpr int kTileRows = 128;
constexpr float kBelow = 8.0f;  // a reference is set this far below the maximum
constexpr float kMost = 15.0f;  // and holds until the maximum is this far above

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;    // of queries
  static constexpr int kKeys = D == 256 ? 64 : 128;  // a step
  static constexpr int kStages = D == 64 ? 8 : 4;    // of K or V of a step
  static constexpr int kChunks = D / 64;             // of 64 elements, 128 bytes a row
  static constexpr int kQueryBytes = kTileRows * D * 2;
  static constexpr int kStageBytes = kKeys * D * 2;
  static constexpr int kRowWarps = 4 * kTiles;
  static constexpr int kThreads = 32 * (kRowWarps + 2);
  static constexpr int kColumns = 512;  // of tensor memory: S of each tile, then O of each
  static constexpr int kOut = kTiles * kKeys;
  static_assert(kOut + kTiles * D <= kColumns, "");
};

template <int D>
struct alignas(1024) Shared {
  using S = Shape<D>;
  uint8_t q[S::kTiles][S::kQueryBytes];
  uint8_t stage[S::kStages][S::kStageBytes];
  float rows[S::kRowWarps][D];  // attend_row's
  unsigned long long q_full, full[S::kStages], empty[S::kStages];
  unsigned long long s_full[S::kTiles], p_ready[S::kTiles], o_full[S::kTiles], drained;
  uint32_t tmem;
  int given_up;
  int first, n, block;  // the unit: its sequence's first row and length, its block (-1: none)
};

struct TileParams {
  Params p;
  unsigned int* status;
  int packed;  // p: query heads of a tile's rows
  int tokens;  // of a tile
  int sets;    // of packed heads: kv_heads * group / packed
  uint32_t q_bytes;  // of a tile's copy
};

// The u-th unit, those that lie furthest back in their sequences first, since
// they see the most keys.  By one warp.
template <int D>
__device__ __forceinline__ void find_unit(const Params& p, int tokens, int u, Shared<D>& s) {
  const int lane = threadIdx.x & 31;
  auto blocks = [&](int b) {
    if (b >= p.num_seqs) return 0;
    const int n = start_of(p, b + 1) - start_of(p, b);
    return n > 0 ? (n + tokens - 1) / tokens : 0;
  };
  int total = 0, most = 0;
  for (int b = lane; b < p.num_seqs; b += 32) {
    const int n = blocks(b);
    total += n;
    most = max(most, n);
  }
  total = __reduce_add_sync(~0u, total);
  most = __reduce_max_sync(~0u, most);
  if (u >= total) {
    if (lane == 0) s.block = -1;
    return;
  }
  // the last block of which there are more than u, counting all behind it
  int lo = 0, hi = most, behind = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int c = 0;
    for (int b = lane; b < p.num_seqs; b += 32) c += max(0, blocks(b) - mid);
    c = __reduce_add_sync(~0u, c);
    if (c > u) lo = mid; else hi = mid, behind = c;
  }
  int left = u - behind;  // among the sequences that have block lo
  for (int base = 0; base < p.num_seqs; base += 32) {
    const unsigned has = __ballot_sync(~0u, blocks(base + lane) > lo);
    const int c = __popc(has);
    if (left < c) {
      const int b = base + __fns(has, 0, left + 1);
      if (lane == 0) {
        s.first = start_of(p, b);
        s.n = start_of(p, b + 1) - s.first;
        s.block = lo;
      }
      return;
    }
    left -= c;
  }
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  uint32_t d;
  if constexpr (kHalf)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <int D>
__device__ __noinline__ void attend_row_again(const Params& p, int first, int n, int i, int h,
                                              float* q_row) {
  attend_row<D>(p, first, n, i, h, q_row);
}

template <int D, bool kHalf, bool kCapped>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
    tiles_kernel(const TileParams a, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<D>;
  constexpr int kKeys = Sh::kKeys, kTiles = Sh::kTiles, kStages = Sh::kStages;
  extern __shared__ uint8_t tiles_smem[];
  Shared<D>& s = *reinterpret_cast<Shared<D>*>(((uintptr_t)tiles_smem + 1023) & ~(uintptr_t)1023);
  const Params& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = blockIdx.x % a.sets;
  const int span = kTiles * a.tokens;  // tokens of a unit
  kv4::grid_dependency_wait();

  if (warp == 0) find_unit<D>(p, span, blockIdx.x / a.sets, s);
  if (warp == Sh::kRowWarps) {
    if (lane == 0) {
      mbar_init(&s.q_full, 1);
      mbar_init(&s.drained, 1);
      for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], 1);
      for (int t = 0; t < kTiles; ++t) {
        mbar_init(&s.s_full[t], 1);
        mbar_init(&s.p_ready[t], kTileRows);
        mbar_init(&s.o_full[t], 1);
      }
      s.given_up = 0;
      mbar_fence_init();
    }
    __syncwarp();
    tmem_allocate(&s.tmem, Sh::kColumns);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();

  const uint32_t tmem = s.tmem;
  const int first = s.first, n = s.n, q0 = s.block * span;
  if (s.block >= 0) {
    const int head0 = set * a.packed, kv = head0 / p.group;
    // the keys that the unit's rows see, and the steps of each tile over them
    const int from = p.window ? max(0, q0 - p.window + 1) : 0;
    int steps[kTiles], most = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int begin = q0 + t * a.tokens;
      const int to = p.causal ? min(n, begin + a.tokens) : n;
      steps[t] = begin < n ? (to - from + kKeys - 1) / kKeys : 0;
      most = max(most, steps[t]);
    }

    if (warp == Sh::kRowWarps + 1) {
      // ------------------------------------------------------------- copies
      if (lane == 0) {
        int tiles = 0;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) tiles += steps[t] > 0;
        mbar_expect_tx(&s.q_full, tiles * a.q_bytes);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < Sh::kChunks; ++c)
            tensor_load_3d(s.q[t] + c * kTileRows * 128, &q_map, c * 64, head0,
                           first + q0 + t * a.tokens, &s.q_full);
        int issued = 0;
        for (int i = 0; i < 2 * most; ++i) {
          const int slot = i % kStages, round = i / kStages;
          if (round && !wait_for(&s.empty[slot], (round - 1) & 1, &s.given_up, a.status)) break;
          mbar_expect_tx(&s.full[slot], Sh::kStageBytes);
          for (int c = 0; c < Sh::kChunks; ++c)
            tensor_load_3d(s.stage[slot] + c * kKeys * 128, i & 1 ? &v_map : &k_map, c * 64, kv,
                           first + from + (i >> 1) * kKeys, &s.full[slot]);
          ++issued;
        }
        if (s.given_up) {  // this thread's copies in flight, each for a limited time
          mbar_wait_bounded(&s.q_full, 0, kPatience);
          for (int i = max(0, issued - kStages); i < issued; ++i)
            mbar_wait_bounded(&s.full[i % kStages], (i / kStages) & 1, kPatience);
        }
      }
      __syncwarp();
    } else if (warp == Sh::kRowWarps) {
      // ----------------------------------------------------------- products
      constexpr uint32_t kScores = mma_shape(!kHalf, kTileRows, kKeys, false, false);
      constexpr uint32_t kOuts = mma_shape(!kHalf, kTileRows, D, false, true);
      // a negative scale: negated queries
      const uint32_t scores = kScores | (p.mult < 0.0f ? 1u << 13 : 0u);
      auto wait = [&](unsigned long long* bar, uint32_t parity) {
        const bool ok = wait_for(bar, parity, &s.given_up, a.status);
        tmem_fence_after();
        return __all_sync(~0u, ok);
      };
      auto multiply_scores = [&](int t, int slot) {
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t in_chunk = (i & 3) * 32;
            mma_smem(tmem + t * kKeys,
                     rows_along_k(smem_u32(s.q[t]) + (i >> 2) * kTileRows * 128 + in_chunk),
                     rows_along_k(smem_u32(s.stage[slot]) + (i >> 2) * kKeys * 128 + in_chunk),
                     scores, i > 0);
          }
          mma_commit(&s.s_full[t]);
        }
        __syncwarp();
      };
      bool ok = wait(&s.q_full, 0) && wait(&s.full[0], 0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          if (steps[t]) multiply_scores(t, 0);
        if (lane == 0 && kStages < 2 * most) mma_commit(&s.empty[0]);
      }
      for (int j = 0; ok && j < most; ++j) {
        const int v_at = 2 * j + 1, k_at = 2 * j + 2;
        const int v_slot = v_at % kStages, k_slot = k_at % kStages;
        ok = wait(&s.full[v_slot], (v_at / kStages) & 1);
        if (!ok) break;
        const int inside = n - from - j * kKeys;  // keys of this step in the sequence
        if (inside < kKeys) {
          for (int i = lane; i < (kKeys - inside) * 8 * Sh::kChunks; i += 32) {
            const int c = i / ((kKeys - inside) * 8), e = i - c * (kKeys - inside) * 8;
            *reinterpret_cast<uint4*>(s.stage[v_slot] + c * kKeys * 128 + inside * 128 + e * 16) =
                make_uint4(0, 0, 0, 0);
          }
          async_proxy_fence();
          __syncwarp();
        }
        bool next = false;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (j >= steps[t]) continue;
          ok = ok && wait(&s.p_ready[t], j & 1);
          if (!ok) break;
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
              mma_tmem(tmem + Sh::kOut + t * D, tmem + t * kKeys + i * 8,
                       rows_across_k(smem_u32(s.stage[v_slot]) + i * 2048, kKeys * 128), kOuts,
                       j > 0 || i > 0);
          }
          __syncwarp();
          if (j + 1 < steps[t]) {
            if (!next) ok = wait(&s.full[k_slot], (k_at / kStages) & 1);
            next = true;
            if (!ok) break;
            multiply_scores(t, k_slot);
          } else if (lane == 0) {
            mma_commit(&s.o_full[t]);
          }
        }
        if (ok && lane == 0) {
          if (v_at + kStages < 2 * most) mma_commit(&s.empty[v_slot]);
          if (next && k_at + kStages < 2 * most) mma_commit(&s.empty[k_slot]);
        }
        __syncwarp();
      }
      if (!ok) {  // the products in flight, for a limited time
        if (lane == 0) {
          mma_commit(&s.drained);
          mbar_wait_bounded(&s.drained, 0, kPatience);
        }
        __syncwarp();
      }
    } else {
      // --------------------------------------------------------------- rows
      const int t = warp >> 2;
      const int row = 32 * (warp & 3) + lane;
      const int token = row / a.packed;
      const int i = q0 + t * a.tokens + token, head = head0 + row - token * a.packed;
      const bool valid = token < a.tokens && i < n;
      // the keys that the row sees, counted from the first step's first
      const int lo = valid && p.window ? max(0, i - p.window + 1) - from : 0;
      const int hi = valid ? (p.causal ? i + 1 : n) - from : INT32_MAX;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t s_at = tmem + lanes + t * kKeys;
      const uint32_t o_at = tmem + lanes + Sh::kOut + t * D;
      const float mult = fabsf(p.mult), late = kCapped ? 1.0f : mult;
      float ref = -INFINITY, l = 0.0f, over = 0.0f;  // over: what l is too large by
      bool ok = true;
      const int my_steps = t == 0 ? steps[0] : steps[kTiles - 1];
      for (int j = 0; j < my_steps; ++j) {
        ok = wait_for(&s.s_full[t], j & 1, &s.given_up, a.status);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        tmem_fence_after();
        uint32_t raw[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys / 64; ++c) tmem_load64(s_at + 64 * c, raw + 64 * c);
        float* x = reinterpret_cast<float*>(raw);
        if constexpr (kCapped) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e) x[e] = p.cap * kv4::tanh_score(x[e] * mult);
        }
        const int base = j * kKeys;
        if (__any_sync(~0u, base < lo || base + kKeys > hi)) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e)
            if (base + e < lo || base + e >= hi) x[e] = -INFINITY;
        }
        float top4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int e = 4; e < kKeys; e += 4)
#pragma unroll
          for (int f = 0; f < 4; ++f) top4[f] = fmaxf(top4[f], x[e + f]);
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * late;
        const bool moves = top > ref + kMost;
        if (__any_sync(~0u, moves)) {
          float shrink = 1.0f;
          if (moves) {
            const float next = top - kBelow;
            shrink = exp2f(ref - next);  // 0 at first
            ref = next;
            l *= shrink;
            over *= shrink;
          }
          // S of this step came after the products with the last one's P
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_load32(o_at + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
              tmem_store32(o_at + c, o);
            }
          }
        }
        const float less = ref == -INFINITY ? 0.0f : -ref;
        float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int c = 0; c < kKeys; c += 64) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float2 y = fma2(make_float2(x[c + e], x[c + e + 1]), make_float2(late, late),
                            make_float2(less, less));
            y.x = kv4::exp2_approx(y.x);
            y.y = kv4::exp2_approx(y.y);
            sum[e / 2 & 1] = add2(sum[e / 2 & 1], y);
            w[e / 2] = round_pair<kHalf>(y.x, y.y);
          }
          tmem_store32(s_at + c / 2, w);
        }
        tmem_wait_store();
        tmem_fence_before();
        mbar_arrive(&s.p_ready[t]);
        const float2 both = add2(sum[0], sum[1]);
        const float add = both.x + both.y - over, now = l + add;
        over = (now - l) - add;
        l = now;
      }
      if (my_steps > 0) {
        ok = ok && wait_for(&s.o_full[t], 0, &s.given_up, a.status);
        ok = __all_sync(~0u, ok);
        tmem_fence_after();
        const float inverse = ok ? (l == 0.0f ? 0.0f : 1.0f / l) : NAN;
        const int64_t out_row = (int64_t)(first + i) * p.q_heads + head;
        bool finite = true;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_load32(o_at + c, o);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float y0 = __uint_as_float(o[e]), y1 = __uint_as_float(o[e + 1]);
            finite = finite && fabsf(y0) <= 3.4028234e38f && fabsf(y1) <= 3.4028234e38f;
            w[e / 2] = round_pair<kHalf>(y0 * inverse, y1 * inverse);
          }
          if (valid) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                                 (out_row * D + c) * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        }
        if (valid)
          p.lse[out_row] = !ok ? NAN : l == 0.0f ? -INFINITY : kLn2 * (ref + log2f(l));
        // a NaN among the scores that the row sees makes the sum NaN, and is right
        unsigned again = __ballot_sync(~0u, ok && valid && !finite && l == l);
        while (again) {
          const int at = __ffs(again) - 1;
          again &= again - 1;
          attend_row_again<D>(p, first, n, __shfl_sync(~0u, i, at), __shfl_sync(~0u, head, at),
                              s.rows[warp]);
        }
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == Sh::kRowWarps) tmem_free(tmem, Sh::kColumns);
}

}  // namespace prompt
}  // namespace dcp
