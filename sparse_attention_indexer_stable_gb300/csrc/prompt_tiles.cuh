// prompt_tiles.cuh -- attention over whole prompts on the tensor cores.
//
// A unit of work is one tile, or two, of 128 query rows of one key/value head.
// It walks over the keys that its rows see, 128 a step:
//
//   S = Q K^T        tensor cores, operands in shared memory, S in tensor memory
//   P = 2^(S mult - ref), l += sum P      four warps a tile, a row a thread
//   O += P V         tensor cores, P and O in tensor memory
//
// A tile's rows are p query heads that share the key/value head times 128 / p
// tokens, so that a short prompt still fills the tile and the diagonal cuts off
// little.  ref is a reference that follows the row's maximum and stands while P
// fits its type, so that O is rarely read before the end:
// - fp16: set 2^4 below the maximum, until P passes 2^15 (of 65504); fp16's
//   smallest step, 2^-24, is then 2^-28 of the largest P or less.
// - bf16, which has fp32's range: set at the maximum, until P passes 2^60.
//
// What bounds a step is the tensor cores' time for both products, or, for heads
// of 64, the chain of a row's thread (wait, load, 128 exponentials, hand over; no
// pipe is above 45%); the rest has to happen meanwhile:
// - Two tiles to an SM: while one's rows are exponentiated, the tensor cores work
//   on the other's.  Heads of 128: one CTA with both tiles, which share the keys
//   (a CTA each: 26% longer for 16384 rows).  Heads of 64: two CTAs
//   of a tile, whose ends do not coincide (one with both: 233 us, instead of 212,
//   for 16 texts of 1200 rows).  Heads of 256 leave room for one tile.
// - Heads of 128: S and O of two tiles fill tensor memory, P takes S's place.
//   Heads of 64 and 256 leave room for P beside S, and the next S is computed as
//   soon as the rows have read the last; P then goes over whole.
// - P over S comes in two halves, and its product begins with the first.
// - A CTA stays on its SM and takes unit after unit: one warp fetches the next
//   unit from the grid's CTAs that have not started yet, one issues the copies,
//   one a tile's products, so that the next unit's copies and first S overlap the
//   last one's end.
//
// Measured: one prompt of 16384 rows, 64 heads of 128 over 8: ten calls in a row, at
// 2070 MHz, 2435 us each, 1.81 PFLOP/s, 93% of the matrix rate measured so; for
// seconds, under the power cap and at 1770 MHz, 2690 us, 1.64 PFLOP/s, 94% of the
// rate measured so.  A step of both tiles takes 2500 to 3200 cycles, its products
// 2048.
//
// Masked scores are -infinity and their P is 0, but 0 times an infinite or NaN
// value is NaN: rows whose O is not finite although their sum is are looked at by
// attend_again, and computed again from what they see alone unless that is what
// makes them so (as are rows whose scores are too large for the exponents' way of
// rounding, see kFar).  Values behind the last sequence, where there may be
// anything, become zeros before the product.
#pragma once

#include <type_traits>

#include "prompt_rows.cuh"
#include "tensor_core.cuh"

namespace dcp {
namespace prompt {

constexpr int kTileRows = 128;
constexpr int kKeys = 128;  // a step
constexpr int kRing = 2;    // units on their way

template <int D>
struct Shape {
  static constexpr int kTiles = D == 128 ? 2 : 1;      // of queries
  static constexpr bool kBeside = D != 128;            // P beside S
  static constexpr int kPart = D < 128 ? D : 128;      // elements of a stage's rows
  static constexpr int kParts = D / kPart;             // stages of a step's K, or V
  static constexpr int kStages = 4;
  static constexpr int kChunks = D / 64;               // of 64 elements, 128 bytes a row
  static constexpr int kPartChunks = kPart / 64;
  static constexpr int kQueryBytes = kTileRows * D * 2;
  static constexpr int kStageBytes = kKeys * kPart * 2;
  static constexpr int kRowWarps = 4 * kTiles;
  static constexpr int kThreads = 32 * (kRowWarps + 4);
  // columns of tensor memory
  static constexpr int kCtas = D == 64 ? 2 : 1;  // of an SM
  static constexpr int kColumns = 512 / kCtas;
  static constexpr int kP = kBeside ? kTiles * kKeys : 0;
  static constexpr int kPStep = kBeside ? kKeys / 2 : kKeys;
  static constexpr int kOut = D == 64 ? 192 : 256;
  static_assert(kOut + kTiles * D <= kColumns && (!kBeside || kP + kTiles * kPStep <= kOut), "");
  // registers of the row warps and of the others: their sum is what the CTA is
  // launched with (168 a thread for heads of 128, 128 for those of 64)
  static constexpr int kRowRegisters = 200, kOtherRegisters = D == 64 ? 56 : 104;
};

struct Unit {
  int first, n;  // its sequence
  int q0;        // its first row there (-1: no more units)
  int set;       // of heads
};

template <int D>
struct alignas(1024) Shared {
  using S = Shape<D>;
  uint8_t q[S::kTiles][S::kQueryBytes];
  uint8_t stage[S::kStages][S::kStageBytes];
  uint4 rows[S::kRowWarps][32][8];  // of 64 outputs on their way to memory
  uint4 fetched;  // the next CTA's index, as the hardware reports it
  unsigned long long fetch_done, drained[S::kTiles];
  unsigned long long unit_full[kRing], unit_empty[kRing];
  unsigned long long full[S::kStages], empty[S::kStages];
  unsigned long long q_full[S::kTiles], q_empty[S::kTiles];
  unsigned long long s_full[S::kTiles], s_read[S::kTiles];
  unsigned long long p_ready[S::kTiles][2];
  unsigned long long o_done[S::kTiles], o_read[S::kTiles];
  unsigned long long turn[S::kTiles];
  Unit unit[kRing];
  uint32_t tmem;
  int given_up, beats;  // see Patience
};

struct TileParams {
  Params p;
  unsigned int* status;
  int packed;  // p: query heads of a tile's rows
  int tokens;  // of a tile
  int sets;    // of packed heads: kv_heads * group / packed
  int sms;
  uint32_t q_bytes;  // of a tile's copy
#ifdef DCP_DEBUG_POISON
  int withheld_cta, withheld_unit, withheld_copy;  // see dcp_prompt_selftest_withhold
#endif
  int out_box;       // whether 32 of a tile's rows are a box of the output
};

// Finds the u-th unit of the sequences (quickly where u grows from call to call):
// those that lie furthest back in their sequences come first, since they see the
// most keys.  By one warp.
struct Finder {
  int level = -1;            // the block whose units are being taken
  int behind = 0, here = 0;  // units of later blocks, and of this one
  int base = 0, passed = 0;  // this block's units in the sequences before base
  int total = -1;            // units, once known
  int kept = 0;              // blocks of the lane's sequence of the first 32

  __device__ int blocks(const Params& p, int tokens, int b) const {
    if (b >= p.num_seqs) return 0;
    const int n = start_of(p, b + 1) - start_of(p, b);
    return n > 0 ? (n + tokens - 1) / tokens : 0;
  }
  __device__ void begin(const Params& p, int tokens) {
    kept = blocks(p, tokens, threadIdx.x & 31);
  }
  // units whose block is `from` or later
  __device__ int count(const Params& p, int tokens, int from) const {
    int c = max(0, kept - from);
#pragma unroll 1
    for (int b = 32 + (threadIdx.x & 31); b < p.num_seqs; b += 32)
      c += max(0, blocks(p, tokens, b) - from);
    return __reduce_add_sync(~0u, c);
  }

  __device__ __forceinline__ Unit find(const Params& p, int tokens, int u) {
    const int lane = threadIdx.x & 31;
    if (u < behind + passed) level = -1, behind = here = base = passed = 0;
    if (total < 0) total = count(p, tokens, 0);
    if (u >= total) return Unit{0, 0, -1, 0};
    if (level < 0 || u >= behind + here) {
      int lo = 0, hi = level, at_hi = behind, at_lo = total;
      if (level < 0) {
        hi = kept;
#pragma unroll 1
        for (int b = 32 + lane; b < p.num_seqs; b += 32) hi = max(hi, blocks(p, tokens, b));
        hi = __reduce_max_sync(~0u, hi);
      } else {
        at_hi += here;
      }
      while (hi - lo > 1) {  // the last block with more than u units from it on
        const int mid = (lo + hi) >> 1;
        const int c = count(p, tokens, mid);
        if (c > u) lo = mid, at_lo = c; else hi = mid, at_hi = c;
      }
      level = lo, behind = at_hi, here = at_lo - at_hi;
      base = passed = 0;
    }
#pragma unroll 1
    for (; base < p.num_seqs; base += 32) {
      const unsigned has =
          __ballot_sync(~0u, (base ? blocks(p, tokens, base + lane) : kept) > level);
      const int left = u - behind - passed;
      if (left < __popc(has)) {
        const int b = base + __fns(has, 0, left + 1);
        const int first = start_of(p, b);
        return Unit{first, start_of(p, b + 1) - first, level * tokens, 0};
      }
      passed += __popc(has);
    }
    return Unit{0, 0, -1, 0};
  }
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
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

// The three-input maximum.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// tanh(u) / u as a polynomial in u^2 for |u| <= 1, relative error below 2^-20.5
// (weighted least squares iterated towards equal extremes).
constexpr int kTanhTerms = 6;
__device__ constexpr float kTanh[kTanhTerms] = {0x1.ffffecp-1f,  -0x1.554a16p-2f, 0x1.1000f8p-3f,
                                                -0x1.a6c0f2p-5f, 0x1.1251b8p-6f,  -0x1.920176p-9f};

// What all of a unit's warps derive from it.
template <int D>
struct Walk {
  static constexpr int kTiles = Shape<D>::kTiles;
  int head0, kv, from;
  int steps[kTiles], most;

  __device__ Walk(const TileParams& a, const Unit& u) {
    const Params& p = a.p;
    head0 = u.set * a.packed;
    kv = head0 / p.group;
    // the first key that a row of the unit sees, and each tile's steps from there
    from = p.window ? max(0, u.q0 - p.window + 1) : 0;
    most = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int begin = u.q0 + t * a.tokens;
      const int to = p.causal ? min(u.n, begin + a.tokens) : u.n;
      steps[t] = begin < u.n ? (to - from + kKeys - 1) / kKeys : 0;
      most = max(most, steps[t]);
    }
  }
};

template <int D, bool kHalf, bool kCapped>
__global__ void __launch_bounds__(Shape<D>::kThreads, Shape<D>::kCtas)
    tiles_kernel(const TileParams a, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map,
                 const __grid_constant__ CUtensorMap out_map) {
  using Sh = Shape<D>;
  constexpr int kTiles = Sh::kTiles, kStages = Sh::kStages, kParts = Sh::kParts;
  extern __shared__ uint8_t tiles_smem[];
  Shared<D>& s = *reinterpret_cast<Shared<D>*>(((uintptr_t)tiles_smem + 1023) & ~(uintptr_t)1023);
  const Params& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == Sh::kRowWarps) {
    if (lane == 0) {
      mbar_init(&s.fetch_done, 1);
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&s.unit_full[i], 1);
        mbar_init(&s.unit_empty[i], Sh::kRowWarps + kTiles + 1);
      }
      for (int i = 0; i < kStages; ++i) mbar_init(&s.full[i], 1), mbar_init(&s.empty[i], kTiles);
      for (int t = 0; t < kTiles; ++t) {
        mbar_init(&s.drained[t], 1);
        mbar_init(&s.q_full[t], 1);
        mbar_init(&s.q_empty[t], 1);
        mbar_init(&s.s_full[t], 1);
        mbar_init(&s.s_read[t], 4);
        mbar_init(&s.p_ready[t][0], 4);
        mbar_init(&s.p_ready[t][1], 4);
        mbar_init(&s.o_done[t], 1);
        mbar_init(&s.o_read[t], 4);
        mbar_init(&s.turn[t], 1);
      }
      s.given_up = s.beats = 0;
      mbar_fence_init();
    }
    __syncwarp();
  }
  if (warp == Sh::kRowWarps) tmem_allocate(&s.tmem, Sh::kColumns);
  Finder finder;
  if (warp == Sh::kRowWarps + 2) finder.begin(p, kTiles * a.tokens);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // Only now, with its tensor memory, does the CTA let the stream's next kernel be
  // scheduled: one that took some first and then waited for this one would stop it.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = s.tmem;

  const Patience patience{&s.given_up, &s.beats, a.status};
  // A wait of a whole warp.
  auto wait = [&](unsigned long long* bar, uint32_t parity) {
    return __all_sync(~0u, wait_for(bar, parity, patience)) != 0;
  };
  // The k-th unit.  All roles take all units, even when the CTA has given up.
  auto unit_at = [&](int k, Unit* u) {
    if (!__all_sync(~0u, outlast(&s.unit_full[k % kRing], (k / kRing) & 1, patience)))
      return false;
    *u = s.unit[k % kRing];
    return u->q0 >= 0;
  };
  auto unit_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.unit_empty[k % kRing]);
  };

  if (warp >= Sh::kRowWarps) {
    if constexpr (D != 256)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kOtherRegisters));
    if (warp == Sh::kRowWarps + 2) {
      // --------------------------------------------------------------- units
      // This CTA's, then those of CTAs that have not started.  No more are taken
      // than the SMs cannot begin at once; what the grid has beyond the last unit
      // is taken too and needs no CTA.
      uint32_t index = blockIdx.x;
      bool here = true, more = gridDim.x > (unsigned)(a.sms * Sh::kCtas);
      int fetches = 0;
#pragma unroll 1
      for (int k = 0;;) {
        // whether the CTA has given up or not: what was taken has to be handed on
        if (k >= kRing && !__all_sync(~0u, outlast(&s.unit_empty[k % kRing], (k / kRing - 1) & 1,
                                                   patience)))
          break;
        if (!here && more && !s.given_up) {
          uint32_t taken = 0, x = 0;
          if (lane == 0) {
            async_proxy_fence();
            mbar_expect_tx(&s.fetch_done, 16);
            asm volatile(
                "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes."
                "b128 [%0], [%1];" ::"r"(smem_u32(&s.fetched)),
                "r"(smem_u32(&s.fetch_done))
                : "memory");
          }
          __syncwarp();
          if (__all_sync(~0u, outlast(&s.fetch_done, fetches++ & 1, patience))) {
            asm volatile(
                "{\n .reg .pred p;\n .reg .b128 h;\n ld.shared.b128 h, [%2];\n"
                " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
                " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
                " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}"
                : "=r"(taken), "=r"(x)
                : "r"(smem_u32(&s.fetched))
                : "memory");
          }
          here = more = taken != 0;
          index = x;
        }
        Unit u{0, 0, -1, 0};
        if (here) {
          u = finder.find(p, kTiles * a.tokens, index / a.sets);
          u.set = index % a.sets;
          here = false;
          if (u.q0 < 0 && more) continue;
        }
        if (lane == 0) {
          s.unit[k % kRing] = u;
          mbar_arrive(&s.unit_full[k % kRing]);
        }
        __syncwarp();
        if (u.q0 < 0) break;
        ++k;
      }
    } else if (warp == Sh::kRowWarps + 1) {
      // -------------------------------------------------------------- copies
      int at = 0;  // stages filled
      int q_round[kTiles] = {};
      bool ok = true;
      Unit u;
      for (int k = 0; unit_at(k, &u); unit_done(k++)) {
        if (!ok || lane != 0) continue;
        const Walk<D> w(a, u);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (!w.steps[t]) continue;
          ok = ok && (q_round[t] == 0 || wait_for(&s.q_empty[t], (q_round[t] - 1) & 1, patience));
          if (!ok) break;
          ++q_round[t];
          mbar_expect_tx(&s.q_full[t], a.q_bytes);
          for (int c = 0; c < Sh::kChunks; ++c)
            tensor_load_3d(s.q[t] + c * kTileRows * 128, &q_map, c * 64, w.head0,
                           u.first + u.q0 + t * a.tokens, &s.q_full[t]);
        }
        // In the order of use: K0 V0 K1 V1 ..., or, with P beside S, K0 K1 V0 K2 V1
        // ...: a stage is filled again only when all before it in this order are
        // (heads of 256, four stages: 325 us in the first order, 210 in the second).
#pragma unroll 1
        for (int i = 0; ok && i < 2 * w.most; ++i) {
          const bool value = Sh::kBeside ? i == 2 * w.most - 1 || (i > 0 && i % 2 == 0) : i % 2;
          const int step = !Sh::kBeside || i == 0 ? i / 2 : value ? (i - 1) / 2 : (i + 1) / 2;
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            const int slot = at % kStages, round = at / kStages;
            ok = round == 0 || wait_for(&s.empty[slot], (round - 1) & 1, patience);
            if (!ok) break;
            ++at;
            mbar_expect_tx(&s.full[slot], Sh::kStageBytes);
#ifdef DCP_DEBUG_POISON
            if ((int)blockIdx.x == a.withheld_cta && k == a.withheld_unit && i == a.withheld_copy)
              continue;
#endif
            for (int c = 0; c < Sh::kPartChunks; ++c)
              tensor_load_3d(s.stage[slot] + c * kKeys * 128, value ? &v_map : &k_map,
                             (part * Sh::kPartChunks + c) * 64, w.kv,
                             u.first + w.from + step * kKeys, &s.full[slot]);
          }
        }
      }
      if (lane == 0 && s.given_up) {  // copies in flight, each for a limited time
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          if (q_round[t]) outlast(&s.q_full[t], (q_round[t] - 1) & 1, patience);
        for (int i = max(0, at - kStages); i < at; ++i)
          outlast(&s.full[i % kStages], (i / kStages) & 1, patience);
      }
      __syncwarp();
    } else if (warp == Sh::kRowWarps || (kTiles == 2 && warp == Sh::kRowWarps + 3)) {
      // ------------------------------------------------------------ products
      // A warp for each tile, so that one's waits pass while the other's products
      // run.  What a warp does between two products is time in which the tensor
      // cores may run dry, so all that it computes is the same in all lanes, and
      // written so that the compiler sees it: descriptors then stay in uniform
      // registers, from which the instruction takes them.  From others an
      // instruction took 87 cycles to issue, more than the 64 it takes to run.
      const int t = same_in_all(warp == Sh::kRowWarps ? 0 : 1);
      const bool leader = elect_one();
      // a negative scale: negated queries
      const uint32_t scores =
          mma_shape(!kHalf, kTileRows, kKeys, false) | (p.mult < 0.0f ? kNegateA : 0u);
      constexpr uint32_t kOuts = mma_shape(!kHalf, kTileRows, Sh::kPart, true);
      constexpr uint32_t kStageStep = Sh::kStageBytes / 16;  // in descriptors
      const uint32_t tm = same_in_all(tmem);
      const uint32_t s_at = tm + t * kKeys, p_at = tm + Sh::kP + t * Sh::kPStep;
      const uint32_t o_at = tm + Sh::kOut + t * D;
      const uint64_t q_rows = rows_along_k(same_in_all(smem_u32(s.q[t])));
      const uint64_t k_rows = rows_along_k(same_in_all(smem_u32(s.stage[0])));
      const uint64_t v_rows = rows_across_k(same_in_all(smem_u32(s.stage[0])), kKeys * 128);
      // the ring's next stages: kParts of them with their phase
      int slot = 0;
      uint32_t phase = 0;
      struct Stages {
        int slot[kParts];
        uint32_t phase[kParts];
      };
      auto take = [&] {
        Stages g;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          g.slot[i] = slot, g.phase[i] = phase;
          if (++slot == kStages) slot = 0, phase ^= 1;
        }
        return g;
      };
      auto part_arrived = [&](const Stages& g, int i) {
        return wait(&s.full[g.slot[i]], g.phase[i]);
      };
      auto free_part = [&](const Stages& g, int i) {
        if (leader) mma_commit(&s.empty[g.slot[i]]);
      };
      auto arrived = [&](const Stages& g) {
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kParts; ++i) ok = ok && part_arrived(g, i);
        return ok;
      };
      auto free = [&](const Stages& g) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) free_part(g, i);
      };
      // P over S: the tiles' products take turns, so that each tile's next S comes
      // soon (mixed they took 3700 cycles a step of both tiles).  A turn begins
      // with P's second half; the first half's product needs none.
      constexpr bool kTurns = !Sh::kBeside;
      uint32_t turns = 0;
      auto my_turn = [&] { return wait(&s.turn[t], (turns & 1) ^ (t == 0)); };
      auto next_turn = [&] {
        if (leader) mbar_arrive(&s.turn[kTiles - 1 - t]);
        ++turns;
      };
      // S from g, which it frees; `first`, `last`: of the unit
      auto multiply_scores = [&](const Stages& g, bool first, bool last) {
        bool ok = true;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (!kTurns || first) ok = ok && part_arrived(g, part);  // else seen before the turn
          if (!ok) return false;
          tmem_fence_after();
          const uint64_t rows = k_rows + g.slot[part] * kStageStep;
#pragma unroll
          for (int i = 0; i < Sh::kPart / 16; ++i) {
            if (leader)
              mma_smem(s_at,
                       q_rows + (part * Sh::kPartChunks + i / 4) * (kTileRows * 8) + i % 4 * 2,
                       rows + (i / 4 * kKeys * 128 + i % 4 * 32) / 16, scores, part > 0 || i > 0);
          }
          if (part + 1 < kParts) free_part(g, part);
        }
        if (leader) mma_commit(&s.s_full[t]);
        if (kTurns && !first) next_turn();
        free_part(g, kParts - 1);
        if (last && leader) mma_commit(&s.q_empty[t]);
        return true;
      };
      uint32_t q_round = 0, s_round = 0;  // units and steps of this tile
      bool ok = true;
      const int rows_end = same_in_all(start_of(p, p.num_seqs));
      Unit u;
      for (int k = 0; unit_at(k, &u); unit_done(k++)) {
        if (!ok) continue;
        u = Unit{same_in_all(u.first), same_in_all(u.n), same_in_all(u.q0), same_in_all(u.set)};
        const Walk<D> w(a, u);
        const int steps = t == 0 ? w.steps[0] : w.steps[kTiles - 1];
        // the first step's scores, then each step's next ones and its products
        // with the values; stages that only the other tile needs are passed on
        const Stages first_k = take();
        if (steps > 0) {
          ok = wait(&s.q_full[t], q_round & 1) &&
               (!Sh::kBeside || s_round == 0 || wait(&s.s_read[t], (s_round - 1) & 1)) &&
               multiply_scores(first_k, true, steps == 1);
        } else {
          ok = arrived(first_k);
          if (ok) free(first_k);
        }
        for (int j = 0; ok && j < w.most; ++j) {
          const bool next = j + 1 < w.most;
          Stages v_at, k_at{};
          if (Sh::kBeside && next) k_at = take();
          v_at = take();
          if (!Sh::kBeside && next) k_at = take();
          auto next_scores = [&] {
            if (j + 1 < steps) {
              if (Sh::kBeside) ok = wait(&s.s_read[t], s_round & 1);
              ok = ok && multiply_scores(k_at, false, j + 2 == steps);
            } else {
              ok = arrived(k_at);
              if (ok) free(k_at);
              if constexpr (kTurns) next_turn();
            }
          };
          if (Sh::kBeside && next) next_scores();
          ok = ok && arrived(v_at);
          if (!ok) break;
          if (j < steps) {
            // rows of this step behind the last sequence (none before it, unless
            // starts does not ascend)
            const int inside = max(0, rows_end - u.first - w.from - j * kKeys);
            if (inside < kKeys) {
              for (int c = 0; c < Sh::kChunks; ++c)
                for (int i = inside * 8 + lane; i < kKeys * 8; i += 32)
                  *reinterpret_cast<uint4*>(s.stage[v_at.slot[c / Sh::kPartChunks]] +
                                            c % Sh::kPartChunks * kKeys * 128 + i * 16) =
                      make_uint4(0, 0, 0, 0);
              async_proxy_fence();
              __syncwarp();
            }
            if (j == 0 && q_round > 0) ok = wait(&s.o_read[t], (q_round - 1) & 1);
            if constexpr (kTurns) ok = ok && (!next || arrived(k_at));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!Sh::kBeside || h == 0)
                ok = ok && wait(&s.p_ready[t][Sh::kBeside ? 1 : h], s_round & 1);
              if (kTurns && h == 1) ok = ok && my_turn();
              if (!ok) break;
              tmem_fence_after();
#pragma unroll
              for (int part = 0; part < kParts; ++part) {
                const uint64_t rows = v_rows + v_at.slot[part] * kStageStep;
#pragma unroll
                for (int i = h * kKeys / 32; i < (h + 1) * kKeys / 32; ++i)
                  if (leader)
                    mma_tmem(o_at + part * Sh::kPart, p_at + i * 8, rows + i * 2048 / 16, kOuts,
                             i > 0 || j > 0);
                if (kParts > 1 && h == 1) free_part(v_at, part);
              }
            }
            if (!ok) break;
            if ((Sh::kBeside || j + 1 == steps) && leader) mma_commit(&s.o_done[t]);
            ++s_round;
          } else if constexpr (kTurns) {
            ok = my_turn();
          }
          if (!ok) break;
          if (!Sh::kBeside && next) next_scores();
          if (kTurns && !next) next_turn();
          if (kParts == 1 || j >= steps) free(v_at);
        }
        q_round += steps > 0;
      }
      // products in flight, and the arrivals that they owe, for a limited time
      if (leader) mma_commit(&s.drained[t]);
      outlast(&s.drained[t], 0, patience);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ rows
    if constexpr (D != 256)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kRowRegisters));
    const int t = warp >> 2;
    const int row = 32 * (warp & 3) + lane;
    const int token = row / a.packed;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + t * kKeys;
    const uint32_t p_at = tmem + lanes + Sh::kP + t * Sh::kPStep;
    const uint32_t o_at = tmem + lanes + Sh::kOut + t * D;
    const float mult = fabsf(p.mult), late = kCapped ? 1.0f : mult;
    float terms[kTanhTerms];
#pragma unroll
    for (int i = 0; i < kTanhTerms; ++i) terms[i] = kTanh[i] * p.cap;
    // how far below the maximum a reference is set, how far above it the maximum
    // may go before it is set anew, and the sum of half a step's P up to which
    // none is too large
    constexpr float kBelow = kHalf ? 4.0f : 0.0f, kMost = kHalf ? 15.0f : 60.0f;
    constexpr float kLargest = kHalf ? 0x1p15f : 0x1p60f;
    // The exponent takes the exact product of score and mult, the reference is a
    // rounded one: P of the maximum itself is off by 2^(half a step of the
    // reference).  Up to here that is 2^(2^-4); from 2^30 on the only P may be 0.
    // Rows whose last reference lies beyond are computed again by attend_row, whose
    // products are all rounded.  (Multiplying such rows' scores before, beside
    // others in the same warp, cost heads of 64 5%.)
    constexpr float kFar = 0x1p20f;
    auto arrive = [&](unsigned long long* bar) {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int s_round = 0, o_round = 0;  // phases of s_full and o_done
    // When the CTA has given up the rest of the unit is computed on whatever there
    // is, and becomes NaN.  (Without a limit of their own, ending because those of
    // the other warps do, these waits took 2% less for 16384 rows of 64 heads of 128,
    // 4% less for 33 x 2048 of 12 of 64.)
    auto wait_here = [&](unsigned long long* bar, uint32_t parity) {
      wait_for(bar, parity, patience);
      __syncwarp();
      tmem_fence_after();
    };
    // the warp's first row, as a box of the output has it
    const int box_token = 32 * (warp & 3) / a.packed;
    const int box_head = 32 * (warp & 3) - box_token * a.packed;
    Unit u;
    for (int k = 0; unit_at(k, &u); unit_done(k++)) {
      const Walk<D> w(a, u);
      const int steps = t == 0 ? w.steps[0] : w.steps[kTiles - 1];
      if (steps == 0) continue;
      const int i = u.q0 + t * a.tokens + token, head = w.head0 + row - token * a.packed;
      const bool valid = token < a.tokens && i < u.n;
      // the keys that the row sees, counted from the first step's first
      const int lo = valid && p.window ? max(0, i - p.window + 1) - w.from : 0;
      const int hi = valid ? (p.causal ? i + 1 : u.n) - w.from : INT32_MAX;
      const int some_lo = __reduce_max_sync(~0u, lo), some_hi = __reduce_min_sync(~0u, hi);
      const int least_lo = __reduce_min_sync(~0u, valid ? lo : INT32_MAX);
      const int most_hi = __reduce_max_sync(~0u, valid ? hi : 0);
      float ref = -INFINITY, l = 0.0f, over = 0.0f;  // over: what l is too large by
      for (int j = 0; j < steps; ++j) {
        wait_here(&s.s_full[t], s_round++ & 1);
        uint32_t raw[kKeys];
        float* x = reinterpret_cast<float*>(raw);
        const int base = j * kKeys;
        const bool edge = base < some_lo || base + kKeys > some_hi;
        auto maximum = [&](int h) {
          float m[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) m[f] = fmaxf(x[64 * h + f], x[64 * h + f + 4]);
#pragma unroll
          for (int e = 64 * h + 8; e < 64 * h + 64; e += 8)
#pragma unroll
            for (int f = 0; f < 4; ++f) m[f] = max3(m[f], x[e + f], x[e + f + 4]);
          return fmaxf(max3(m[0], m[1], m[2]), m[3]) * late;
        };
        // P of a half, in place, and its sum
        auto exponentials = [&](int h) {
          const float less = ref == -INFINITY ? 0.0f : -ref;
          float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float2 y = fma2(make_float2(x[64 * h + e], x[64 * h + e + 1]), make_float2(late, late),
                            make_float2(less, less));
            y.x = kv4::exp2_approx(y.x);
            y.y = kv4::exp2_approx(y.y);
            sum[e / 2 & 1] = add2(sum[e / 2 & 1], y);
            raw[64 * h + e / 2] = round_pair<kHalf>(y.x, y.y);
          }
          const float2 both = add2(sum[0], sum[1]);
          return both.x + both.y;
        };
        // P beside S: the last product may still be reading it, and adding to O.
        // P over S: this step's S came after it.
        bool last_done = !Sh::kBeside || j == 0;
        auto wait_last = [&] {
          if (!last_done) wait_here(&s.o_done[t], o_round++ & 1);
          last_done = true;
        };
        // Most steps leave the reference where it is.  So the first half is
        // exponentiated with it before its maximum is known: its sum says whether
        // it was good, as does the second half's maximum, which is found beside the
        // exponentials.  What most steps do not do stands apart, so that they run
        // straight through their instructions.
        // Caps and masks: in tensor memory, in a loop.  (Unrolled over the registers
        // they were so much code that instructions came from the second-level
        // cache: with caps 1977 us instead of 577, without 419 instead of 317, for 33
        // prompts of 2048 rows with a window of 1000.  Caps by 32 scores: 466 us
        // there where all are within the cap, 657 where many are beyond; by 16
        // scores 516 and 704.)
        auto finish_scores = [&] {
          constexpr int kPiece = kCapped ? 32 : 16;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += kPiece) {
            const bool inside = base + c + kPiece <= some_hi && base + c >= some_lo;
            if (!kCapped && inside) continue;
            uint32_t piece[kPiece];
            float* y = reinterpret_cast<float*>(piece);
            auto put = [&] {
              if constexpr (kCapped) tmem_store32(s_at + c, piece);
              else tmem_store16(s_at + c, piece);
            };
            if (base + c >= most_hi || base + c + kPiece <= least_lo) {
#pragma unroll
              for (int e = 0; e < kPiece; ++e) y[e] = -INFINITY;
              put();
              continue;
            }
            if constexpr (kCapped) tmem_load32(s_at + c, piece);
            else tmem_load16(s_at + c, piece);
            const int from = lo - base - c, to = hi - base - c;  // what the row sees of them
            if constexpr (kCapped) {
              if (!inside) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e)
                  if (e < from || e >= to) y[e] = 0.0f;
              }
              float most[4] = {};
#pragma unroll
              for (int e = 0; e < kPiece; e += 8)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                  most[f] = max3(most[f], fabsf(y[e + 2 * f]), fabsf(y[e + 2 * f + 1]));
              const float top = fmaxf(max3(most[0], most[1], most[2]), most[3]);
              // Which formula a score takes is its own affair (they differ by their
              // errors); the warp decides only whether the second one is needed, and
              // lanes without a row, whose scores may be anything, have no say.
              const bool some_beyond = __any_sync(~0u, valid && !(top * mult <= 1.0f));
              auto cap = [&](auto beyond) {
#pragma unroll
                for (int e = 0; e < kPiece; e += 2) {
                  const float2 u = mul2(make_float2(y[e], y[e + 1]), make_float2(mult, mult));
                  const float2 square = mul2(u, u);
                  float2 r = make_float2(terms[kTanhTerms - 1], terms[kTanhTerms - 1]);
#pragma unroll
                  for (int i = kTanhTerms - 2; i >= 0; --i)
                    r = fma2(r, square, make_float2(terms[i], terms[i]));
                  r = mul2(r, u);
                  if constexpr (beyond.value) {
                    const float2 far = make_float2(p.cap * kv4::tanh_far(u.x), p.cap * kv4::tanh_far(u.y));
                    r.x = fabsf(u.x) > 1.0f ? far.x : r.x;
                    r.y = fabsf(u.y) > 1.0f ? far.y : r.y;
                  }
                  y[e] = r.x, y[e + 1] = r.y;
                }
              };
              if (some_beyond) cap(std::true_type{});
              else cap(std::false_type{});
            }
            if (!inside) {
#pragma unroll
              for (int e = 0; e < kPiece; ++e)
                if (e < from || e >= to) y[e] = -INFINITY;
            }
            put();
          }
          tmem_wait_store();
          tmem_load128(s_at, raw);
        };
        if (!kCapped && __builtin_expect(!edge, 1)) tmem_load128(s_at, raw);
        else finish_scores();
        float sum = 0.0f;
        bool good = false;
        if (__builtin_expect(j > 0, 1)) {
          sum = exponentials(0);
          // lanes without a row hold anything, NaN too: no reason for the slow way
          good = !valid || (sum <= kLargest && maximum(1) <= ref + kMost && ref > -INFINITY);
        }
        if (__builtin_expect(!__all_sync(~0u, good), 0)) {
          if (j > 0) {
            tmem_load64(s_at, raw);
          }
          const float top = fmaxf(maximum(0), maximum(1));
          float shrink = 1.0f;
          if (!good && top > ref + kBelow) {
            const float next = top - kBelow;
            shrink = exp2f(ref - next);  // 0 at first
            ref = next;
            // nothing is left of the sum, even if it was infinite (kFar)
            l = shrink > 0.0f ? l * shrink : 0.0f;
            over = shrink > 0.0f ? over * shrink : 0.0f;
          }
          if (j > 0) {
            wait_last();
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
          sum = exponentials(0);
        }
        if constexpr (Sh::kBeside) {
          // the rows, not the products, are what a step waits for: P at once
          arrive(&s.s_read[t]);
          sum += exponentials(1);
          wait_last();
          tmem_store32(p_at, raw);
          tmem_store32(p_at + 32, raw + 64);
        } else {
          tmem_store32(p_at, raw);
          tmem_wait_store();
          arrive(&s.p_ready[t][0]);
          sum += exponentials(1);
          tmem_store32(p_at + 32, raw + 64);
        }
        tmem_wait_store();
        arrive(&s.p_ready[t][1]);
        const float add = sum - over, now = l + add;
        over = (now - l) - add;
        l = now;
      }
      wait_here(&s.o_done[t], o_round++ & 1);
      const bool ok = !*(volatile int*)&s.given_up;
      const float inverse = ok ? (l == 0.0f ? 0.0f : 1.0f / l) : NAN;
      const int out_row = (u.first + i) * p.q_heads + head;  // rows * q_heads fit
      const unsigned written = __ballot_sync(~0u, valid);
      float2 zero[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // NaN once an O is not finite
      // 64 elements of the warp's rows at a time through shared memory: from there
      // by a tensor copy where the rows make a box and all are there, otherwise
      // eight lanes write a row's 128 bytes together.  (Each lane its own row, 16
      // bytes at a time, took 5000 cycles a unit; the copies are not waited for.)
      const bool box = a.out_box && written == ~0u;
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
        uint32_t o[64];
        tmem_load64(o_at + c, o);
        if (c + 64 == D) arrive(&s.o_read[t]);
        if (lane == 0) bulk_wait_read();  // what was copied from here before
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = make_float2(__uint_as_float(o[8 * b + 2 * e]),
                                         __uint_as_float(o[8 * b + 2 * e + 1]));
            zero[e & 1] = fma2(v, make_float2(0.0f, 0.0f), zero[e & 1]);
            y[e] = round_pair<kHalf>(v.x * inverse, v.y * inverse);
          }
          s.rows[warp][lane][b ^ (lane & 7)] = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (box) {
          async_proxy_fence();
          __syncwarp();
          if (lane == 0) {
            tensor_store_3d(&out_map, s.rows[warp], c, w.head0 + box_head,
                            u.first + u.q0 + t * a.tokens + box_token);
            bulk_commit();
          }
          continue;
        }
        __syncwarp();
#pragma unroll
        for (int r = lane >> 3; r < 32; r += 4) {
          const int to = __shfl_sync(~0u, out_row, r);
          if (written >> r & 1)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + ((int64_t)to * D + c) * 2 +
                                      (lane & 7) * 16) = s.rows[warp][r][(lane ^ r) & 7];
        }
        __syncwarp();
      }
      if (valid) p.lse[out_row] = !ok ? NAN : l == 0.0f ? -INFINITY : kLn2 * (ref + log2f(l));
      const float2 none = add2(zero[0], zero[1]);
      const bool finite = none.x + none.y == 0.0f;
      // a NaN among the scores that the row sees makes the sum NaN, and is right
      const unsigned bad = __ballot_sync(~0u, ok && valid && !finite && l == l);
      const unsigned far = __ballot_sync(
          ~0u, !kCapped && ok && valid && fabsf(ref) > kFar && fabsf(ref) < INFINITY);
      if (bad | far) {
        if (lane == 0) bulk_wait();  // such rows are read, and written once more
        __syncwarp();
        attend_again<D, kHalf>(p, u.first, u.n, p.window ? max(0, u.q0 - p.window + 1) : 0,
                               steps * kKeys, i, head, bad & ~far, far, &s.beats);
      }
    }
  }
  if (warp < Sh::kRowWarps && lane == 0) bulk_wait_read();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == Sh::kRowWarps) tmem_free(tmem, Sh::kColumns);
}

}  // namespace prompt
}  // namespace dcp
