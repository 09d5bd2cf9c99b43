// kv4_pages.cuh -- how the warps of all key/value heads bring the tiles of a
// range in together: runs of 8 tokens, whose rows of all heads are one piece of
// a page, by bulk copies.
//
// Copied by the warps themselves, a tile at dim 128 takes L1 about 290 cycles
// (see kv4_team.cuh), more than the 226 that its arithmetic takes an SM; the
// bulk copies go past that: 16 of them, 37 KB, bring the tiles of 8 warps.  256
// rows of 64 to 8192 tokens, 8 heads x 128: 213 us against 233; the copies alone
// take 190, the arithmetic alone took 187 with a plain running sum (210 us in all).
//
// What the barriers cost depends on who has to wait: the warp that fills a stage
// at once when it has read it itself waits for the slowest of the group (253
// us); one that does so a tile later seldom does, with one barrier for K and V
// 214, with one each 208.  A tile and a half later the copies come too late
// (230), and filling by whichever warp reads a stage last puts the work on the
// slowest (285).
#pragma once

#include "bulk_copy.cuh"
#include "kv4_team.cuh"

namespace dcp {
namespace kv4 {

// A stage of a group of kHeads warps: 32 tokens as four runs of 8, each as it
// lies in its page.  The runs lie 32 bytes (scales 16) further apart than they
// are long, and a tile's rows are dealt to the tokens so that the lanes that
// are served at a time read from different runs: they touch all banks.
template <int D, int kHeads>
struct PageStage {
  static constexpr int kStages = 3;
  static constexpr int kRun = 8, kRuns = kTile / kRun;
  static constexpr int kCodeRow = kHeads * (D / 2), kScaleRow = kHeads * (D / 16);  // of a token
  static constexpr int kCodeRun = kRun * kCodeRow + 32, kScaleRun = kRun * kScaleRow + 16;
  static constexpr int kScales = kRuns * kCodeRun;             // K, and likewise V:
  static constexpr int kHalf = kScales + kRuns * kScaleRun;    // codes, scales
  static constexpr int kBytes = 2 * kHalf;
  static constexpr int kGroups = 8 / kHeads;  // of a CTA
  // their stages, then K's and V's barriers, the masks, and whether a wait ran out
  static constexpr int kRings = kGroups * kStages * kBytes;
  static constexpr int kGaveUp = kRings + kGroups * kStages * (4 * 8 + 4);
  static constexpr int kSmem = kGaveUp + 4;
};

// A group's part of that.
template <int D, int kHeads>
struct PageRing {
  using S = PageStage<D, kHeads>;
  uint8_t* stages;
  unsigned long long* bars;  // [K landed, V landed, K read, V read][kStages]
  uint32_t* masks;           // of present tokens
  __device__ PageRing(int sub, uint8_t* smem) {
    stages = smem + sub * S::kStages * S::kBytes;
    bars = reinterpret_cast<unsigned long long*>(smem + S::kRings) + sub * 4 * S::kStages;
    masks = reinterpret_cast<uint32_t*>(smem + S::kRings + S::kGroups * S::kStages * 32) +
            sub * S::kStages;
  }
  __device__ unsigned long long* landed(int v, uint32_t stage) const {
    return bars + v * S::kStages + stage;
  }
  __device__ unsigned long long* read(int v, uint32_t stage) const {
    return bars + (2 + v) * S::kStages + stage;
  }
};

// A thread's operands in a stage (see attend_tile).  The accumulator's row i
// stands for token i % 2 + 2 (i / 8) + 4u of run (i / 2) % 4 ^ 2 (i % 2).
template <int D, int kHeads, typename KRead, typename VWait>
struct PageAt {
  using S = PageStage<D, kHeads>;
  static constexpr int kSubStep = 4, kHalfStep = 2;
  static constexpr bool kRaw = true;
  const uint8_t *k0, *v0, *v1, *ks0, *vs0, *vs1;
  int tq;
  const KRead& k_read;
  const VWait& v_wait;

  static __device__ __forceinline__ constexpr int run(int i) {
    return ((i >> 1) & 3) ^ ((i & 1) << 1);
  }
  static __device__ __forceinline__ constexpr int token(int i) { return 8 * run(i) + (i & 1); }
  // of the V rows' tokens: i as in v()
  __device__ int v_token(int u, int i) const {
    return token(2 * tq + (i & 1)) + 2 * (i >> 1) + 4 * u;
  }
  __device__ PageAt(const uint8_t* stage, int head, int g, int tq_, const KRead& k_read_,
                    const VWait& v_wait_)
      : tq(tq_), k_read(k_read_), v_wait(v_wait_) {
    const uint8_t* codes = stage + head * (D / 2);
    const uint8_t* scales = stage + S::kScales + head * (D / 16);
    k0 = codes + run(g) * S::kCodeRun + (g & 1) * S::kCodeRow + tq * (D == 64 ? 8 : 16);
    ks0 = scales + run(g) * S::kScaleRun + (g & 1) * S::kScaleRow + (D == 64 ? tq : 2 * tq);
    v0 = codes + S::kHalf + tq * S::kCodeRun + g * (D / 16);
    v1 = codes + S::kHalf + (tq ^ 2) * S::kCodeRun + S::kCodeRow + g * (D / 16);
    scales += S::kHalf + (D == 256 ? 2 * g : D == 128 ? g : g >> 1);
    vs0 = scales + tq * S::kScaleRun;
    vs1 = scales + (tq ^ 2) * S::kScaleRun + S::kScaleRow;
  }
  __device__ const uint8_t* k(int u, int i) const { return k0 + (2 * u + i) * 2 * S::kCodeRow; }
  __device__ const uint8_t* k_second(int u, int i) const { return k(u, i) + 64; }
  __device__ const uint8_t* k_scale(int u, int i) const {
    return ks0 + (2 * u + i) * 2 * S::kScaleRow;
  }
  __device__ const uint8_t* v(int u, int i) const {
    return (i & 1 ? v1 : v0) + (2 * u + (i >> 1)) * 2 * S::kCodeRow;
  }
  __device__ const uint8_t* v_scale(int u, int i) const {
    return (i & 1 ? vs1 : vs0) + (2 * u + (i >> 1)) * 2 * S::kScaleRow;
  }
};

// Cycles that a copy is waited for.  When they have passed, the CTA gives up:
// its warps bring nothing in any more, wait for nothing any more, and write NaN
// for what they have not finished; before it ends it lets the same time pass
// once more, for copies that are still on their way into its shared memory.
#ifdef DCP_DEBUG_POISON
constexpr unsigned long long kPageWaitLimit = 1ull << 22;  // about 2 ms
#else
constexpr unsigned long long kPageWaitLimit = 1ull << 31;  // about 1 s
#endif

template <int D, int kHeads>
__device__ __forceinline__ volatile uint32_t* gave_up(uint8_t* smem) {
  return reinterpret_cast<volatile uint32_t*>(smem + PageStage<D, kHeads>::kGaveUp);
}

// Waits for phase `parity` of `bar`, the whole warp, with one answer: false if
// the CTA has given up.
__device__ __forceinline__ bool page_wait(unsigned long long* bar, uint32_t parity,
                                          volatile uint32_t* over, unsigned int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const bool late = clock64() - t0 >= kPageWaitLimit;
    if (late) {
      atomicOr(status, kStatusCopyTimeout);
      *over = 1u;
    }
    if (__any_sync(0xffffffffu, late || *over)) return false;
  }
}

// A barrier of the CTA has to follow.
template <int D, int kHeads>
__device__ __forceinline__ void begin_pages(uint8_t* smem) {
  using S = PageStage<D, kHeads>;
  constexpr int kBars = 4 * S::kStages;  // of a group
  if (threadIdx.x == 0) *gave_up<D, kHeads>(smem) = 0u;
  if (threadIdx.x < S::kGroups * kBars)
    mbar_init(PageRing<D, kHeads>(0, smem).bars + threadIdx.x,
              threadIdx.x % kBars < 2 * S::kStages ? 1 : kHeads);
  mbar_fence_init();
}

// The CTA's end.
template <int D, int kHeads>
__device__ __forceinline__ void end_pages(uint8_t* smem) {
  if (!*gave_up<D, kHeads>(smem)) return;
  const unsigned long long t0 = clock64();
  while (clock64() - t0 < kPageWaitLimit) {
  }
}

// attend_tiles for one of the kHeads warps of a group, this one's head being
// `head`.  The group's tiles are numbered over all its calls, `walked` of them
// so far; warp n % kHeads brings tile n in.  It does so when it has read tile
// n - 2 itself, so that the others have had a tile's time to read tile n - 3,
// whose stage n takes.
template <int D, int NT, int kHeads>
__device__ __forceinline__ void attend_pages(const AttentionParams& p, const RowSpan& r, int t,
                                             int head, int head0, int q_heads, int tile0,
                                             int tile1, int sub, uint8_t* smem, uint32_t& walked,
                                             Heads<D, NT>& hd) {
  using S = PageStage<D, kHeads>;
  constexpr int kOf = S::kGroups;
  const PageRing<D, kHeads> ring(sub, smem);
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  volatile uint32_t* const over = gave_up<D, kHeads>(smem);
  const int mine = tile1 - tile0 > sub && !__any_sync(0xffffffffu, *over)
                       ? (int)((unsigned)(tile1 - tile0 - sub + kOf - 1) / (unsigned)kOf)
                       : 0;
  hd.fetch(p, t, head0, q_heads);
  const int32_t* table = p.table + (int64_t)r.seq * p.table_stride;

  const uint32_t done = walked;
  auto wait = [&](unsigned long long* bar, uint32_t parity) {
    return page_wait(bar, parity, over, p.status);
  };
  // a run's first position (r.start is a multiple of 8) and page
  const int run = lane & 3;
  auto place = [&](int k) {
    return (uint32_t)r.start + (uint32_t)kTile * (uint32_t)(tile0 + sub + kOf * k) + S::kRun * run;
  };
  const uint32_t end = (uint32_t)max(r.end, 0);
  auto look = [&](int k) {
    const uint32_t pos = place(k);
    return k < mine && pos < end ? __ldg(table + (pos >> p.c.page_shift)) : -1;
  };
  int next = (int)((uint32_t)(head - (int)done) % (uint32_t)kHeads);  // this warp's next tile
  int page = look(next);
  // K (v = 0) or V (1) of tile `next`: lanes 0 to 3 copy a run's codes, 4 to 7 its
  // scales.  False if the CTA has given up.
  auto issue = [&](int v) {
    const uint32_t n = done + (uint32_t)next, stage = n % S::kStages;
    if (n >= S::kStages && !wait(ring.read(v, stage), (n / S::kStages - 1) & 1)) return false;
#ifdef DCP_DEBUG_POISON
    if ((int)blockIdx.x == p.withheld_share && (int)n == p.withheld_tile) return false;
#endif
    const uint32_t pos = place(next);
    // the runs that are in the cache, as lanes 0 to 3 see it
    const uint32_t runs = __ballot_sync(0xffffffffu, (uint32_t)page < p.c.num_pages) & 0xFu;
    const bool ok = (runs >> run) & 1u;
    if (v == 0 && lane < S::kRuns) {
      const int lo = max(0, r.start + r.skip - (int)pos), hi = min(8, r.end - (int)pos);
      reinterpret_cast<uint8_t*>(ring.masks + stage)[run] =
          ok ? (uint8_t)((0xFFu << lo) & (0xFFu >> (8 - hi))) : (uint8_t)0;
    }
    // lane 0's arrival publishes the others' bytes too; it completes the phase
    // at once where no run is in the cache
    __syncwarp();
    if (lane == 0)
      mbar_expect_tx(ring.landed(v, stage),
                     (uint32_t)(__popc(runs) * S::kRun * (S::kCodeRow + S::kScaleRow)));
    __syncwarp();
    if (lane < 2 * S::kRuns && ok) {
      const int64_t slot =
          ((int64_t)page << p.c.page_shift) | (pos & ((1u << p.c.page_shift) - 1u));
      uint8_t* to = ring.stages + stage * S::kBytes + v * S::kHalf;
      if (lane < S::kRuns)
        tma_load_1d(to + run * S::kCodeRun, (v ? p.c.v_codes : p.c.k_codes) + slot * S::kCodeRow,
                    S::kRun * S::kCodeRow, ring.landed(v, stage));
      else
        tma_load_1d(to + S::kScales + run * S::kScaleRun,
                    (v ? p.c.v_scales : p.c.k_scales) + slot * S::kScaleRow,
                    S::kRun * S::kScaleRow, ring.landed(v, stage));
    }
    if (v == 1) {
      next += kHeads;
      page = look(next);
    }
    return true;
  };
  auto bring = [&] {
    if (issue(0)) issue(1);
  };

#pragma unroll 1
  for (int k = 0; k < S::kStages - 1; ++k)
    if (k == next && k < mine) bring();
  hd.begin(p, t, head0, q_heads, tile0 == 0 && sub == 0);

  uint32_t stage = done % S::kStages, parity = done / S::kStages & 1;
#pragma unroll 1
  for (int k = 0; k < mine; ++k) {
    if (!wait(ring.landed(0, stage), parity)) break;
    const uint32_t mask = ring.masks[stage];
    auto k_read = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.read(0, stage));
    };
    auto v_wait = [&] { wait(ring.landed(1, stage), parity); };
    attend_tile<D, NT>(p, r, t, head0, q_heads,
                       PageAt<D, kHeads, decltype(k_read), decltype(v_wait)>(
                           ring.stages + stage * S::kBytes, head, g, tq, k_read, v_wait),
                       mask, (int64_t)kTile * (tile0 + sub + (int64_t)kOf * k), hd);
    __syncwarp();
    if (lane == 0) mbar_arrive(ring.read(1, stage));
    if (k + S::kStages - 1 == next && next < mine) bring();
    if (++stage == S::kStages) stage = 0, parity ^= 1;
  }
  walked += mine;
  hd.end();
}

}  // namespace kv4
}  // namespace dcp
