// kv4.cu -- C ABI of the 4-bit key/value cache (include/dcp_kv4.h).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include <atomic>
#include <mutex>

#include "dcp_kv4.h"
#include "kv4_attention.cuh"
#include "kv4_evict.cuh"
#include "kv4_shares.cuh"
#include "kv4_slices.cuh"
#include "kv4_store.cuh"

namespace dcp {
namespace kv4 {

static bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

static bool power_of_two(float f) {
  uint32_t b;
  static_assert(sizeof b == sizeof f, "");
  __builtin_memcpy(&b, &f, sizeof b);
  return (b & 0x807FFFFFu) == 0u && b != 0u && b != 0x7F800000u;
}

// Checks a cache and fills the kernels' view of it.
static dcp_status planes_of(const dcp_kv4_cache* c, Planes* out) {
  if (!c || c->num_pages < 0 || c->page_size < 1 || c->heads < 1 || c->dim < 1 ||
      !power_of_two(c->k_unit) || !power_of_two(c->v_unit))
    return DCP_ERR_INVALID;
  if ((c->dim != 64 && c->dim != 128 && c->dim != 256) || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)) || c->heads > 65536)
    return DCP_ERR_UNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  if (c->num_pages >= (((int64_t)1 << 32) >> shift)) return DCP_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales))
    return DCP_ERR_INVALID;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16))
    return DCP_ERR_INVALID;
  out->k_codes = c->k_codes;
  out->v_codes = c->v_codes;
  out->k_scales = c->k_scales;
  out->v_scales = c->v_scales;
  out->num_pages = (uint32_t)c->num_pages;
  out->page_shift = shift;
  out->heads = c->heads;
  out->k_unit = c->k_unit;
  out->v_unit = c->v_unit;
  return DCP_OK;
}

static dcp_status status_of(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA; }

// -------------------------------------------------------------- attention
#ifdef DCP_DEBUG_POISON
static std::atomic<int> g_withheld[2] = {{-1}, {-1}};  // see dcp_kv4_selftest_withhold
#endif
static std::atomic<bool> g_ready[64];
static unsigned int* g_status[64];  // each device's status word, before g_ready
static std::mutex g_dev_mutex;

template <typename Kernel>
static cudaError_t allow_smem(Kernel* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, int NT>
static cudaError_t allow_attention() {
  constexpr int kSlice = SliceShape<D, NT, false>::kSmem;
  constexpr int kShare = ShareShape<D, NT>::kSmem;
  cudaError_t e;
  if ((e = allow_smem(attention_slices_kernel<D, NT, false, false>, kSlice)) != cudaSuccess ||
      (e = allow_smem(attention_slices_kernel<D, NT, true, false>, kSlice)) != cudaSuccess ||
      (e = allow_smem(attention_shares_kernel<D, NT, false, kByRing>, kShare)) != cudaSuccess ||
      (e = allow_smem(attention_shares_kernel<D, NT, true, kByRing>, kShare)) != cudaSuccess ||
      (e = allow_smem(attention_shares_kernel<D, NT, false, 8>, PageStage<D, 8>::kSmem)) !=
          cudaSuccess)
    return e;
  if constexpr (D > 64) {
    e = allow_smem(attention_shares_kernel<D, NT, false, 4>, PageStage<D, 4>::kSmem);
    if (e != cudaSuccess) return e;
  }
  if constexpr (D < 256) {
    e = allow_smem(attention_shares_kernel<D, NT, true, kByTeam>, kShare);
    if (e == cudaSuccess)
      e = allow_smem(attention_slices_kernel<D, NT, true, true>, SliceShape<D, NT, true>::kSmem);
  }
  if constexpr (D == 64)
    if (e == cudaSuccess) e = allow_smem(attention_shares_kernel<D, NT, false, kByTeam>, kShare);
  return e;
}

// Per-device kernel attributes, set once (the first call on a device must
// therefore not be inside a stream capture).
static cudaError_t prepare_device(unsigned int** status) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_ready[dev].load(std::memory_order_acquire)) {
    *status = g_status[dev];
    return cudaSuccess;
  }
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if ((e = allow_attention<64, 1>()) != cudaSuccess ||
      (e = allow_attention<64, 2>()) != cudaSuccess ||
      (e = allow_attention<128, 1>()) != cudaSuccess ||
      (e = allow_attention<128, 2>()) != cudaSuccess ||
      (e = allow_attention<256, 1>()) != cudaSuccess)
    return e;
  if ((e = device_status_word(&g_status[dev])) != cudaSuccess) return e;
  *status = g_status[dev];
  g_ready[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

// How a call is cut up (see kv4_slices.cuh, kv4_shares.cuh), and where its parts of the
// workspace lie.
struct Plan {
  int heads_per_cta, head_tiles, limit, width;
  int slices;  // CTAs of a row and head, or a row and team, when > 0
  int team;    // heads of a slice
  int shares;  // even shares, when > 0
  int together;  // key/value heads that a share walks at the same time
  int cuts;    // units, where a CTA joins one head of a unit (0: a warp does)
  size_t records, cut_at, part_out, part_ml, scores, row_mult, row_ml, bytes;
};

// The SM count that a call is cut up for: the workspace's size may not depend
// on a device being present.
constexpr int kPlanSms = 152;
// What even shares cost beyond their tiles, in tiles of a warp: finding the
// share's row, and the second launch.
constexpr int64_t kShareCost = 3;
// And what a piece costs: its queries, filling the ring, the join of its warps.
constexpr int64_t kPieceCost = 2;

static dcp_status plan_of(const dcp_kv4_cache* c, const Planes& planes,
                          const dcp_kv4_attention_args* a, Plan* plan) {
  if (!a || (a->dtype != DCP_F16 && a->dtype != DCP_BF16) || a->rows < 0 || a->q_heads < 1 ||
      a->q_heads % c->heads || a->num_seqs < 0 || a->table_width < 0 || a->max_len < 0 ||
      (a->ids && a->num_ids < 0) || (a->weights && a->owner) || !std::isfinite(a->scale) ||
      !std::isfinite(a->softcap) || a->softcap < 0.0f || a->weights_width < 0)
    return DCP_ERR_INVALID;
  const int64_t capacity = (int64_t)a->table_width << planes.page_shift;
  if (capacity > INT_MAX) return DCP_ERR_UNSUPPORTED;
  plan->limit = (int)(a->max_len && a->max_len < capacity ? a->max_len : capacity);
  plan->width = a->ids ? a->num_ids : plan->limit;
  const int group = a->q_heads / c->heads;
  plan->heads_per_cta = group > 8 && c->dim <= 128 ? 16 : 8;
  plan->head_tiles = (group + plan->heads_per_cta - 1) / plan->heads_per_cta;
  // Slices or shares, whichever has fewer tiles on its longest warp.  Lengths
  // are on the device: slices, as long as the longest row, are judged by that,
  // shares by three quarters of it where rows may differ.
  const int64_t units = (int64_t)a->rows * c->heads * plan->head_tiles;
  const int64_t tiles = ((int64_t)plan->width + kTile - 1) / kTile;
  // before anything is multiplied by more: units <= rows * query heads, so
  // units * tiles * dim then stays below 2^63
  if ((int64_t)a->rows * a->q_heads > INT_MAX || units * 8 > INT_MAX ||
      units * (tiles + kPieceTiles + 2) / kPlanSms > INT_MAX)
    return DCP_ERR_UNSUPPORTED;
  const int64_t warps = c->dim * plan->heads_per_cta >= 2048 ? 8 : 16;  // of an SM
  auto ceil_div = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  // Slices of ids in teams (kv4_team.cuh) where there are whole teams and an SM
  // gets 20 tiles of 128 elements or more, so that lines bound it and not
  // latency (2048 ids, 8 heads x 128, without and with teams: 4 rows 10.1 us
  // and 11.3, 8 rows 13.1 and 12.3, 16 rows 24.3 and 17.7, 64 rows 51 and 47;
  // 8 heads x 64, 8 rows: 9.7 and 11.1, 16 rows 13.6 and 12.0).
  const int members = c->dim < 256 ? 256 / c->dim : 1;
  const bool enough = units * tiles * c->dim >= (int64_t)20 * 128 * kPlanSms;
  plan->team = a->ids && enough && c->heads % members == 0 ? members : 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 8; s *= 2) {
    const int64_t steps =
        ceil_div(units / plan->team * s, kPlanSms * warps / kSliceWarps) *
        (ceil_div(ceil_div(tiles, s), kSliceWarps / plan->team) + kPieceCost);
    if (steps < least) least = steps, plan->slices = s;
  }
  // the largest power of two that leaves at most a fifth of the warps idle
  plan->together = kMostTogether;
  while (ceil_div(c->heads, plan->together) * plan->together * 4 > c->heads * 5)
    plan->together /= 2;
  const int64_t padded = units / c->heads * ceil_div(c->heads, plan->together) * plan->together;
  plan->shares = 0;
  const int64_t mean = a->ids || a->rows == 1 ? tiles : tiles * 3 / 4;
  if (ceil_div(padded * mean, kPlanSms * warps) + kPieceCost + kShareCost < least) {
    plan->slices = 0;
    plan->shares = (int)(kPlanSms * warps / kSliceWarps);  // as many CTAs of 8 warps as fit
  }
  // A unit is cut into about shares / (rows * units) pieces: from 16 on, two
  // for each warp of a CTA, a CTA joins one head, otherwise a warp does.
  const int64_t cuts = a->rows * ceil_div(c->heads, plan->together) * plan->head_tiles;
  plan->cuts = cuts * 16 <= plan->shares ? (int)cuts : 0;
  const size_t heads = (size_t)a->rows * a->q_heads;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 15) & ~(size_t)15;
    return here;
  };
  plan->records = plan->cut_at = plan->part_out = plan->part_ml = plan->scores = 0;
  plan->row_mult = plan->row_ml = 0;
  if (plan->shares) {
    const size_t pieces = (size_t)plan->shares * 2 * plan->together * plan->heads_per_cta;
    plan->records = take(plan->shares * sizeof(int4));
    plan->cut_at = take(plan->cuts * sizeof(int2));
    plan->part_out = take(pieces * c->dim * sizeof(float));
    plan->part_ml = take(pieces * sizeof(float2));
  }
  if (a->weights) {
    // the grid and the shared memory of the kernel that adds the weights up
    if (a->q_heads > kMostWeightHeads ||
        a->rows * (((int64_t)plan->width + kWeightTokens - 1) / kWeightTokens) > INT_MAX)
      return DCP_ERR_UNSUPPORTED;
    plan->scores = take(heads * plan->width * sizeof(float));
    plan->row_mult = take(heads * sizeof(float));
    plan->row_ml = take(heads * sizeof(float2));
  }
  plan->bytes = at;
  return DCP_OK;
}

template <int D, int NT>
static cudaError_t launch_attention(const AttentionParams& p, const Plan& plan,
                                    cudaStream_t stream) {
  if (plan.slices) {
    const unsigned grid =
        (unsigned)p.rows * p.head_tiles * (p.c.heads / plan.team) * plan.slices;
    if constexpr (D < 256)
      if (plan.team > 1)
        return launch(attention_slices_kernel<D, NT, true, true>, dim3(grid), kSliceThreads,
                      SliceShape<D, NT, true>::kSmem, plan.slices, stream, p);
    return launch(p.ids ? attention_slices_kernel<D, NT, true, false>
                        : attention_slices_kernel<D, NT, false, false>,
                  dim3(grid), kSliceThreads, SliceShape<D, NT, false>::kSmem, plan.slices, stream,
                  p);
  }
  using Shape = ShareShape<D, NT>;
  auto* kernel = p.ids ? attention_shares_kernel<D, NT, true, kByRing>
                       : attention_shares_kernel<D, NT, false, kByRing>;
  size_t smem = Shape::kSmem;
  // Teams of heads whose codes fill a line, where the heads walked together are
  // whole teams, for tokens by ids (1024 rows x 2048 ids, 8 heads x 128: 518 us
  // against 539) and at dim 64 (33 rows of 12 heads: 23 us against 25).  With
  // ranges at dim 128 their barriers cost more than the lines saved: 248 us
  // against 232 for 256 rows of up to 8192 tokens.  (Pairs measured with a plain
  // running sum of the probabilities; compensated, the first takes 529 us.)
  if constexpr (D < 256)
    if (p.ids && p.together % Shape::kTeam == 0)
      kernel = attention_shares_kernel<D, NT, true, kByTeam>;
  if constexpr (D == 64)
    if (!p.ids && p.together % Shape::kTeam == 0)
      kernel = attention_shares_kernel<D, NT, false, kByTeam>;
  // Ranges of caches whose runs of 8 tokens are 2 KB of codes or more, 8 heads
  // or 4 (256 rows as above, with a ring or teams and by runs: 8 heads x 64 161
  // us and 146, x 128 233 and 213, x 256 437 and 393; 4 heads x 128 129 and 125,
  // x 256 236 and 222; but, with a plain running sum, 4 heads x 64 84 and 85, 2
  // heads x 256 139 and 147).
  if (!p.ids && p.c.page_shift >= 3 && p.c.heads == 8) {
    kernel = attention_shares_kernel<D, NT, false, 8>;
    smem = PageStage<D, 8>::kSmem;
  }
  if constexpr (D > 64)
    if (!p.ids && p.c.page_shift >= 3 && p.c.heads == 4) {
      kernel = attention_shares_kernel<D, NT, false, 4>;
      smem = PageStage<D, 4>::kSmem;
    }
  const cudaError_t e = launch(kernel, dim3((unsigned)plan.shares), Shape::kThreads, smem, 1,
                               stream, p);
  if (e != cudaSuccess) return e;
  const int heads = p.together * 8 * NT;
  if (!plan.cuts)
    return launch(join_shares_kernel<D, NT, false>,
                  dim3((unsigned)plan.shares, (unsigned)(heads / kJoinWarps)), 32 * kJoinWarps, 0,
                  1, stream, p);
  // By unit, as many warps to a query head as the SMs hold at the same time (32
  // each): rows of 100003 and 131072 tokens 75, 68, 66, 64 us with 4, 8, 16, 32
  // warps, 16 rows of up to 16384 43, 45, 51, 62 (measured when the shares
  // before the join still walked by rings, 6 us longer).
  int warps = kMostJoinWarps;
  while (warps > kLeastJoinWarps && plan.cuts * heads * warps > kPlanSms * 32) warps /= 2;
  return launch(join_shares_kernel<D, NT, true>, dim3((unsigned)plan.cuts, (unsigned)heads),
                32 * warps, 0, 1, stream, p);
}

static cudaError_t launch_all(const AttentionParams& p, int dim, const Plan& plan,
                              cudaStream_t stream) {
  cudaError_t e;
  if (dim == 64)
    e = plan.heads_per_cta == 16 ? launch_attention<64, 2>(p, plan, stream)
                                 : launch_attention<64, 1>(p, plan, stream);
  else if (dim == 128)
    e = plan.heads_per_cta == 16 ? launch_attention<128, 2>(p, plan, stream)
                                 : launch_attention<128, 1>(p, plan, stream);
  else
    e = launch_attention<256, 1>(p, plan, stream);
  if (e != cudaSuccess || !p.weights || p.width == 0) return e;
  const int64_t tiles = ((int64_t)p.width + kWeightTokens - 1) / kWeightTokens;
  return launch(p.ids ? weights_kernel<true> : weights_kernel<false>,
                dim3((unsigned)(p.rows * tiles)), 256,
                (size_t)((p.q_heads + 3) & ~3) * 3 * sizeof(float), 1, stream, p);
}

}  // namespace kv4
}  // namespace dcp

using namespace dcp::kv4;

extern "C" {

static dcp_status store_args(const dcp_kv4_cache* cache, const void* k, const void* v, int dtype,
                             int64_t N, const int64_t* slots, StoreParams* p) {
  const dcp_status st = planes_of(cache, &p->c);
  if (st != DCP_OK) return st;
  if (dtype != DCP_F16 && dtype != DCP_BF16 && dtype != DCP_F32) return DCP_ERR_INVALID;
  if (N < 0) return DCP_ERR_INVALID;
  p->blocks = cache->dim / kBlock;
  p->N = N;
  p->dtype = dtype;
  p->slots = slots;
  if (N == 0) return DCP_OK;
  if (!k || !v || !slots) return DCP_ERR_INVALID;
  if (N > (int64_t)INT_MAX * 256 / ((int64_t)cache->heads * p->blocks)) return DCP_ERR_UNSUPPORTED;
  return DCP_OK;
}

static dim3 store_grid(const StoreParams& p) {
  return dim3((unsigned)((p.N * p.c.heads * p.blocks + 255) / 256));
}

dcp_status dcp_kv4_append(const dcp_kv4_cache* cache, const void* k, const void* v, int dtype,
                          int64_t N, int64_t k_row_stride, int64_t k_head_stride,
                          int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots,
                          dcp_stream_t stream) {
  StoreParams p{};
  const dcp_status st = store_args(cache, k, v, dtype, N, slots, &p);
  if (st != DCP_OK || N == 0) return st;
  p.in[0] = k, p.in[1] = v;
  p.row_stride[0] = k_row_stride, p.row_stride[1] = v_row_stride;
  p.head_stride[0] = k_head_stride, p.head_stride[1] = v_head_stride;
  const int64_t per = dtype == DCP_F32 ? 4 : 8;  // elements in 16 bytes
  for (int i = 0; i < 2; ++i)
    p.vec[i] = aligned(p.in[i], 16) && p.row_stride[i] % per == 0 && p.head_stride[i] % per == 0;
  return status_of(launch(append_kernel, store_grid(p), 256, 0, 1, (cudaStream_t)stream, p));
}

dcp_status dcp_kv4_read(const dcp_kv4_cache* cache, void* k, void* v, int dtype, int64_t N,
                        const int64_t* slots, dcp_stream_t stream) {
  StoreParams p{};
  const dcp_status st = store_args(cache, k, v, dtype, N, slots, &p);
  if (st != DCP_OK || N == 0) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return DCP_ERR_INVALID;
  p.out[0] = k, p.out[1] = v;
  return status_of(launch(read_kernel, store_grid(p), 256, 0, 1, (cudaStream_t)stream, p));
}

dcp_status dcp_kv4_attention_workspace_size(const dcp_kv4_cache* cache,
                                            const dcp_kv4_attention_args* args, size_t* bytes) {
  Planes planes;
  Plan plan;
  if (!bytes) return DCP_ERR_INVALID;
  dcp_status st = planes_of(cache, &planes);
  if (st == DCP_OK) st = plan_of(cache, planes, args, &plan);
  if (st == DCP_OK) *bytes = plan.bytes;
  return st;
}

dcp_status dcp_kv4_attention(const dcp_kv4_cache* cache, const dcp_kv4_attention_args* a,
                             dcp_stream_t stream) {
  AttentionParams p{};
  Plan plan;
  dcp_status st = planes_of(cache, &p.c);
  if (st == DCP_OK) st = plan_of(cache, p.c, a, &plan);
  if (st != DCP_OK || a->rows == 0) return st;
  if (!a->q || !a->lens || !a->out || !a->lse ||
      (!a->table && plan.limit > 0 && a->num_seqs > 0) ||
      (a->owner == nullptr && a->num_seqs < a->rows))
    return DCP_ERR_INVALID;
  if (!aligned(a->out, 16) || !aligned(a->workspace, 16)) return DCP_ERR_INVALID;
  if (plan.bytes > 0 && (!a->workspace || a->workspace_bytes < plan.bytes)) return DCP_ERR_INVALID;
  p.q = a->q;
  p.q_row_stride = a->q_row_stride;
  p.q_head_stride = a->q_head_stride;
  p.q_vec = aligned(a->q, 16) && a->q_row_stride % 8 == 0 && a->q_head_stride % 8 == 0;
  p.table = a->table;
  p.table_stride = a->table_stride;
  p.lens = a->lens;
  p.starts = a->starts;
  p.owner = a->owner;
  p.ids = a->ids;
  p.ids_stride = a->ids_stride;
  p.num_ids = a->num_ids;
  p.row_starts = a->row_starts;
  p.out = a->out;
  p.lse = a->lse;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  if (plan.shares) {
    p.shares = reinterpret_cast<int4*>(ws + plan.records);
    if (plan.cuts) p.cuts = reinterpret_cast<int2*>(ws + plan.cut_at);
    p.part_out = reinterpret_cast<float*>(ws + plan.part_out);
    p.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml);
  }
  if (a->weights) {
    p.scores = reinterpret_cast<float*>(ws + plan.scores);
    p.row_mult = reinterpret_cast<float*>(ws + plan.row_mult);
    p.row_ml = reinterpret_cast<float2*>(ws + plan.row_ml);
  }
  p.weights = a->weights;
  p.weights_stride = a->weights_stride;
  p.weights_width = a->weights_width;
  p.dtype = a->dtype;
  p.rows = a->rows;
  p.q_heads = a->q_heads;
  p.group = a->q_heads / cache->heads;
  p.head_tiles = plan.head_tiles;
  p.together = plan.together;
  p.num_seqs = a->num_seqs;
  p.limit = plan.limit;
  p.width = plan.width;
  p.score_pairs = a->q_heads % 2 == 0 && p.group % 2 == 0;
  p.scale = (a->scale != 0.0f ? a->scale : 1.0f / sqrtf((float)cache->dim)) * cache->k_unit;
  p.softcap = a->softcap;
#ifdef DCP_DEBUG_POISON
  p.withheld_share = g_withheld[0], p.withheld_tile = g_withheld[1];
#endif
  if (prepare_device(&p.status) != cudaSuccess) return DCP_ERR_CUDA;
  return status_of(launch_all(p, cache->dim, plan, (cudaStream_t)stream));
}

dcp_status dcp_kv4_evict(const dcp_kv4_cache* cache, const dcp_kv4_evict_args* a,
                         dcp_stream_t stream) {
  EvictParams p{};
  const dcp_status st = planes_of(cache, &p.c);
  if (st != DCP_OK) return st;
  if (!a || a->num_seqs < 0 || a->table_width < 0 || a->weights_width < 0 || a->budget < 1 ||
      a->sinks < 0 || a->recent < 0 || (int64_t)a->sinks + a->recent > a->budget)
    return DCP_ERR_INVALID;
  const int64_t capacity = (int64_t)a->table_width << p.c.page_shift;
  const int64_t limit = capacity < a->weights_width ? capacity : a->weights_width;
  if (capacity > INT_MAX || (int64_t)a->num_seqs * a->budget > (int64_t)INT_MAX * 8 ||
      a->num_seqs > INT_MAX / 8)
    return DCP_ERR_UNSUPPORTED;
  if (a->num_seqs == 0) return DCP_OK;
  if (!a->lens || !a->out_table || !a->kept || !a->out_lens || !a->out_weights ||
      (limit > 0 && (!a->table || !a->weights)))
    return DCP_ERR_INVALID;
  p.table = a->table;
  p.table_stride = a->table_stride;
  p.lens = a->lens;
  p.weights = a->weights;
  p.weights_stride = a->weights_stride;
  p.out_table = a->out_table;
  p.out_table_stride = a->out_table_stride;
  p.kept = a->kept;
  p.out_lens = a->out_lens;
  p.out_weights = a->out_weights;
  p.num_seqs = a->num_seqs;
  p.limit = (int)limit;
  p.budget = a->budget;
  p.sinks = a->sinks;
  p.recent = a->recent;
  p.row_codes = cache->heads * cache->dim / 2;
  p.row_scales = cache->heads * cache->dim / kBlock;
  // CTAs per sequence: a round of weights each, up to a portable cluster.  More
  // CTAs with fewer weights gain nothing, since each pass then pays the cluster's
  // barrier and remote loads (32 sequences of up to 16384 weights: four CTAs each
  // 20.4 us, one 19.8).
  int ctas = 1;
  while (ctas < kSelMostCtas && (int64_t)ctas * kSelRound < limit) ctas *= 2;
  cudaError_t e = launch(evict_select_kernel, dim3((unsigned)(a->num_seqs * ctas)), kSelThreads, 0,
                         ctas, (cudaStream_t)stream, p);
  if (e != cudaSuccess) return DCP_ERR_CUDA;
  const int64_t items = (int64_t)a->num_seqs * a->budget;
  e = launch(evict_copy_kernel, dim3((unsigned)((items + 8 * kCopy - 1) / (8 * kCopy))), 256, 0, 1,
             (cudaStream_t)stream, p);
  return status_of(e);
}

#ifdef DCP_DEBUG_POISON
// Race-check build: from now on attention by runs of a page (kv4_pages.cuh)
// does not bring in the given tile of the given share (-1: none), so that the
// waits for it run out, after a limit that is short in this build.
void dcp_kv4_selftest_withhold(int share, int tile) {
  g_withheld[0] = share, g_withheld[1] = tile;
}
#endif

}  // extern "C"
