// prompt.cu -- C ABI of attention over whole prompts (include/dcp_prompt.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include <atomic>
#include <mutex>

#include "dcp_prompt.h"
#include "prompt_tiles.cuh"

using namespace dcp;
using namespace dcp::prompt;

static dcp_status status_of(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA; }

// ------------------------------------------------------------------ devices
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static std::atomic<bool> g_ready[64];
static unsigned int* g_status[64];  // each device's status word, before g_ready
static int g_sms[64];               // and its SMs
static EncodeTiled g_encode;        // likewise
static std::mutex g_mutex;
#ifdef DCP_DEBUG_POISON
static std::atomic<int> g_withheld[3] = {{-1}, {-1}, {-1}};  // see dcp_prompt_selftest_withhold
#endif

template <int D, bool kHalf>
static cudaError_t allow_tiles() {
  constexpr int kBytes = sizeof(Shared<D>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(tiles_kernel<D, kHalf, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(tiles_kernel<D, kHalf, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  return e;
}

// Per-device kernel attributes, set once (the first call on a device must
// therefore not be inside a stream capture).
static cudaError_t prepare_device(TileParams* p) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!g_ready[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if ((e = allow_tiles<64, false>()) != cudaSuccess ||
        (e = allow_tiles<64, true>()) != cudaSuccess ||
        (e = allow_tiles<128, false>()) != cudaSuccess ||
        (e = allow_tiles<128, true>()) != cudaSuccess ||
        (e = allow_tiles<256, false>()) != cudaSuccess ||
        (e = allow_tiles<256, true>()) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev)) !=
            cudaSuccess ||
        (e = device_status_word(&g_status[dev])) != cudaSuccess)
      return e;
    if (!g_encode) {
      void* f = nullptr;
      cudaDriverEntryPointQueryResult found;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                           &found);
      if (e != cudaSuccess) return e;
      if (found != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
      g_encode = reinterpret_cast<EncodeTiled>(f);
    }
    g_ready[dev].store(true, std::memory_order_release);
  }
  p->status = g_status[dev];
  p->sms = g_sms[dev];
  return cudaSuccess;
}

// ------------------------------------------------------------- tensor copies
// Whether tensor copies can read heads laid out so: 16-byte steps, none of 0.
static bool fits(const void* x, int64_t rows, int64_t row_stride, int heads, int64_t head_stride) {
  const int64_t most = (int64_t)1 << 38;  // elements: 2^39 bytes
  return ((uintptr_t)x & 15) == 0 &&
         (rows == 1 || (row_stride > 0 && row_stride < most && row_stride % 8 == 0)) &&
         (heads == 1 || (head_stride > 0 && head_stride < most && head_stride % 8 == 0));
}

// Whether rows x heads laid out so, `bytes` each, share memory with [begin, end).
static bool overlaps(const void* x, int64_t rows, int64_t row_stride, int heads,
                     int64_t head_stride, int64_t bytes, const void* begin, const void* end) {
  row_stride *= 2, head_stride *= 2;  // bytes
  const int64_t whole = (rows > 1 ? (rows - 1) * row_stride : 0) +
                        (heads > 1 ? (heads - 1) * head_stride : 0) + bytes;
  if (static_cast<const char*>(x) + whole <= begin || x >= end) return false;  // as a rule
  for (int h = 0; h < heads; ++h) {
    const char* at = static_cast<const char*>(x) + h * head_stride;
    // the first row that ends behind `begin`
    const int64_t before = static_cast<const char*>(begin) - at - bytes;
    const int64_t row = before < 0 ? 0 : rows == 1 ? 1 : before / row_stride + 1;
    if (row < rows && at + row * row_stride < static_cast<const char*>(end)) return true;
  }
  return false;
}

// Whether the outputs share memory with each other or with an input.
static bool outputs_overlap(const dcp_prompt_attention_args* a) {
  const int64_t bytes = 2 * a->dim, n = a->rows * a->q_heads;
  const char* begin[2] = {static_cast<const char*>(a->out), reinterpret_cast<const char*>(a->lse)};
  const char* end[2] = {begin[0] + n * bytes, begin[1] + n * 4};
  const char* starts = reinterpret_cast<const char*>(a->starts);
  for (int i = 0; i < 2; ++i)
    if (overlaps(a->q, a->rows, a->q_row_stride, a->q_heads, a->q_head_stride, bytes, begin[i],
                 end[i]) ||
        overlaps(a->k, a->rows, a->k_row_stride, a->kv_heads, a->k_head_stride, bytes, begin[i],
                 end[i]) ||
        overlaps(a->v, a->rows, a->v_row_stride, a->kv_heads, a->v_head_stride, bytes, begin[i],
                 end[i]) ||
        (starts < end[i] && begin[i] < starts + 4 * ((int64_t)a->num_seqs + 1)))
      return true;
  return begin[0] < end[1] && begin[1] < end[0];
}

// Boxes of `tokens` rows of `packed` heads, 64 elements each.
static bool map_of(CUtensorMap* map, const void* x, int dtype, int64_t rows, int64_t row_stride,
                   int heads, int64_t head_stride, int dim, int packed, int tokens) {
  const cuuint64_t sizes[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  // a dimension of one element may have any stride
  const cuuint64_t strides[2] = {(cuuint64_t)(heads == 1 ? dim : head_stride) * 2,
                                 (cuuint64_t)(rows == 1 ? dim : row_stride) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)packed, (cuuint32_t)tokens};
  const cuuint32_t steps[3] = {1, 1, 1};
  return g_encode(map, dtype == DCP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  3, const_cast<void*>(x), sizes, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static dcp_status launch_tiles(const dcp_prompt_attention_args* a, TileParams p,
                               cudaStream_t stream) {
  using S = Shape<D>;
  const int group = p.p.group;
  p.packed = group < kTileRows ? group : kTileRows;
  while (group % p.packed) --p.packed;
  p.tokens = kTileRows / p.packed;
  p.sets = a->q_heads / p.packed;
  p.q_bytes = S::kChunks * p.packed * p.tokens * 128;
  // 32 rows of a tile: whole tokens of its heads, or heads of one token
  p.out_box = 32 % p.packed == 0 || p.packed % 32 == 0;
  const int out_heads = p.packed < 32 ? p.packed : 32;
  CUtensorMap q, k, v, out;
  if (!map_of(&q, a->q, a->dtype, a->rows, a->q_row_stride, a->q_heads, a->q_head_stride, D,
              p.packed, p.tokens) ||
      !map_of(&k, a->k, a->dtype, a->rows, a->k_row_stride, a->kv_heads, a->k_head_stride, D, 1,
              kKeys) ||
      !map_of(&v, a->v, a->dtype, a->rows, a->v_row_stride, a->kv_heads, a->v_head_stride, D, 1,
              kKeys) ||
      !map_of(&out, a->out, a->dtype, a->rows, (int64_t)a->q_heads * D, a->q_heads, D, D,
              p.out_box ? out_heads : 1, p.out_box ? 32 / out_heads : 1))
    return DCP_ERR_CUDA;
  // as many units as there can be, whatever the lengths
  const int64_t by_span = a->rows / (S::kTiles * p.tokens) + a->num_seqs;
  const int64_t units = by_span < a->rows ? by_span : a->rows;
  const bool half = a->dtype == DCP_F16;
  auto* kernel = half ? (p.p.capped ? tiles_kernel<D, true, true> : tiles_kernel<D, true, false>)
                      : (p.p.capped ? tiles_kernel<D, false, true> : tiles_kernel<D, false, false>);
  return status_of(kv4::launch(kernel, dim3((unsigned)(units * p.sets)), S::kThreads,
                               sizeof(Shared<D>) + 1024, 1, stream, p, q, k, v, out));
}

extern "C" dcp_status dcp_prompt_attention(const dcp_prompt_attention_args* a,
                                           dcp_stream_t stream) {
  if (!a || (a->dtype != DCP_F16 && a->dtype != DCP_BF16) || a->rows < 0 || a->num_seqs < 0 ||
      a->q_heads < 1 || a->kv_heads < 1 || a->q_heads % a->kv_heads || a->window < 0 ||
      !std::isfinite(a->scale) || !std::isfinite(a->softcap) || a->softcap < 0.0f)
    return DCP_ERR_INVALID;
  if ((a->dim != 64 && a->dim != 128 && a->dim != 256) || a->rows > INT_MAX / a->q_heads ||
      a->q_heads > 65536)
    return DCP_ERR_UNSUPPORTED;
  if (a->rows == 0 || a->num_seqs == 0) return DCP_OK;
  if (!a->q || !a->k || !a->v || !a->starts || !a->out || !a->lse || ((uintptr_t)a->out & 15))
    return DCP_ERR_INVALID;
  if (!fits(a->q, a->rows, a->q_row_stride, a->q_heads, a->q_head_stride) ||
      !fits(a->k, a->rows, a->k_row_stride, a->kv_heads, a->k_head_stride) ||
      !fits(a->v, a->rows, a->v_row_stride, a->kv_heads, a->v_head_stride))
    return DCP_ERR_UNSUPPORTED;
  if (outputs_overlap(a)) return DCP_ERR_INVALID;
  TileParams t{};
  Params& p = t.p;
  p.q = a->q, p.k = a->k, p.v = a->v;
  p.q_row_stride = a->q_row_stride, p.q_head_stride = a->q_head_stride;
  p.k_row_stride = a->k_row_stride, p.k_head_stride = a->k_head_stride;
  p.v_row_stride = a->v_row_stride, p.v_head_stride = a->v_head_stride;
  p.starts = a->starts;
  p.out = a->out;
  p.lse = a->lse;
  p.rows = (int)a->rows;
  p.num_seqs = a->num_seqs;
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.group = a->q_heads / a->kv_heads;
  p.dtype = a->dtype;
  p.causal = a->causal != 0;
  p.window = a->window;
  const float scale = a->scale != 0.0f ? a->scale : 1.0f / sqrtf((float)a->dim);
  // A cap that the scores' factor or its own cannot be written beside is so far
  // away that tanh changes nothing: none.
  const float ratio = fabsf(scale) / a->softcap;
  p.capped = a->softcap > 0.0f && ratio >= FLT_MIN && std::isfinite(a->softcap * kLog2e);
  p.cap = a->softcap * kLog2e;
  // finite, and above 0: 0 times it stays 0, an infinity one
  p.mult = copysignf(fminf(fmaxf(p.capped ? ratio : fabsf(scale) * kLog2e, FLT_MIN), FLT_MAX),
                     scale);
#ifdef DCP_DEBUG_POISON
  t.withheld_cta = g_withheld[0], t.withheld_unit = g_withheld[1], t.withheld_copy = g_withheld[2];
#endif
  if (prepare_device(&t) != cudaSuccess) return DCP_ERR_CUDA;
  const cudaStream_t st = (cudaStream_t)stream;
  return a->dim == 64    ? launch_tiles<64>(a, t, st)
         : a->dim == 128 ? launch_tiles<128>(a, t, st)
                         : launch_tiles<256>(a, t, st);
}

#ifdef DCP_DEBUG_POISON
// Race-check build: from now on the given CTA does not bring in the given copy (K
// or V of a step, in the order of use) of its given unit (-1: none), so that the
// waits for it run out, after a limit that is short in this build.
extern "C" void dcp_prompt_selftest_withhold(int cta, int unit, int copy) {
  g_withheld[0] = cta, g_withheld[1] = unit, g_withheld[2] = copy;
}
#endif
