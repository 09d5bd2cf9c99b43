// batch.cu -- C ABI of a batch's bookkeeping (dcp_kv4_extend) and of rotary
// positions (dcp_rotary).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include <atomic>
#include <mutex>

#include "dcp_kv4.h"
#include "dcp_prompt.h"
#include "kv4_extend.cuh"
#include "rotary.cuh"

namespace dcp {
namespace {

dcp_status status_of(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA; }

// extend_kernel's shared memory beyond the default, once per device.
cudaError_t allow_extend() {
  static std::atomic<bool> ready[64];
  static std::mutex mutex;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mutex);
  e = cudaFuncSetAttribute(kv4::extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kv4::kMostExtendSeqs * kv4::kExtendRow);
  if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
  return e;
}

// The current device's SMs, asked for once.
cudaError_t count_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if ((*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

// Whether n numbers at a and m at b share memory.
bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  return n > 0 && m > 0 && (uintptr_t)a < (uintptr_t)(b + m) && (uintptr_t)b < (uintptr_t)(a + n);
}

// Whether 16-byte pieces fit a plane of heads: its address and its strides.
bool fits(const void* p, int64_t row, int64_t head, int64_t per) {
  return ((uintptr_t)p & 15) == 0 && row % per == 0 && head % per == 0;
}

template <typename T, int V>
cudaError_t launch_rotary(const RotaryParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  return kv4::launch(interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, grid,
                     kRotaryThreads, (size_t)p.tokens_per_cta * p.pairs * sizeof(float2), 1,
                     stream, p);
}

}  // namespace
}  // namespace dcp

using namespace dcp;

extern "C" {

dcp_status dcp_kv4_extend(const dcp_kv4_extend_args* a, dcp_stream_t stream) {
  if (!a || a->num_pages < 0 || a->page_size < 1 || a->num_seqs < 0 || a->table_width < 0 ||
      a->num_free < 0 || a->places < 0)
    return DCP_ERR_INVALID;
  if (a->page_size > 65536 || (a->page_size & (a->page_size - 1)) ||
      a->num_seqs > kv4::kMostExtendSeqs)
    return DCP_ERR_UNSUPPORTED;
  kv4::ExtendParams p{};
  while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
  if (a->num_pages >= (((int64_t)1 << 32) >> p.page_shift) ||
      ((int64_t)a->table_width << p.page_shift) > INT_MAX)
    return DCP_ERR_UNSUPPORTED;
  if (!a->used || !a->starts || !a->out_used ||
      (a->num_seqs > 0 && (!a->lens || !a->counts || !a->out_lens ||
                           (a->table_width > 0 && !a->table))) ||
      (a->num_free > 0 && !a->free_pages) ||
      (a->places > 0 && (!a->slots || !a->positions || !a->owner || !a->row_lens)))
    return DCP_ERR_INVALID;
  p.table = a->table;
  p.table_stride = a->table_stride;
  p.lens = a->lens;
  p.counts = a->counts;
  p.free_pages = a->free_pages;
  p.used = a->used;
  p.slots = a->slots;
  p.positions = a->positions;
  p.owner = a->owner;
  p.row_lens = a->row_lens;
  p.starts = a->starts;
  p.out_lens = a->out_lens;
  p.out_used = a->out_used;
  p.num_pages = (uint32_t)a->num_pages;
  p.num_seqs = a->num_seqs;
  p.table_width = a->table_width;
  p.num_free = a->num_free;
  p.places = a->places;
  const bool in_place = overlap(a->out_lens, a->num_seqs, a->lens, a->num_seqs) ||
                        overlap(a->out_lens, a->num_seqs, a->used, 1) ||
                        overlap(a->out_used, 1, a->lens, a->num_seqs) ||
                        overlap(a->out_used, 1, a->used, 1);
  int ctas = 1;
  while (ctas < (in_place ? 8 : 64) && (int64_t)ctas * kv4::kExtendThreads < a->places) ctas *= 2;
  if (allow_extend() != cudaSuccess) return DCP_ERR_CUDA;
  return status_of(kv4::launch(kv4::extend_kernel, dim3((unsigned)ctas), kv4::kExtendThreads,
                               (size_t)a->num_seqs * kv4::kExtendRow, in_place ? ctas : 1,
                               (cudaStream_t)stream, p));
}

dcp_status dcp_rotary(const dcp_rotary_args* a, dcp_stream_t stream) {
  if (!a || (a->dtype != DCP_F16 && a->dtype != DCP_BF16 && a->dtype != DCP_F32) ||
      a->tokens < 0 || a->q_heads < 0 || a->k_heads < 0 || a->turned < 2 || a->turned % 2 ||
      a->turned > a->dim || !std::isfinite(a->magnitude))
    return DCP_ERR_INVALID;
  if (a->dim > 2 * kRotaryPairs || a->q_heads > 65536 || a->k_heads > 65536 ||
      a->tokens > INT_MAX)
    return DCP_ERR_UNSUPPORTED;
  if (a->tokens == 0 || a->q_heads + a->k_heads == 0) return DCP_OK;
  if (!a->positions || !a->turns || (a->q_heads > 0 && (!a->q || !a->q_out)) ||
      (a->k_heads > 0 && (!a->k || !a->k_out)))
    return DCP_ERR_INVALID;
  RotaryParams p{};
  p.in[0] = a->q, p.in[1] = a->k;
  p.out[0] = a->q_out, p.out[1] = a->k_out;
  p.row_stride[0] = a->q_row_stride, p.row_stride[1] = a->k_row_stride;
  p.head_stride[0] = a->q_head_stride, p.head_stride[1] = a->k_head_stride;
  p.out_row_stride[0] = a->q_out_row_stride, p.out_row_stride[1] = a->k_out_row_stride;
  p.out_head_stride[0] = a->q_out_head_stride, p.out_head_stride[1] = a->k_out_head_stride;
  p.positions = a->positions;
  p.turns = a->turns;
  p.tokens = a->tokens;
  p.q_heads = a->q_heads;
  p.heads = a->q_heads + a->k_heads;
  p.pairs = a->turned / 2;
  p.dim = a->dim;
  p.magnitude = a->magnitude;
  const int per = a->dtype == DCP_F32 ? 4 : 8;  // elements in 16 bytes
  bool vec = p.pairs % per == 0 && (a->dim - a->turned) % per == 0;
  for (int i = 0; i < 2; ++i)
    if (i == 0 ? a->q_heads : a->k_heads)
      vec = vec && fits(p.in[i], p.row_stride[i], p.head_stride[i], per) &&
            fits(p.out[i], p.out_row_stride[i], p.out_head_stride[i], per);
  const int v = vec ? per : 1;
  p.turn_items = p.pairs / v;
  p.items = p.turn_items + (a->dim - a->turned) / v;
  // Tokens together until a CTA has 1024 items, unless that leaves SMs without
  // work.  (Items of a CTA stay below the 2^16 that divide() is exact for: more
  // heads than that take the grid's second dimension.)
  p.heads_per_cta = p.heads;
  while ((int64_t)p.heads_per_cta * p.items > 32768) p.heads_per_cta = (p.heads_per_cta + 1) / 2;
  p.per_token = p.heads_per_cta * p.items;
  int sms;
  if (count_sms(&sms) != cudaSuccess) return DCP_ERR_CUDA;
  p.tokens_per_cta = 1;
  while (p.tokens_per_cta < 8 && p.tokens_per_cta * p.per_token < 1024 &&
         a->tokens > (int64_t)p.tokens_per_cta * 8 * sms)
    p.tokens_per_cta *= 2;
  p.by_token = division_by((uint32_t)p.per_token);
  p.by_head = division_by((uint32_t)p.items);
  p.by_pairs = division_by((uint32_t)p.pairs);
  const dim3 grid((unsigned)((a->tokens + p.tokens_per_cta - 1) / p.tokens_per_cta),
                  (unsigned)((p.heads + p.heads_per_cta - 1) / p.heads_per_cta));
  const bool il = a->interleaved != 0;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (a->dtype == DCP_F32)
    e = vec ? launch_rotary<float, 4>(p, il, grid, s) : launch_rotary<float, 1>(p, il, grid, s);
  else if (a->dtype == DCP_F16)
    e = vec ? launch_rotary<__half, 8>(p, il, grid, s) : launch_rotary<__half, 1>(p, il, grid, s);
  else
    e = vec ? launch_rotary<__nv_bfloat16, 8>(p, il, grid, s)
            : launch_rotary<__nv_bfloat16, 1>(p, il, grid, s);
  return status_of(e);
}

}  // extern "C"
