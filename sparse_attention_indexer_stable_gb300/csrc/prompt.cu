// prompt.cu -- C ABI of attention over whole prompts (include/dcp_prompt.h).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "dcp_prompt.h"
#include "prompt_rows.cuh"

using namespace dcp;
using namespace dcp::prompt;

static dcp_status status_of(cudaError_t e) { return e == cudaSuccess ? DCP_OK : DCP_ERR_CUDA; }

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
  Params p{};
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
  p.capped = a->softcap > 0.0f;
  p.cap = fminf(a->softcap * kLog2e, 3e38f);
  // finite, and above 0: 0 times it stays 0, an infinity one
  p.mult = copysignf(fminf(fmaxf(fabsf(p.capped ? scale / a->softcap : scale * kLog2e), 1e-37f),
                           3e38f), scale);
  const dim3 grid((unsigned)p.rows, (unsigned)((p.q_heads + kRowWarps - 1) / kRowWarps));
  auto* kernel = a->dim == 64 ? rows_kernel<64> : a->dim == 128 ? rows_kernel<128> : rows_kernel<256>;
  return status_of(kv4::launch(kernel, grid, 32 * kRowWarps, 0, 1, (cudaStream_t)stream, p));
}
