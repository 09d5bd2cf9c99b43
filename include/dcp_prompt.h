/*
 * dcp_prompt.h -- C ABI of what a batch's new tokens pass on their way into
 * the 4-bit cache (dcp_kv4.h): rotary positions of queries and keys, and
 * attention of whole prompts over their own keys and values.  GB300 (sm_103a).
 *
 * The conventions of dcp_topk.h hold: device pointers owned by the caller,
 * work enqueued on `stream` without synchronising, capturable after a first
 * call, argument errors reported before anything is enqueued, outputs that do
 * not overlap inputs (the one exception is named at dcp_rotary).  Results are
 * deterministic.
 */
#ifndef DCP_PROMPT_H
#define DCP_PROMPT_H

#include "dcp_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dcp_rotary -- turns pairs of elements of every head by their token's
 * position.
 *
 * Pair i of a head's first `turned` elements is (x[i], x[i + turned / 2]), or
 * (x[2i], x[2i + 1]) where interleaved; with a = positions[t] * turns[i] / 2^64
 * whole turns,
 *   y = magnitude * (x0 cos 2 pi a - x1 sin 2 pi a, x1 cos 2 pi a + x0 sin 2 pi a)
 * and the head's other elements are copied.  The product is taken modulo 2^64,
 * so the angle is exact to 2^-34 of a turn for every position, and to fp32's
 * 2^-24 of itself from there; a negative position turns back.  Products and sums are fp32, rounded once at the end.
 */
typedef struct {
    const void* q;          /* [tokens][q_heads][dim] of dtype, dim contiguous */
    const void* k;          /* [tokens][k_heads][dim], or NULL with k_heads 0 */
    void* q_out;            /* the same shapes; q_out may be q (and k_out k), with its strides */
    void* k_out;
    int64_t q_row_stride;   /* elements */
    int64_t q_head_stride;
    int64_t k_row_stride;
    int64_t k_head_stride;
    int64_t q_out_row_stride;
    int64_t q_out_head_stride;
    int64_t k_out_row_stride;
    int64_t k_out_head_stride;
    const int32_t* positions; /* [tokens] */
    const uint64_t* turns;    /* [turned / 2]: 2^64 * frequency / (2 pi) */
    int64_t tokens;
    int dtype;
    int q_heads;
    int k_heads;
    int dim;                /* at most 1024 */
    int turned;             /* even, at most dim */
    int interleaved;
    float magnitude;
} dcp_rotary_args;

/*
 * Errors: DCP_ERR_INVALID for a bad dtype, negative sizes, a turned that is odd,
 * below 2 or above dim, a magnitude that is not finite, or a NULL pointer with
 * tokens and heads > 0; DCP_ERR_UNSUPPORTED for a dim above 1024, more than
 * 65536 heads, or 2^31 tokens or more; DCP_ERR_CUDA if the launch fails.
 * tokens == 0 is a no-op.
 */
dcp_status dcp_rotary(const dcp_rotary_args* args, dcp_stream_t stream);

/*
 * dcp_prompt_attention -- every row of packed sequences against the rows of
 * its own sequence.
 *
 * Sequence b is the rows starts[b] <= t < starts[b + 1] of q, k and v.  Its
 * row i sees its rows j with j <= i (causal) and j > i - window (window > 0).
 * Query head h reads key/value head h / (q_heads / kv_heads).
 *
 *   s_j   = scale * q . k_j, then softcap * tanh(s_j / softcap) if softcap > 0
 *   lse   = ln sum_j exp(s_j);  out = sum_j exp(s_j - lse) v_j
 *
 * Products of the inputs are exact and summed in fp32; the probabilities are
 * rounded to dtype for the second product only, their sum is kept in fp32
 * (compensated).  Scores may be of any size, as long as q . k_j and s_j / ln 2
 * are finite in fp32; rows with a largest score beyond 2^20 ln 2 are computed on
 * the plain units, some 200 times slower.  What a row does not see has no
 * influence on it, whatever its value; only, an infinity or NaN among the values
 * up to 128 rows behind what it sees has it computed on the plain units too, which
 * round differently within the same bounds.  Rows of no sequence are neither read
 * nor written.  starts ascends from 0 or more to at most rows; values outside
 * are cut there.
 */
typedef struct {
    const void* q;          /* [rows][q_heads][dim] of dtype (fp16 or bf16), dim contiguous */
    const void* k;          /* [rows][kv_heads][dim] */
    const void* v;
    int64_t q_row_stride;   /* elements */
    int64_t q_head_stride;
    int64_t k_row_stride;
    int64_t k_head_stride;
    int64_t v_row_stride;
    int64_t v_head_stride;
    const int32_t* starts;  /* [num_seqs + 1] */
    void* out;              /* [rows][q_heads][dim] of dtype, contiguous, 16-byte aligned */
    float* lse;             /* [rows][q_heads], natural logarithm */
    int64_t rows;
    int dtype;
    int q_heads;            /* a multiple of kv_heads */
    int kv_heads;
    int dim;                /* 64, 128 or 256 */
    int num_seqs;
    int causal;
    int window;             /* 0: none */
    float scale;            /* 0: dim^-1/2; its magnitude is cut to 2^-126 to 2e38 */
    float softcap;          /* 0, above 2^126 |scale|, or too large to be
                               divided by ln 2 in fp32: none */
} dcp_prompt_attention_args;

/*
 * Errors: DCP_ERR_INVALID for a bad dtype, negative sizes or window, a softcap
 * that is negative, a softcap or scale that is not finite, q_heads not a
 * multiple of kv_heads, a NULL pointer with rows and num_seqs > 0, or an out or
 * lse that shares memory with an input or the other;
 * DCP_ERR_UNSUPPORTED for a dim outside the limits, sizes whose products pass
 * 2^31 - 1 (rows * q_heads), more than 65536 heads, or a q, k or v that tensor
 * copies cannot read: it is not 16-byte aligned, or a stride (of a dimension of
 * more than one element) is not a positive multiple of 8 elements;
 * DCP_ERR_CUDA if a launch fails.  rows == 0 and num_seqs == 0 are no-ops.
 * Waits are bounded: a CTA one of whose copies does not land within about a
 * second gives up.  Then DCP_DEVICE_COPY_TIMEOUT is set in the device status
 * word (dcp_topk_device_status), and the rows that it had not finished are NaN.
 */
dcp_status dcp_prompt_attention(const dcp_prompt_attention_args* args, dcp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DCP_PROMPT_H */
