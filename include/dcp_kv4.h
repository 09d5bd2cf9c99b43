/*
 * dcp_kv4.h -- C ABI of the 4-bit key/value cache that the selected token ids
 * are read from: pages and slots for new tokens, writing and reading tokens,
 * attention over a visible range or over the ids of the top-K (dcp_topk.h), and
 * eviction by accumulated attention weight.  GB300 (sm_103a).
 *
 * Format.  A token's K (or V) of one head is D elements in blocks of 16.  A
 * block's scale is s = e4m3(min(amax / (6 * unit), 448)) and its codes are
 * e2m1(x / (unit * s)), saturating, both rounded to nearest even; an element
 * stands for unit * s * e2m1(code).  Blocks whose scale rounds to 0 hold
 * zeros; NaN counts as 0 and infinities saturate.  A code and a scale have at
 * most 6 significant bits together, so the product is exact in fp16.
 *
 *   codes   uint8 [num_pages][page_size][heads][dim / 2], element 2i in the
 *           low nibble of byte i
 *   scales  uint8 [num_pages][page_size][heads][dim / 16], e4m3 bits
 *
 * A slot is page * page_size + offset.  A block table names the pages that
 * hold a sequence's positions: position p is offset p % page_size of page
 * table[p / page_size].  Table entries outside [0, num_pages) are holes: their
 * tokens are absent (never visible, not written).
 *
 * The conventions of dcp_topk.h hold: device pointers owned by the caller,
 * work enqueued on `stream` without synchronising, capturable after a first
 * call, argument errors reported before anything is enqueued, outputs that do
 * not overlap inputs.  Results are deterministic (the one exception is named
 * at `weights`).
 */
#ifndef DCP_KV4_H
#define DCP_KV4_H

#include "dcp_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of K, V, queries and outputs. */
typedef enum { DCP_F16 = 0, DCP_BF16 = 1, DCP_F32 = 2 } dcp_dtype;

typedef struct {
    uint8_t* k_codes;  /* the four planes, each 16-byte aligned */
    uint8_t* v_codes;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int64_t num_pages; /* num_pages * page_size < 2^32 */
    int page_size;     /* a power of two, at most 65536 */
    int heads;         /* key/value heads */
    int dim;           /* 64, 128 or 256 */
    float k_unit;      /* powers of two */
    float v_unit;
} dcp_kv4_cache;

/*
 * dcp_kv4_append -- quantises N tokens and writes them to their slots.
 *
 *   k, v           [N][heads][dim] of `dtype`, dim contiguous; row (token) and
 *                  head strides in elements.
 *   slots          int64 [N]; a slot outside the cache (for example -1) skips
 *                  its token.  Slots of one call are distinct.
 *
 * Errors: DCP_ERR_INVALID for a bad cache, dtype, N < 0 or a NULL pointer with
 * N > 0; DCP_ERR_UNSUPPORTED for a dim or page size outside the limits;
 * DCP_ERR_CUDA if the launch fails.  N == 0 is a no-op.
 */
dcp_status dcp_kv4_append(const dcp_kv4_cache* cache, const void* k, const void* v, int dtype,
                          int64_t N, int64_t k_row_stride, int64_t k_head_stride,
                          int64_t v_row_stride, int64_t v_head_stride, const int64_t* slots,
                          dcp_stream_t stream);

/*
 * dcp_kv4_read -- what N slots stand for: k, v [N][heads][dim] of `dtype`,
 * contiguous, 16-byte aligned.  Slots outside the cache read as zeros; slots
 * may repeat.  fp16 outputs saturate at infinity where unit lifts a value
 * beyond 65504.  Errors as dcp_kv4_append.
 */
dcp_status dcp_kv4_read(const dcp_kv4_cache* cache, void* k, void* v, int dtype, int64_t N,
                        const int64_t* slots, dcp_stream_t stream);

/*
 * dcp_kv4_attention -- one query row against the tokens that it sees.
 *
 * Row t belongs to sequence b = owner[t] (owner NULL: b = t) and sees the
 * positions p with starts[t] <= p < lens[t] (starts NULL: 0) whose page is in
 * the table; with ids, only those among the row's ids.  Query head h reads
 * key/value head h / (q_heads / heads).
 *
 *   s_j   = scale * q . k_j, then softcap * tanh(s_j / softcap) if softcap > 0
 *   lse   = ln sum_j exp(s_j);  out = sum_j exp(s_j - lse) v_j
 *
 * A row that sees nothing gives out = 0 and lse = -inf.  Products are exact
 * (fp16 operands: a query row is scaled by a power of two into fp16's range,
 * the cache's values are exact in fp16) and summed in fp32; the probabilities
 * are rounded to fp16 for the second product only, their sum is kept in fp32
 * (compensated).  Scores beyond 1e8 in magnitude, where fp32's steps span most
 * of the exponent's range, may give NaN, or lose their weight without a sign.
 */
typedef struct {
    const void* q;          /* [rows][q_heads][dim] of dtype (fp16 or bf16), dim contiguous */
    int64_t q_row_stride;   /* elements */
    int64_t q_head_stride;
    const int32_t* table;   /* block table [num_seqs][table_width] */
    int64_t table_stride;   /* elements between sequences */
    const int32_t* lens;    /* [rows]; negative counts as 0, beyond the table as its end */
    const int32_t* starts;  /* [rows] or NULL */
    const int32_t* owner;   /* [rows] or NULL (row t is sequence t); outside
                               [0, num_seqs): the row sees nothing */
    const int32_t* ids;     /* [rows][num_ids] or NULL (every visible position); -1 is padding;
                               an id is position + row_starts[t]; a repeated id counts as often
                               as it is listed */
    int64_t ids_stride;     /* elements between rows */
    const int32_t* row_starts; /* [rows] or NULL (all zero), as given to the top-K */
    float* weights;         /* [rows][weights_stride] or NULL: weights[t][p] += the row's
                               probability of position p, summed over the query heads.  Needs
                               owner == NULL; positions beyond weights_width are dropped.  With
                               ids, an id listed twice adds twice, in either order (the one
                               result whose last bits may vary). */
    int64_t weights_stride;
    int64_t weights_width;
    void* out;              /* [rows][q_heads][dim] of dtype, contiguous, 16-byte aligned */
    float* lse;             /* [rows][q_heads] */
    void* workspace;        /* dcp_kv4_attention_workspace_size bytes, 16-byte aligned */
    size_t workspace_bytes;
    int dtype;
    int rows;
    int q_heads;            /* a multiple of the cache's heads */
    int num_seqs;
    int table_width;        /* pages per sequence */
    int num_ids;
    int max_len;            /* positions from here on are not seen, whatever lens says (0: the
                               table's end); the split of the work and the workspace go by it */
    float scale;            /* 0: dim^-1/2 */
    float softcap;          /* 0: none */
} dcp_kv4_attention_args;

/*
 * Workspace bytes of a call with these arguments; the pointers are not read,
 * only whether ids and weights are NULL.  Errors as dcp_kv4_attention's size
 * checks.
 */
dcp_status dcp_kv4_attention_workspace_size(const dcp_kv4_cache* cache,
                                            const dcp_kv4_attention_args* args, size_t* bytes);

/*
 * Errors: DCP_ERR_INVALID for a bad cache or dtype, negative sizes, a softcap
 * that is negative, a softcap or scale that is not finite, q_heads not a
 * multiple of heads, a NULL required pointer with rows > 0, weights with
 * owner, or a workspace smaller than reported; DCP_ERR_UNSUPPORTED for a dim
 * or page size outside the limits, more than 2^31 - 1 positions, or weights of
 * more than 4096 query heads;
 * DCP_ERR_CUDA if a launch fails.  rows == 0 is a no-op.
 * Waits for copies are bounded: a CTA one of whose copies does not land within
 * about a second gives up and ends a second later.  Then
 * DCP_DEVICE_COPY_TIMEOUT is set in the device status word
 * (dcp_topk_device_status), and the rows that the CTA had not finished are NaN.
 */
dcp_status dcp_kv4_attention(const dcp_kv4_cache* cache, const dcp_kv4_attention_args* args,
                             dcp_stream_t stream);

/*
 * dcp_kv4_evict -- copies the tokens worth keeping into other pages.
 *
 * A sequence of n = lens[b] <= budget tokens keeps them all.  A longer one
 * keeps its first `sinks` and last `recent` positions and, of the others, the
 * budget - sinks - recent with the largest weights (equal weights: the lowest
 * position; NaN ranks below everything).  Kept tokens move in their order to
 * positions 0, 1, ... of out_table.  A kept token on a hole of table becomes
 * zeros, as it reads; what falls on a hole of out_table is not written.  The
 * source pages are left as they are; the pages of out_table must not be among
 * them.
 */
typedef struct {
    const int32_t* table;      /* [num_seqs][table_width] */
    int64_t table_stride;
    const int32_t* lens;       /* [num_seqs]; beyond the table's or the weights' width: cut there */
    const float* weights;      /* [num_seqs][weights_width] */
    int64_t weights_stride;
    const int32_t* out_table;  /* [num_seqs][ceil(budget / page_size)] */
    int64_t out_table_stride;
    int32_t* kept;             /* [num_seqs][budget]: kept positions, ascending, then -1 */
    int32_t* out_lens;         /* [num_seqs]: min(n, budget) */
    float* out_weights;        /* [num_seqs][budget]: the kept tokens' weights, then 0 */
    int num_seqs;
    int table_width;
    int weights_width;
    int budget;
    int sinks;
    int recent;                /* sinks + recent <= budget */
} dcp_kv4_evict_args;

/*
 * Errors: DCP_ERR_INVALID for a bad cache, negative sizes, budget < 1,
 * sinks + recent > budget or a NULL pointer with num_seqs > 0;
 * DCP_ERR_UNSUPPORTED as above; DCP_ERR_CUDA if a launch fails.
 * num_seqs == 0 is a no-op.
 */
dcp_status dcp_kv4_evict(const dcp_kv4_cache* cache, const dcp_kv4_evict_args* args,
                         dcp_stream_t stream);

/*
 * dcp_kv4_extend -- pages and slots for the new tokens of a batch.
 *
 * Sequence b holds lens[b] tokens and gets counts[b] more (negative values
 * count as 0).  The new tokens of all sequences take `places` places, one
 * sequence after the other; tokens behind the last place are not taken in.
 * Where a sequence's tokens reach beyond the pages that its lens[b] tokens
 * fill, it takes further pages from the list of free ones, sequence by
 * sequence, from entry used[0] on, and they are written into its row of the
 * table.  Pages wanted beyond the list's end are holes (-1); pages beyond the
 * table's width are not taken.
 *
 * Of a place's token: its slot (-1 where its page is a hole or beyond the
 * table), position, sequence (owner) and the number of positions that it sees
 * with itself (row_lens).  Places behind the last token: slot -1, position 0,
 * owner -1, row_lens 0, which dcp_kv4_append skips and dcp_kv4_attention
 * answers with zeros.  starts[b] is the first place of sequence b, as
 * dcp_prompt_attention takes it.
 */
typedef struct {
    int32_t* table;             /* [num_seqs][table_width]; the new pages are written */
    int64_t table_stride;       /* elements between sequences */
    const int32_t* lens;        /* [num_seqs] */
    const int32_t* counts;      /* [num_seqs] */
    const int32_t* free_pages;  /* [num_free], distinct */
    const int32_t* used;        /* [1]: entries of free_pages given away so far; negative
                                   counts as 0 */
    int64_t* slots;             /* [places] */
    int32_t* positions;         /* [places] */
    int32_t* owner;             /* [places] */
    int32_t* row_lens;          /* [places] */
    int32_t* starts;            /* [num_seqs + 1] */
    int32_t* out_lens;          /* [num_seqs]: lens with the new tokens; may be lens */
    int32_t* out_used;          /* [1]: used with the pages wanted, beyond num_free by as many as
                                   were missing; may be used */
    int64_t num_pages;          /* of the cache; num_pages * page_size < 2^32 */
    int page_size;              /* a power of two, at most 65536 */
    int num_seqs;               /* at most 16384 */
    int table_width;            /* pages per sequence */
    int num_free;
    int places;
} dcp_kv4_extend_args;

/*
 * Errors: DCP_ERR_INVALID for negative sizes or a NULL pointer that is needed;
 * DCP_ERR_UNSUPPORTED for a page size or num_pages outside the limits, more
 * than 16384 sequences, or more than 2^31 - 1 positions; DCP_ERR_CUDA if the
 * launch fails.  Positions and lengths stop at 2^31 - 1.
 */
dcp_status dcp_kv4_extend(const dcp_kv4_extend_args* args, dcp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DCP_KV4_H */
