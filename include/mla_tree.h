/*
 * mla_tree.h -- C ABI of libmla_decode.so: several drafted tokens per request
 * over the latent cache.
 *
 * Request b has d_pos[b] committed cache rows (its rows row_offset[b] + 0 ..
 * d_pos[b] - 1) and n_tokens[b] drafted tokens; drafted token j's row is
 * row_offset[b] + d_pos[b] + j (mla_rope_append writes it).  Token i attends
 * every committed row and the drafted rows j whose bit is set in its mask
 * (its ancestors in the tree of drafts, and itself):
 *
 *     s_t = (q_lat . c_t + q_rope . k_rope_t) * scale
 *     lse = ln sum_t exp(s_t),     out = sum_t exp(s_t - lse) c_t
 *
 * With one token and mask 1 this is mla_decode_forward's dense decode (with
 * fp32 outputs within its error, too).
 *
 * Products of q and k are exact; their fp32 sums (the tensor cores') drop what
 * does not fit, towards zero: a score is within 2^-13 of the sum of its
 * products' magnitudes, and exact where nothing is dropped.  With normal
 * queries and rows scores come out smaller by about 4e-7 of themselves (in
 * mla_tree_weights, which adds two sums of half the length, by 1e-7).
 *
 * What a token does not attend does not reach its result, whatever it holds
 * (NaN and infinities too): rows behind the drafts, drafted rows its mask
 * leaves out, rows outside [0, kv_rows), rows t >= 2^31 - 256 of a request.
 * An attended row with a NaN, or whose score is NaN or +infinity, makes the
 * whole result of the (token, head) NaN; one whose score is -infinity adds
 * nothing, or a NaN to those elements of the result where its latent is infinite.
 * A token that attends no row gets out = 0 and lse = -infinity.  Outputs of
 * the tokens behind n_tokens[b] are left as they were.
 *
 * Conventions as in mla_decode.h.
 */
#ifndef MLA_TREE_H_
#define MLA_TREE_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_TREE_MAX_TOKENS 64   /* one mask word per token */

typedef struct {
    int batch;            /* 1 .. 4096 requests */
    int tokens;           /* Q: largest number of drafted tokens per request, 1 .. 64 */
    int heads;            /* 1 .. 128 */
    float scale;          /* softmax scale, > 0 and below 2.3e38 */
    int num_sms;          /* SMs to plan for; 0 = query the current device and prepare the kernels there */
    int pdl;              /* 1 = launch with programmatic dependent launch */
    int stall_test;       /* test hook, as in mla_decode_shape */
} mla_tree_shape;

/* Launch plan (plain data).  Every launch checks it against its shape. */
typedef struct {
    mla_tree_shape shape;
    int magic;
    int num_sms;
    int grid;                  /* CTAs of the attention kernel */
    size_t scratch_bytes;
    size_t status_offset;      /* int32 status word: 0 healthy, else an mla_status */
    size_t part_offset;        /* fp32 pieces of outputs */
    size_t lse_part_offset;    /* fp32 log-sum-exps of the pieces */
} mla_tree_plan_t;

typedef struct {
    const void *q;               /* (device) bf16 [B][Q][heads][576], 16-byte aligned */
    const void *kv;              /* (device) bf16 cache rows, 16-byte aligned */
    long long kv_rows;           /* rows addressable in kv, below 2^31 - 256 */
    long long row_stride;        /* elements between rows: >= 576, a multiple of 8 */
    const int *d_pos;            /* (device) int32 [B] committed rows; a request with d_pos < 0 attends nothing */
    const long long *row_offset; /* (device) int64 [B]; may be NULL for a batch of 1 */
    const unsigned long long *mask; /* (device) uint64 [B][Q], bit j of word i: token i attends drafted token j;
                                    NULL = a chain (token i attends drafts 0 .. i).  Bits at or above
                                    n_tokens[b] are ignored */
    const int *n_tokens;         /* (device) int32 [B], clamped to 0 .. Q; NULL = Q for every request */
    void *out;                   /* (device) bf16 or fp32 [B][Q][heads][512], 16-byte aligned */
    int out_fp32;                /* 1 = fp32 outputs (e.g. for mla_decode_project): probabilities enter the product
                                    in 16 bits and more, as in the decode.  0 = bf16 outputs: they enter as one
                                    bf16 each (2^-8), which over few rows can show beside the output's own rounding */
    float *lse;                  /* (device) fp32 [B][Q][heads], natural log */
} mla_tree_args;

/* Plan for a shape.  With num_sms == 0 call it before any capture.
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED, MLA_ECUDA. */
MLA_API int mla_tree_plan(const mla_tree_shape *shape, mla_tree_plan_t *plan);

/* Attention of the drafted tokens.  `scratch` (device) as in mla_decode_run:
 * 256-byte aligned, plan->scratch_bytes, zeroed once (mla_decode_scratch_init),
 * not shared by calls that may overlap.  Results are the same bit for bit in
 * every run of the same plan and inputs.
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED (kv_rows), MLA_EALIGN, MLA_ESCRATCH,
 * MLA_ENOTREADY, MLA_ECUDA. */
MLA_API int mla_tree_forward(const mla_tree_plan_t *plan, const mla_tree_args *args, void *scratch,
                             size_t scratch_bytes, void *stream);

/* Attention weight that each cache row got, summed over the call's tokens and
 * heads, added to a decayed running sum:
 *     weights[row] = decay * weights[row] + sum_{i, h} exp(s - lse[i][h])
 * for the rows row = row_offset[b] + t, t < d_pos[b] + n_tokens[b], inside
 * [0, kv_rows); other entries are left as they are.  args as for
 * mla_tree_forward, whose lse it reads (out is not used; a (token, head) with
 * lse = -infinity adds nothing).  weights: (device) fp32 [kv_rows].  decay:
 * finite, 0 .. 1; with 0 the old weights are not read.  Requests must not
 * share cache rows.  Needs the plan's scratch (status word); one launch.
 * Errors as mla_tree_forward. */
MLA_API int mla_tree_weights(const mla_tree_plan_t *plan, const mla_tree_args *args, float *weights, float decay,
                             void *scratch, size_t scratch_bytes, void *stream);

typedef struct {
    void *kv;                    /* (device) cache rows, 16-byte aligned */
    long long kv_rows, row_stride;   /* as in mla_decode_args (bytes for an E4M3 cache) */
    int kv_fp8;                  /* 1 = rows of 576 bytes */
    int batch;                   /* 1 .. 65535 */
    int tokens;                  /* entries per path, 1 .. 64 */
    const int *accept;           /* (device) int32 [B][tokens]: the accepted drafts in path order, any order */
    const int *n_accept;         /* (device) int32 [B], clamped to 0 .. tokens */
    const int *d_pos;            /* (device) int32 [B] committed rows (>= 0; a negative one is left alone) */
    int *d_pos_out;              /* (device) int32 [B]: d_pos + n_accept; may be d_pos; NULL = not written */
    const long long *row_offset; /* (device) int64 [B]; may be NULL for a batch of 1 */
    int *row_positions;          /* (device) int32 [kv_rows] or NULL: moved with the rows */
    float *row_weights;          /* (device) fp32 [kv_rows] or NULL: moved with the rows */
} mla_tree_commit_args;

/* Move the accepted drafts' rows together behind the committed rows: row
 * d_pos + k takes what row d_pos + accept[k] held before the call, for
 * k < n_accept.  An entry outside 0 .. 63, or a row outside [0, kv_rows),
 * leaves its destination as it was.  Requests must not share cache rows.  One
 * launch.  Errors: MLA_EINVAL, MLA_EALIGN, MLA_ECUDA. */
MLA_API int mla_tree_commit(const mla_tree_commit_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_TREE_H_ */
