/*
 * mla_evict.h -- C ABI of libmla_decode.so: a bounded latent cache.  Rows are
 * evicted by the attention weight they have gathered (mla_tree_weights).
 *
 * Request b has n = d_pos[b] rows.  If n > keep, `keep` of them stay: first
 * those with positions[row] < sink or positions[row] >= next_pos[b] - recent,
 * then by weight, the largest first (NaN counts as -infinity); ties go to the
 * lowest row.  Attention does not depend on the order of the rows, so rows
 * stay where they are, and the kept rows behind `keep` (ascending) move to the
 * evicted places below it (ascending): the fewest bytes moved, in place.
 * Weights and positions move with their rows.
 *
 * Conventions as in mla_decode.h.
 */
#ifndef MLA_EVICT_H_
#define MLA_EVICT_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void *kv;                    /* (device) cache rows, 16-byte aligned */
    long long kv_rows, row_stride;   /* as in mla_decode_args (bytes for an E4M3 cache) */
    int kv_fp8;                  /* 1 = rows of 576 bytes */
    int batch;                   /* 1 .. 65535 */
    int keep;                    /* rows that stay, >= 1 */
    int sink;                    /* positions 0 .. sink - 1 stay first (>= 0) */
    int recent;                  /* and the last `recent` positions before next_pos (>= 0) */
    int max_rows;                /* largest d_pos expected (>= 1): sizes the launch only */
    const float *weights;        /* (device) fp32 [kv_rows] */
    const int *positions;        /* (device) int32 [kv_rows] */
    const int *d_pos;            /* (device) int32 [B] rows of each request (clamped to the rows inside
                                    [0, kv_rows); negative = none) */
    const int *next_pos;         /* (device) int32 [B]: position of the next token; may be d_pos */
    const long long *row_offset; /* (device) int64 [B], >= 0; may be NULL for a batch of 1 */
    float *weights_out;          /* (device) fp32 [kv_rows]: may be `weights`, else no overlap with it; the
                                    first min(n, keep) entries of each request are written */
    int *positions_out;          /* (device) int32 [kv_rows], likewise */
    int *d_pos_out;              /* (device) int32 [B]: min(n, keep), 0 for a negative d_pos; may be d_pos */
} mla_evict_args;

/* Scratch bytes of a call (256-byte aligned device memory, no initial value;
 * not shared by calls that may overlap).  0 for arguments out of range. */
MLA_API size_t mla_evict_scratch_bytes(int batch, int keep);

/* Select and move (two launches).  Requests must not share cache rows.
 * Errors: MLA_EINVAL, MLA_EALIGN, MLA_ESCRATCH, MLA_ECUDA. */
MLA_API int mla_evict(const mla_evict_args *args, void *scratch, size_t scratch_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_EVICT_H_ */
