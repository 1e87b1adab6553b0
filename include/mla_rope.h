/*
 * mla_rope.h -- C ABI of libmla_decode.so: rotary positions of an MLA decode
 * step, and the write of the rotated rows to the latent cache.
 *
 * The decode kernels of mla_decode.h take q = [q_lat | q_rope] and cache rows
 * [c | k_rope] whose rope parts are rotated already.  mla_rope_append does
 * that for the new tokens of each request: it rotates the 64 rope elements of
 * every query head into the query's rope columns, rotates k_rope, and writes
 * [c | k_rope] to the cache rows behind the request's committed rows.
 *
 * A pair (x, y) of token position p and pair index j < rot_dim / 2 becomes
 *     (A (x cos t - y sin t), A (y cos t + x sin t)),   t = p * f_j
 * pairs being elements (2j, 2j + 1) (interleaved) or (j, j + rot_dim / 2);
 * elements rot_dim .. 63 are copied unscaled.  f_j is held as a 64-bit fraction
 * of a turn, so p * f_j is reduced exactly in integer arithmetic however far
 * the position; sums and products are fp32, rounded once to the output type.
 *
 * Conventions as in mla_decode.h: device pointers owned by the caller, no
 * allocation, no synchronisation, asynchronous on `stream`, legal inside
 * capture, arguments checked on the host, an mla_status returned.
 */
#ifndef MLA_ROPE_H_
#define MLA_ROPE_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_ROPE_MAX_PAIRS 32

typedef enum { MLA_ROPE_PLAIN = 0, MLA_ROPE_LINEAR = 1, MLA_ROPE_YARN = 2 } mla_rope_scaling;

/* The angle per position of each pair: f_j = base^(-2j / rot_dim), then
 *   MLA_ROPE_LINEAR: f_j / factor;
 *   MLA_ROPE_YARN:   f_j (1 - r_j) + (f_j / factor) r_j, where r_j rises from
 *     0 to 1 between the pair that turns beta_fast times over original_ctx
 *     positions and the one that turns beta_slow times (both rounded outwards
 *     to whole pairs and held within 0 .. rot_dim - 1). */
typedef struct {
    int rot_dim;            /* rotated elements of the 64: a multiple of 8, 8 .. 64 */
    int scaling;            /* mla_rope_scaling */
    double base;            /* finite, >= 1 */
    double factor;          /* finite, >= 1 (LINEAR, YARN) */
    double original_ctx;    /* finite, >= 1 (YARN) */
    double beta_fast;       /* beta_fast > beta_slow > 0, finite (YARN) */
    double beta_slow;
} mla_rope_spec;

/* Fill turns[0 .. rot_dim / 2) with f_j / (2 pi) as 64-bit fractions of a turn
 * (host memory; copy them to the device for mla_rope_append).  Host only.
 * Errors: MLA_EINVAL. */
MLA_API int mla_rope_table(const mla_rope_spec *spec, unsigned long long *turns);

typedef struct {
    int batch;                  /* B: 1 .. 65535 requests */
    int tokens;                 /* N: new tokens per request (the largest), 1 .. 2^28 */
    int heads;                  /* 0 .. 128; 0 = no queries */
    int rot_dim;                /* as in the table */
    int interleaved;            /* 1 = pairs (2j, 2j + 1); 0 = pairs (j, j + rot_dim / 2) */
    float amplitude;            /* A: finite and > 0; the caller's to give (YaRN's usual one: 0.1 ln(factor) + 1) */
    const unsigned long long *turns; /* (device) mla_rope_table's values */
    const int *positions;       /* (device) int32 [B][N], >= 0 */
    const int *n_tokens;        /* (device) int32 [B], new tokens of each request (clamped to 0 .. N);
                                   NULL = N.  Nothing is read or written for the tokens behind them */
    /* queries (heads > 0): bf16, 16-byte aligned, strides in elements, multiples of 8 */
    const void *q_rope;         /* (device) [B][N][heads][64] */
    long long q_rope_batch, q_rope_token, q_rope_head;
    void *q_out;                /* (device) where element 0 of the rotated part goes: q + 512 for q rows of
                                   576; may be q_rope itself (same pointer and strides), else no overlap */
    long long q_out_batch, q_out_token, q_out_head;
    /* cache rows: all of c, k_rope, kv, d_pos, or none (NULL) for queries alone */
    const void *c;              /* (device) bf16 [B][N][512], 16-byte aligned, strides multiples of 8 */
    long long c_batch, c_token;
    const void *k_rope;         /* (device) bf16 [B][N][64], likewise */
    long long k_rope_batch, k_rope_token;
    void *kv;                   /* (device) cache rows; token n of request b goes to row
                                   row_offset[b] + d_pos[b] + n (not written outside [0, kv_rows)) */
    long long kv_rows, row_stride;   /* as in mla_decode_args (bytes for an E4M3 cache) */
    int kv_fp8;                 /* 0 = bf16 rows; 1 = E4M3 bytes of value / kv_scale, to nearest even,
                                   beyond +-448 the largest finite value, NaN stays NaN */
    float kv_scale;             /* finite and > 0 (E4M3) */
    const int *d_pos;           /* (device) int32 [B]: committed rows; a request with d_pos < 0 writes no row */
    const long long *row_offset;/* (device) int64 [B]; may be NULL for a batch of 1 */
    int *row_positions;         /* (device) int32 [kv_rows] or NULL: the new rows' positions (for mla_evict) */
    float *row_weights;         /* (device) fp32 [kv_rows] or NULL: set to 0 for the new rows */
} mla_rope_args;

/* Rotate the new tokens' queries and keys and append their rows (one launch).
 * Requests must not share cache rows.  d_pos is not advanced
 * (mla_tree_commit or mla_decode_advance does that).
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED (heads, rot_dim), MLA_EALIGN, MLA_ECUDA. */
MLA_API int mla_rope_append(const mla_rope_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_ROPE_H_ */
