/*
 * mla_paged.h -- C ABI of libmla_decode.so: a latent cache in 4 bits, in pages.
 *
 * A row is 416 bytes (26 units of 16):
 *
 *     bytes   0 .. 255   512 latent values in 4 bits, E2M1 (sign, 2 exponent bits, 1 mantissa bit:
 *                        0, 0.5, 1, 1.5, 2, 3, 4, 6); feature 2 i in the low half of byte i
 *     bytes 256 .. 287   32 scales, E4M3, one per 16 features
 *     bytes 288 .. 415   64 rotated key values, bf16
 *
 * and a latent value is code * scale * kv_scale, kv_scale a power of two.  That
 * product has six significant bits at most: it is exact in bf16 and in f16.
 *
 * A page is page_rows rows, one after the other, page_stride bytes from page to
 * page (a pool may hold several layers: pages + layer * page_rows * 416, with the
 * stride of all layers).  Row t of request b is row t % page_rows of page
 * page_table[b][t / page_rows].  Entries outside [0, n_pages) name no page: their
 * rows are not attended, not written and read as zeros.
 *
 * d_pos[b] rows of a request are committed, and new token i stands in row
 * d_pos[b] + i, as in mla_tree.h.
 *
 * Conventions as in mla_decode.h: device pointers owned by the caller, no
 * allocation, no synchronisation, asynchronous on `stream`, legal inside
 * capture, arguments checked on the host, an mla_status returned.
 */
#ifndef MLA_PAGED_H_
#define MLA_PAGED_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_Q4_ROW 416           /* bytes of a row */
#define MLA_Q4_BLOCK 16          /* features per scale */
#define MLA_PAGED_MAX_TOKENS 64  /* new tokens per request of one attention call */

/* The pages that a call works on, and each request's. */
typedef struct {
    void *pages;             /* (device) 16-byte aligned */
    long long page_stride;   /* bytes from page to page: a multiple of 16, at least a page */
    int n_pages;             /* 1 .. 2^31 - 1 */
    int page_rows;           /* rows per page: a power of two, 8 .. 1024 */
    const int *page_table;   /* (device) int32 [B][columns] */
    int columns;             /* pages per request, 1 .. (2^31 - 256) / page_rows */
    float kv_scale;          /* a power of two, 2^-64 .. 2^64 */
} mla_paged_cache;

/* ---- writing rows ------------------------------------------------------------
 *
 * New tokens' latents, keys and queries, normalised, rotated and written, in one
 * pass.  Each norm is x * (mean(x^2) + eps)^(-1/2) * weight over the vector: 512
 * latent values, 64 key values, 64 rotated query values of each head.  Keys and
 * queries are rotated as in mla_rope.h after their norm.  Sums are fp32 (those of the
 * latents keep the bits that fp32 drops: a mean is right to 2^-40); squares
 * have to stay below 2^127.
 *
 * A block of 16 latent values is written as
 *     scale = E4M3(min(max|x| / 6 / kv_scale, 448)),  code = E2M1(x / (scale * kv_scale)),
 * both to nearest, halfway to the even code, codes beyond +-6 as +-6 (1 / 6 and the
 * reciprocal of scale * kv_scale are fp32 values that x is multiplied by).  A block whose
 * scale comes out as 0 is written as zeros; one with a NaN as NaN, all of it. */
typedef struct {
    mla_paged_cache cache;
    int batch;                  /* B: 1 .. 65535 requests */
    int tokens;                 /* N: new tokens per request (the largest), 1 .. 2^28 */
    int heads;                  /* 0 .. 128; 0 = no queries */
    int rot_dim;                /* as in mla_rope_args, and so on */
    int interleaved;
    float amplitude;
    const unsigned long long *turns;
    const int *positions;       /* (device) int32 [B][N], >= 0 */
    const int *n_tokens;        /* (device) int32 [B], clamped to 0 .. N; NULL = N */
    const void *q_rope;         /* (device) bf16 [B][N][heads][64], 16-byte aligned, strides multiples of 8 */
    long long q_rope_batch, q_rope_token, q_rope_head;
    void *q_out;                /* (device) as in mla_rope_args; heads in places of their own: strides of 64 or more
                                   (or -64 or less) where there are several requests, tokens, heads */
    long long q_out_batch, q_out_token, q_out_head;
    const void *c;              /* (device) bf16 [B][N][512] */
    long long c_batch, c_token;
    const void *k_rope;         /* (device) bf16 [B][N][64] */
    long long k_rope_batch, k_rope_token;
    const void *c_norm;         /* (device) bf16 [512] weights, 16-byte aligned, or NULL: no norm */
    const void *k_norm;         /* (device) bf16 [64], likewise */
    const void *q_norm;         /* (device) bf16 [64], likewise (only with heads > 0) */
    float eps;                  /* finite, >= 0 */
    const int *d_pos;           /* (device) int32 [B]; a request with d_pos < 0 writes no row */
} mla_paged_append_args;

/* One launch.  Rows must not be written twice by one call (pages that two requests share hold
 * rows before their d_pos only).  c, k_rope, cache.pages and d_pos may all be NULL: queries
 * alone.  d_pos is not advanced.
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED (heads, rot_dim), MLA_EALIGN, MLA_ECUDA. */
MLA_API int mla_paged_append(const mla_paged_append_args *args, void *stream);

/* Rows back as bf16 [c | k_rope] rows of 576: out[b][n] = row first[b] + n of request b, for
 * n < n_rows[b] (what lies behind is left as it was); zeros for a row without a page. */
typedef struct {
    mla_paged_cache cache;
    int batch;                  /* 1 .. 65535 */
    int rows;                   /* N: largest number of rows per request, 1 .. 2^28 */
    const int *first;           /* (device) int32 [B]; NULL = 0 */
    const int *n_rows;          /* (device) int32 [B], clamped to 0 .. N; NULL = N */
    void *out;                  /* (device) bf16 [B][N][576], 16-byte aligned */
    long long out_batch, out_row;   /* strides in elements, multiples of 8, out_row >= 576; requests in places
                                       of their own: |out_batch| >= 576 where batch > 1 */
} mla_paged_read_args;
MLA_API int mla_paged_read(const mla_paged_read_args *args, void *stream);

/* ---- attention ---------------------------------------------------------------
 *
 * Token i of request b stands in row r = d_pos[b] + i and attends the rows t <= r with
 *     window == 0   or   t > r - window   or   t < sink
 * whose page exists:
 *     s_t = (q_lat . c_t + q_rope . k_rope_t) * scale
 *     lse = ln sum_t exp(s_t),     out = sum_t exp(s_t - lse) c_t
 *
 * q_lat enters the product in f16 times a power of two per query row, set by the largest of
 * |q_lat| and |q_rope| / kv_scale: values down to 2^-31 of it are exact, smaller ones off by at
 * most 2^-39 of it.  (Where that largest times scale * kv_scale is below 2^-110, scores are off by less
 * than 2^-100 instead; above 2^141, scores that are not 0 may come out smaller than they are, or infinite.)
 * Latents are exact; key values and q_rope are bf16.  Probabilities enter the second product in f16, for
 * bf16 and fp32 outputs alike: off by up to 2^-11 each, those below 2^-21 of the largest by up to 2^-32 of
 * it; sums and statistics are fp32.
 *
 * What a token does not attend does not reach its result, whatever the bytes are.  An attended
 * row with a NaN, or whose score is NaN or +infinity, makes the whole result of the (token,
 * head) NaN.  A token that attends no row gets out = 0 and lse = -infinity.  Outputs of the
 * tokens behind n_tokens[b] are left as they were.  Results are the same bit for bit in every run
 * of the same plan and inputs. */
typedef struct {
    int batch;            /* 1 .. 4096 requests */
    int tokens;           /* Q: largest number of new tokens per request, 1 .. 64 */
    int heads;            /* 1 .. 128 */
    float scale;          /* softmax scale, > 0 and below 2^60 */
    int num_sms;          /* SMs to plan for; 0 = query the current device and prepare the kernels there */
    int pdl;              /* 1 = launch with programmatic dependent launch */
    int stall_test;       /* test hook, as in mla_decode_shape */
} mla_paged_shape;

typedef struct {
    mla_paged_shape shape;
    int magic;
    int num_sms;
    int grid;                  /* CTAs of the attention kernel */
    size_t scratch_bytes;
    size_t status_offset;      /* int32 status word: 0 healthy, else an mla_status */
    size_t part_offset;        /* fp32 pieces of outputs */
    size_t lse_part_offset;    /* fp32 log-sum-exps of the pieces */
} mla_paged_plan_t;

typedef struct {
    mla_paged_cache cache;
    const void *q;               /* (device) bf16 [B][Q][heads][576], 16-byte aligned */
    const int *d_pos;            /* (device) int32 [B]; a request with d_pos < 0 attends nothing */
    const int *n_tokens;         /* (device) int32 [B], clamped to 0 .. Q; NULL = Q */
    int window;                  /* >= 0; 0 = all rows */
    int sink;                    /* >= 0 (with a window) */
    void *out;                   /* (device) bf16 or fp32 [B][Q][heads][512], 16-byte aligned */
    int out_fp32;
    float *lse;                  /* (device) fp32 [B][Q][heads], natural log */
} mla_paged_args;

/* Plan for a shape.  With num_sms == 0 call it before any capture.
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED, MLA_ECUDA. */
MLA_API int mla_paged_plan(const mla_paged_shape *shape, mla_paged_plan_t *plan);

/* `scratch` (device) as in mla_tree_forward.
 * Errors: MLA_EINVAL, MLA_EUNSUPPORTED, MLA_EALIGN, MLA_ESCRATCH, MLA_ENOTREADY, MLA_ECUDA. */
MLA_API int mla_paged_forward(const mla_paged_plan_t *plan, const mla_paged_args *args, void *scratch,
                              size_t scratch_bytes, void *stream);

/* ---- pages -------------------------------------------------------------------
 *
 * For pages of any rows (row_bytes a multiple of 16): 4-bit rows, E4M3 rows, bf16 rows. */
typedef struct {
    void *pages;                /* (device) 16-byte aligned */
    long long page_stride;      /* bytes, a multiple of 16, >= page_rows * row_bytes */
    int n_pages;                /* 1 .. 2^30 */
    int page_rows;              /* a power of two, 8 .. 1024 */
    int row_bytes;              /* a multiple of 16, 16 .. 65536 */
    int batch;                  /* 1 .. 4096 */
    int columns;                /* 1 .. (2^31 - 256) / page_rows, batch * columns below 2^30 */
    const int *page_table;      /* (device) int32 [B][columns] */
    const int *d_pos;           /* (device) int32 [B] rows of each request (negative = none) */
    const int *parent;          /* (device) int32 [B]: request b goes on from request parent[b]'s rows; outside
                                   [0, B) it ends.  NULL = every request from its own */
    const int *rows;            /* (device) int32 [B]: how many of them, at most (negative = 0).  NULL = all */
    int reserve;                /* >= 0: pages for so many rows more are taken */
    int window, sink;           /* as in mla_paged_args, for the next call: full pages that no token from here on
                                   attends are given back (window 0: none) */
    int *page_table_out;        /* (device) int32 [B][columns]; may be page_table */
    int *d_pos_out;             /* (device) int32 [B]: n; may be d_pos */
    int *refs;                  /* (device) int32 [n_pages]: how many entries of page_table_out name each page */
    int *missing;               /* (device) int32 [1]: pages that there were too few of */
} mla_pages_fork_args;

/* Pages that a request of the next step names, after n = min(rows[b], d_pos[parent[b]]) rows, rounded down to full
 * pages where the page that they would end in is missing (those rows are not there):
 *   - full ones (rows 0 .. n - 1 fill them) are its parent's, shared;
 *   - a last one that n ends in: its parent's, if no request has that page as a full one and of those that
 *     end in it this one comes first; otherwise a copy of its n % page_rows rows in a page of its own;
 *   - pages of its own for the rows n .. n + reserve - 1.
 * All other entries are -1, and pages that no entry names are free (there is no list of free
 * pages: refs is made anew from the tables).  Pages are taken, in the order of requests and columns,
 * the lowest free number first.  Where they run out, entries stay -1 and `missing` counts them; a
 * request whose last page could not be copied gets n rounded down to full pages too (a window has given pages back by
 * the n before that).  Columns past the table's end are not reserved.
 * Rows appended where an entry is -1 are not written.  A caller that finds `missing` above 0 does not count them in d_pos:
 * a later call takes them back where n ends in a missing page, but full pages that are missing stay gaps.
 * Errors: MLA_EINVAL, MLA_EALIGN, MLA_ESCRATCH, MLA_ECUDA. */
MLA_API int mla_pages_fork(const mla_pages_fork_args *args, void *scratch, size_t scratch_bytes, void *stream);

typedef struct {
    void *pages;                /* as above */
    long long page_stride;
    int n_pages, page_rows, row_bytes, batch, columns;
    const int *page_table;      /* (device) int32 [B][columns] */
    const int *refs;            /* (device) int32 [n_pages]: a page is in use where this is above 0 */
    int *page_table_out;        /* (device) int32 [B][columns]; may be page_table */
    int *refs_out;              /* (device) int32 [n_pages]; may be refs */
    int *used;                  /* (device) int32 [1]: pages in use (-1: a copy did not arrive in time) */
} mla_pages_compact_args;

/* Move the pages in use to the pages 0 .. used - 1: those behind `used`, in ascending order, to the
 * unused ones before it, in ascending order; the others stay.  Entries of the table follow their
 * pages; an entry that names no page, or an unused one, becomes -1.
 * Errors: MLA_EINVAL, MLA_EALIGN, MLA_ESCRATCH, MLA_ECUDA. */
MLA_API int mla_pages_compact(const mla_pages_compact_args *args, void *scratch, size_t scratch_bytes, void *stream);

/* Scratch bytes of both calls (256-byte aligned device memory, no initial value; not shared by
 * calls that may overlap).  0 for arguments out of range. */
MLA_API size_t mla_pages_scratch_bytes(int batch, int columns, int n_pages);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGED_H_ */
