// mla_tree.cuh -- what the kernels over drafted tokens share: their parameters,
// a request's rows, and the visibility of its rows to a token.
#pragma once

#include <cstdint>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_tree.h"

namespace mla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeTileKeys = 128;                         // cache rows per tile of a CTA pair
constexpr int kTreeBlockRows = 128;                        // (token, head) rows per CTA pair

// What a cluster leaves for the merge: its last piece is the first one of a row
// block that `pieces` consecutive clusters share (0: nothing to merge).
struct TreeMerge {
    int b, rb, pieces, rows;
};

struct TreeParams {
    mla_tree_args a;
    int batch, tokens, heads;
    int clusters, min_tiles;
    float scale_log2;                                      // scale * log2(e): scores in base-2 units
    float* part;                                           // fp32 [clusters][2][128][512], normalised
    float* lse_part;                                       // fp32 [clusters][2][128], base 2
    TreeMerge* merge;                                      // [clusters]
    int* status;
    int stall_test;
    float* weights;
    float decay;
};

struct TreeRequest {
    long long base;
    int d_pos, n_tok;
    int lo, hi;                                            // rows [lo, hi) of the request lie inside the cache
};

__device__ __forceinline__ TreeRequest load_tree_request(const TreeParams& p, int b) {
    TreeRequest r;
    r.base = p.a.row_offset ? p.a.row_offset[b] : 0;
    r.d_pos = p.a.d_pos[b];
    r.n_tok = p.a.n_tokens ? min(max(p.a.n_tokens[b], 0), p.tokens) : p.tokens;
    const long long rows = r.d_pos < 0 ? 0 : static_cast<long long>(r.d_pos) + r.n_tok;
    const long long lo = r.base < 0 ? -r.base : 0, end = p.a.kv_rows - r.base;
    const long long hi = end < rows ? end : rows;
    // base > kv_rows or base <= -rows: none of the rows is inside (and base + t
    // fits 32 bits for every t < hi otherwise)
    r.hi = hi > lo ? static_cast<int>(hi) : 0;
    r.lo = hi > lo ? static_cast<int>(lo) : 0;
    return r;
}

// Mask word of a token, without the bits behind the request's drafts.
__device__ __forceinline__ unsigned long long tree_mask(const TreeParams& p, int b, int i, int n_tok) {
    const unsigned long long m =
        p.a.mask ? p.a.mask[static_cast<long long>(b) * p.tokens + i] : (~0ull >> (63 - i));
    return n_tok < 64 ? m & ((1ull << n_tok) - 1) : m;
}

__device__ __forceinline__ unsigned long long low_bits(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
// Which of the request's rows t0 .. t0 + 63 a token with this mask attends.
__device__ __forceinline__ unsigned long long visible64(const TreeRequest& r, unsigned long long mask, int t0) {
    const int d = r.d_pos - t0;                            // place of the first drafted row
    unsigned long long v = low_bits(d);
    if (d >= 0)
        v |= d < 64 ? mask << d : 0ull;
    else
        v |= -d < 64 ? mask >> -d : 0ull;
    return v & low_bits(r.hi - t0) & ~low_bits(r.lo - t0);
}

cudaError_t tree_attend_prepare();
size_t tree_attend_smem_bytes();
struct TreeMaps {
    CUtensorMap kv;                                        // boxes of 64 rows x 2 column chunks
    CUtensorMap rope;                                      // boxes of 64 rows x 1 column chunk
    CUtensorMap q;                                         // boxes of 64 rows x 9 column chunks
};
cudaError_t launch_tree_attend(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream);
cudaError_t launch_tree_weights(const TreeMaps& maps, const TreeParams& p, int num_sms, bool pdl, cudaStream_t stream);

}  // namespace mla
