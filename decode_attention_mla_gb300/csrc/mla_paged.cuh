// mla_paged.cuh -- what the host side and the kernels of the attention over the
// 4-bit paged cache share.
#pragma once

#include "mla_q4.cuh"
#include "mla_tree.cuh"

namespace mla {

struct PagedParams : TreeParams {                          // (of a.*: d_pos, n_tokens, out, out_fp32, lse)
    PagedCache cache;
    const uint16_t* q;
    float kv_scale;
    float unit;                                            // scale * log2(e) * kv_scale = unit * 2^unit_exp, unit in [1, 2)
    int unit_exp, least_exp;
    int window, sink;
};

// A query row is held times 2^-e, which brings its largest value, `top`, to 2^14 .. 2^15, and its scores are the sums of
// products times unit * 2^(e + unit_exp).  That factor is neither 0 nor infinite: a masked score is -infinity, and times 0
// it would be NaN, as a score of 0 would be times infinity.  So e is not below least_exp (the row is held smaller, where
// the scores' factor is 2^-126 .. 2^-125); a factor above fp32's range is its largest.
__device__ __forceinline__ int query_exp(const PagedParams& p, float top) {
    return min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, p.least_exp), 126);
}
// -126 .. 127: the scores' factor is unit times 2 to it.
__device__ __forceinline__ int factor_exp(const PagedParams& p, int e) { return min(p.unit_exp + e, 127); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

constexpr int kDecodeBlockRows = 16;                       // query rows per block of the kernel for few of them

// A request's rows, in tiles of kRows, those that no token attends left out: the first `lo` tiles (the
// rows before `sink`), then those `base` further on; hi: tiles * kRows.
template <int kRows>
__device__ __forceinline__ TreeRequest load_paged_request(const PagedParams& p, int b) {
    TreeRequest r;
    r.d_pos = p.a.d_pos[b];
    r.n_tok = p.a.n_tokens ? min(max(p.a.n_tokens[b], 0), p.tokens) : p.tokens;
    r.base = 0;
    r.lo = r.hi = 0;
    if (r.d_pos < 0 || r.n_tok == 0) return r;
    const int end = static_cast<int>(min(static_cast<long long>(r.d_pos) + r.n_tok, static_cast<long long>(paged_rows(p.cache))));
    int tiles = (end + kRows - 1) / kRows;
    if (p.window > 0) {
        r.lo = min(p.sink / kRows + (p.sink % kRows != 0), tiles);
        const int first = min(max(max(r.d_pos - p.window + 1, 0) / kRows, r.lo), tiles);
        r.base = first - r.lo;
        tiles -= first - r.lo;
    }
    r.hi = tiles * kRows;
    return r;
}
__device__ __forceinline__ TreeRequest load_tree_request(const PagedParams& p, int b) {
    return load_paged_request<kTreeTileKeys>(p, b);
}
// Views {416 bytes, page_rows, n_pages} of the pages; boxes of min(page_rows, 32) rows.
struct PagedMaps {
    CUtensorMap codes;                                     // 64 bytes of a row, 64-byte swizzled
    CUtensorMap scales;                                    // 16 bytes
    CUtensorMap rope;                                      // 128 bytes, 128-byte swizzled
};

cudaError_t paged_decode_prepare();
cudaError_t launch_paged_decode(const PagedParams& p, bool pdl, cudaStream_t stream);
cudaError_t paged_attend_prepare();
cudaError_t launch_paged_attend(const PagedMaps& maps, const PagedParams& p, bool pdl, cudaStream_t stream);

}  // namespace mla
