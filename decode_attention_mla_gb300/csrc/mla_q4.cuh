// mla_q4.cuh -- rows of the 4-bit cache (include/mla_paged.h): their places and
// the widening of their values.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "mla_internal.h"
#include "mla_paged.h"

namespace mla {

constexpr int kQ4Scales = kDLatent / 2;                    // byte of the first scale
constexpr int kQ4Rope = kQ4Scales + kDLatent / MLA_Q4_BLOCK;   // ... of the key values
static_assert(kQ4Rope + 2 * kDRope == MLA_Q4_ROW, "a row's parts");

// A call's pages: rows are found by shifts.
struct PagedCache {
    uint8_t* pages;
    long long page_stride;
    const int* table;
    int n_pages, columns;
    int row_shift;                                         // log2(page_rows)
};

// Number of the page that row t >= 0 of request b lies in, or -1.
__device__ __forceinline__ int page_of(const PagedCache& c, int b, int t) {
    const int column = t >> c.row_shift;
    if (column >= c.columns) return -1;
    const int page = c.table[static_cast<long long>(b) * c.columns + column];
    return page >= 0 && page < c.n_pages ? page : -1;
}
// Place of row t in a page.
__device__ __forceinline__ uint8_t* row_in(const PagedCache& c, int page, int t) {
    return c.pages + page * c.page_stride + (t & ((1 << c.row_shift) - 1)) * MLA_Q4_ROW;
}
// The first row behind the table.
__device__ __forceinline__ int paged_rows(const PagedCache& c) { return c.columns << c.row_shift; }

// Eight codes as f16 pairs: out[i] = features 2 i, 2 i + 1.
__device__ __forceinline__ void widen_e2m1(uint32_t w, uint32_t (&out)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}
// Two E4M3 bytes as f16, exact.
__device__ __forceinline__ uint32_t widen_e4m3(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Host: the cache's fields as the kernels take them, checked.
int check_cache(const mla_paged_cache* c);
int encode_q4_boxes(CUtensorMap* map, const mla_paged_cache* c, uint32_t box_bytes, CUtensorMapSwizzle swizzle);
PagedCache paged_cache(const mla_paged_cache* c);

}  // namespace mla
