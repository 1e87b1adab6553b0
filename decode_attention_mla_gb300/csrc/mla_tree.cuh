// mla_tree.cuh -- what the kernels over drafted tokens share: their parameters,
// a request's rows, and the visibility of its rows to a token.
#pragma once

#include <cstdint>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_tree.h"
#include "tc_pair_utils.cuh"

namespace mla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeTileKeys = 128;                         // cache rows per tile of a CTA pair
constexpr int kTreeBlockRows = 128;                        // (token, head) rows per CTA pair
constexpr long long kTreeMaxRow = 0x7fffff00;              // rows of a request from here on are not attended

// What a cluster leaves for the merge: its last piece is the first one of a row
// block that `pieces` consecutive clusters share (0: nothing to merge).
struct TreeMerge {
    int b, rb, pieces, rows;
};

struct TreeParams {
    mla_tree_args a;
    int batch, tokens, heads;
    int clusters;
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
    // (an offset at which no row can lie inside is as good as any other such)
    r.base = p.a.row_offset ? max(p.a.row_offset[b], -(1ll << 40)) : 0;
    r.d_pos = p.a.d_pos[b];
    r.n_tok = p.a.n_tokens ? min(max(p.a.n_tokens[b], 0), p.tokens) : p.tokens;
    const long long rows = r.d_pos < 0 ? 0 : static_cast<long long>(r.d_pos) + r.n_tok;
    const long long lo = r.base < 0 ? -r.base : 0, end = p.a.kv_rows - r.base;
    const long long hi = min(min(end, rows), kTreeMaxRow);
    // hi <= lo: none of the rows is inside (otherwise base + t fits 32 bits for
    // every t < hi, and so does the last tile's end)
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


// ---- runs of tiles -------------------------------------------------------------
// The units (request, row block, tile of cache rows), in this order, are cut into
// equal runs, one per pair of CTAs, from the lengths on the device.
struct TreeWork {                                          // a cluster's run
    long long count, per;                                  // units of the run, and of every cluster's
    TreeRequest r;                                         // its first unit
    int b, rb, tile;
};

// Quotient of non-negative numbers; 64-bit division is a slow call.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Walks the tiles of a run.  kByBlocks: one unit per row block and tile of a
// request; otherwise one per tile.
template <int kKeys, bool kByBlocks>
struct TreeCursor {
    TreeRequest r;
    int b, rb, n_rb, tile, n_tiles;
    int left;                                              // tiles of the run from here on, this one included
    int g;                                                 // tiles of the run before this one
    int item;                                              // row blocks (or parts) before this one
    bool first;                                            // first tile of its item

    static __device__ __forceinline__ int blocks_of(const TreeParams& p, const TreeRequest& r) {
        return kByBlocks ? (r.n_tok * p.heads + kTreeBlockRows - 1) / kTreeBlockRows : 1;
    }
    static __device__ __forceinline__ int tiles_of(const TreeRequest& r) { return (r.hi + kKeys - 1) / kKeys; }

    __device__ __forceinline__ void request(const TreeParams& p) {
        r = load_tree_request(p, b);
        n_rb = blocks_of(p, r);
        n_tiles = tiles_of(r);
    }
    __device__ __forceinline__ void start(const TreeParams& p, const TreeWork& w) {
        b = w.b;
        rb = w.rb;
        tile = w.tile;
        left = static_cast<int>(w.count);
        g = item = 0;
        first = true;
        r = w.r;
        n_rb = blocks_of(p, r);
        n_tiles = tiles_of(r);
    }
    __device__ __forceinline__ bool last() const { return left == 1 || tile == n_tiles - 1; }
    __device__ __forceinline__ void next(const TreeParams& p) {
        first = last();
        if (first) ++item;
        ++g;
        --left;
        if (++tile < n_tiles) return;
        tile = 0;
        if (left > 0) next_item(p);
    }
    // to the next item's first tile (b, rb, n_tiles alone; there is one)
    __device__ __forceinline__ void next_item(const TreeParams& p) {
        if (++rb < n_rb) return;
        rb = 0;
        do {
            ++b;
            request(p);
        } while (n_rb == 0 || n_tiles == 0);
    }
    // the tile holds drafted rows or rows behind them
    __device__ __forceinline__ bool special() const { return (tile + 1) * kKeys > r.d_pos; }

    // One warp: this cluster's run.  All units in order of (request, row block,
    // tile); run length = ceil(units / clusters).
    static __device__ void find_work(const TreeParams& p, int cluster, int lane, TreeWork* out) {
        auto request_of = [&](int b) {
            TreeRequest r{};
            if (b < p.batch) r = load_tree_request(p, b);
            return r;
        };
        auto units_of = [&](const TreeRequest& r) { return static_cast<long long>(blocks_of(p, r)) * tiles_of(r); };
        TreeRequest r = request_of(lane);                      // requests 0 .. 31 stay in registers
        long long total = units_of(r);
        for (int b0 = 32; b0 < p.batch; b0 += 32) total += units_of(request_of(b0 + lane));
        if (p.batch > 1) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        } else {
            total = __shfl_sync(0xffffffffu, total, 0);
        }
        long long per = quotient(total + p.clusters - 1, p.clusters);
        if (per < 1) per = 1;
        const long long u0 = per * cluster;
        const long long count = u0 >= total ? 0 : (total - u0 < per ? total - u0 : per);
        if (lane == 0) {
            out->per = per;
            out->count = count;
        }
        long long before = 0;
        for (int b0 = 0; b0 < p.batch && count > 0; b0 += 32) {
            if (b0 > 0) r = request_of(b0 + lane);
            const long long u = units_of(r);
            long long incl = u;
            if (p.batch > 1) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
            }
            const long long first = before + incl - u;         // this lane's request is units [first, first + u)
            const bool here = u0 >= first && u0 < first + u;
            if (here) {
                const int n_tiles = tiles_of(r);
                out->rb = static_cast<int>(quotient(u0 - first, n_tiles));
                out->tile = static_cast<int>(u0 - first - static_cast<long long>(out->rb) * n_tiles);
                out->b = b0 + lane;
                out->r = r;
            }
            if (__any_sync(0xffffffffu, here)) break;
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
};

// ---- waits -----------------------------------------------------------------------
// Tell both CTAs of the pair to leave their loops (neither exits before both
// have reached the closing cluster barrier).
__device__ __forceinline__ void raise_tree_error(int* abort_flag, int* status) {
    st_cluster_s32(map_to_rank(abort_flag, 0), 1);
    st_cluster_s32(map_to_rank(abort_flag, 1), 1);
    if (status) atomicCAS(status, 0, static_cast<int>(MLA_EDEVICE));
}
// Bounded wait whose usual case (the phase is over) is one instruction inline.
static __device__ __noinline__ bool wait_slowly(uint64_t* bar, uint32_t parity, int* abort_flag) {
    return mbar_wait_bounded(bar, parity, abort_flag);
}
// By a whole warp (every thread polls: with one lane polling for the others each
// hand-off took longer), with one answer for all of its lanes.
__device__ __forceinline__ bool warp_wait(int* abort_flag, uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_slowly(bar, parity, abort_flag));
    tc_fence_after_sync();
    return ok;
}

// ---- launches ----------------------------------------------------------------------
struct TreeMaps {                                          // boxes of 64-column chunks, 128-byte swizzled
    CUtensorMap kv;                                        // attention: cache, 64 rows x 2 chunks
    CUtensorMap rope;                                      // attention: cache, 64 rows x 1 chunk
    CUtensorMap k;                                         // weights: cache, 128 rows x 1 chunk
    CUtensorMap q;                                         // attention: queries, 64 rows x 9 chunks; weights: x 1
};
cudaError_t tree_attend_prepare();
cudaError_t launch_tree_attend(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream);
cudaError_t tree_weights_prepare();
cudaError_t launch_tree_weights(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream);

}  // namespace mla
