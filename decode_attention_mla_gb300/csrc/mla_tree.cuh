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
constexpr int kTreePieceRate = 14;                         // pieces written and merged in a tile's time ...
constexpr int kTreeFewPieces = 16;                         // ... fewer cost next to nothing
constexpr int kTreeCutTiles = 96;                          // tiles per run from which row blocks are cut
constexpr long long kTreeMaxRow = 0x7fffff00;              // rows of a request from here on are not attended

// Pieces that a cluster's run can leave: the run's first item, its last one, and at
// most one between them (see TreeSegments).
constexpr int kTreePieces = 3;
// Note of a piece that opens a row block shared by several runs.
struct __align__(16) TreeMerge {
    int b, rb;
    int rows;                                              // of the row block; the piece's place in its run << 16
    int pieces;                                            // the piece and the first ones of the runs behind it
                                                           // (0: no note, -1: in segments, see TreeCut)
};
struct __align__(16) TreeCut {
    int n_rb, n_tiles, per;                                // as in the cursor
    int begin;                                             // the request's first unit, relative to the run's
};

struct TreeParams {
    mla_tree_args a;
    int batch, tokens, heads;
    int q_tail;                                            // tokens * heads mod 64, rounded up to 8 (64: no rest)
    int clusters;
    int block_rows;                                        // query rows per block: kTreeBlockRows, or what a kernel that
                                                           // leaves pieces of fewer takes
    float scale_log2;                                      // scale * log2(e): scores in base-2 units
    float* part;                                           // fp32 [clusters][3][128 x 512], normalised, by feature quads
    float* lse_part;                                       // fp32 [clusters][3][128], base 2
    TreeMerge* merge;                                      // [3][clusters] (without segments the first row alone)
    TreeCut* cut;                                          // [3][clusters]
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
// A request's work is a list of jobs, in units of a tile: its row blocks (over all
// of its cache), one after the other.  All requests' units, in order, are cut into
// equal runs, one per pair of CTAs, from the lengths on the device.
//
// The row blocks of a request read the same cache rows, at about the same time
// if run lengths and cache lengths happen to fit; otherwise, with more cache than L2
// holds, each reads them from DRAM again (16 requests of 5 row blocks: 1.35 GB for
// 0.38 GB of rows; 0.61 in the order below).  Hence
//   - tiles go by the clock: a job done whole by one run starts at the tile that it
//     would have reached if it had begun with the run, and goes round; of a job cut
//     between two runs, the first takes the far tiles, so that the second begins
//     at the near ones with the others.  At any time the pairs of a request then
//     are at one of two places;
//   - row blocks longer than a run are cut into segments of a run's length, and the
//     jobs are (segment, row block).  The last one or two segments are 0.5 to 1.25
//     runs long, so that a run has at most one whole job between its first and its
//     last item, and a job is in three runs at most.
// Measured (5 tokens x 128 heads): 16 requests of 4096 .. 32768 rows 285 -> 262 us,
// by the clock alone; one of 300000 rows 330 -> 316 by the clock, 279 with
// segments.  Segments leave more pieces to merge: with runs of 14 tiles (8 requests
// of 16384 rows, 16 x 16) 48 us where uncut row blocks take 43, with 120 tiles 203
// and 205 us, so they are made from kTreeCutTiles per run on.
struct TreeSegments {
    int full, len, a, b;                                   // `full` segments of len tiles, one of a, one of b (0: none)

    __device__ __forceinline__ void set(int n_tiles, int n_rb, int seg_tiles) {
        full = 0;
        len = seg_tiles;
        a = n_tiles;
        b = 0;
        if (n_rb > 1 && n_tiles > seg_tiles) {
            full = n_tiles / seg_tiles - 1;
            const int rest = n_tiles - full * seg_tiles;   // one length or more, below two
            a = rest - seg_tiles <= seg_tiles / 4 ? rest : (rest + 1) / 2;
            b = rest - a;
        }
    }
    __device__ __forceinline__ int count() const { return full + (b > 0 ? 2 : 1); }
    __device__ __forceinline__ int start(int seg) const { return seg <= full ? seg * len : full * len + a; }
    __device__ __forceinline__ int tiles(int seg) const { return seg < full ? len : seg == full ? a : b; }
};

struct TreeWork {                                          // a cluster's run
    long long count, per;                                  // units of the run, and of every cluster's
    TreeRequest r;                                         // of its first unit
    int b, seg, rb, at;                                    // the first unit's job, and its place in it
    int begin;                                             // the request's first unit, relative to the run's
    int seg_tiles;                                         // tiles per segment
};

// Quotient of non-negative numbers; 64-bit division is a slow call.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Walks the tiles of a run.  kByBlocks: a request's jobs are its row blocks;
// otherwise it has one job, its tiles.  An item is what one run does of a job.
// Params: TreeParams, or what is derived from it with a load_tree_request of its own.
template <int kKeys, bool kByBlocks, class Params = TreeParams>
struct TreeCursor {
    TreeRequest r;
    TreeSegments sg;
    int b, seg, rb, n_rb, n_tiles, seg_tiles;
    int begin;                                             // place of the request's first unit in the run (may be < 0)
    int tile, lo, hi;                                      // the item's tiles, and the one at hand
    int item_left;                                         // tiles of the item from here on, this one included
    int left;                                              // ... of the run
    int g;                                                 // tiles of the run before this one
    int item;                                              // items before this one
    bool first;                                            // first tile of its item

    static __device__ __forceinline__ int blocks_of(const Params& p, const TreeRequest& r) {
        return kByBlocks ? (r.n_tok * p.heads + kTreeBlockRows - 1) / kTreeBlockRows : 1;
    }
    static __device__ __forceinline__ int tiles_of(const TreeRequest& r) { return (r.hi + kKeys - 1) / kKeys; }

    __device__ __forceinline__ void request(const Params& p) {
        n_rb = blocks_of(p, r);
        n_tiles = tiles_of(r);
        if constexpr (kByBlocks)
            sg.set(n_tiles, n_rb, seg_tiles);
        else
            sg = TreeSegments{0, 0, n_tiles, 0};
    }
    // the item that begins with unit `at` of the job
    __device__ __forceinline__ void enter(int at) {
        const int len = sg.tiles(seg);
        item_left = min(len - at, left);
        // (of a cut row block the first run takes the far tiles)
        lo = sg.start(seg) + (kByBlocks ? len - at - item_left : at);
        hi = lo + item_left;
        tile = kByBlocks && g > 0 && item_left == len ? lo + g % len : lo;
    }
    __device__ __forceinline__ void start(const Params& p, const TreeWork& w) {
        b = w.b;
        seg = w.seg;
        rb = w.rb;
        seg_tiles = w.seg_tiles;
        begin = w.begin;
        left = static_cast<int>(w.count);
        g = item = 0;
        first = true;
        r = w.r;
        request(p);
        enter(w.at);
    }
    __device__ __forceinline__ bool last() const { return item_left == 1; }
    // the item has its job's first unit; is all of the request's tiles
    __device__ __forceinline__ bool opens() const { return hi == sg.start(seg) + sg.tiles(seg); }
    __device__ __forceinline__ bool whole() const { return hi - lo == n_tiles; }
    __device__ __forceinline__ void next(const Params& p) {
        ++g;
        --left;
        first = --item_left == 0;
        if (!first) {
            if (++tile == hi) tile = lo;
            return;
        }
        ++item;
        if (left > 0) next_item(p);
    }
    // to the next item's first tile, the g-th of the run (there is one)
    __device__ __forceinline__ void next_item(const Params& p) {
        if (++rb == n_rb) {
            rb = 0;
            if (++seg == sg.count()) {
                seg = 0;
                do {
                    r = load_tree_request(p, ++b);
                    request(p);
                } while (n_rb == 0 || n_tiles == 0);
                begin = g;
            }
        }
        enter(0);
    }
    // the tile holds drafted rows or rows behind them
    __device__ __forceinline__ bool special() const { return (tile + 1) * kKeys > r.d_pos; }

    // Whether row blocks go whole into the run that their first unit falls into: some runs
    // then are longer, but no pieces are written and merged.  (64 x 128 rows over 4096: 32
    // tiles for 27, 56 us for 63; 64 requests of 1 x 128 over 4000 70 for 83; 16 of 8 x 128
    // over 500 .. 1400 47 for 57; but 8 of 4 x 64 over 1000, 8 tiles for 2, 20 for 17.)
    // `longest`, `alike`: of the lengths of the first 32 requests.
    static __device__ __forceinline__ bool keep_whole(const Params& p, const TreeRequest& r, int longest,
                                                      bool alike, int lane, uint32_t total, uint32_t per) {
        uint32_t blocks = r.hi > 0 ? blocks_of(p, r) : 0;
        if (p.batch > 1) {
            const int first = longest;
            for (int b = 32 + lane; b < p.batch; b += 32) {
                const TreeRequest next = load_tree_request(p, b);
                const int n = next.hi > 0 ? blocks_of(p, next) : 0;
                blocks += n;
                alike &= n == 0 || tiles_of(next) == first;
                longest = max(longest, n == 0 ? 0 : tiles_of(next));
            }
            longest = __reduce_max_sync(0xffffffffu, longest);
            alike = __all_sync(0xffffffffu, alike);
            blocks = __reduce_add_sync(0xffffffffu, blocks);
        }
        const uint32_t more = alike ? (per + longest - 1) / longest * longest - per : longest - 1;
        if (more > 1 + 2u * p.clusters / kTreePieceRate) return false;
        // pieces: one per run and one more where a run ends inside a block, two at most
        const uint32_t runs = total / per;
        const uint32_t pieces = min(runs + (alike && longest % per == 0 ? 0 : blocks), 2 * runs);
        return pieces >= kTreeFewPieces && more <= 1 + pieces / kTreePieceRate;
    }

    // The run of the row blocks whose first unit lies in [u0, u1).
    static __device__ __forceinline__ void find_whole(const Params& p, TreeRequest r, bool one, long long u0,
                                                      long long u1, long long total, int lane, TreeWork* out) {
        long long before = 0, s0 = -1, s1 = total;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            if (b0 > 0) r = b0 + lane < p.batch ? load_tree_request(p, b0 + lane) : TreeRequest{};
            const int len = max(tiles_of(r), 1), n_rb = r.hi > 0 ? blocks_of(p, r) : 0;
            const long long u = static_cast<long long>(n_rb) * len;
            long long incl = u;
            if (!one) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
            }
            const long long first = before + incl - u;
            // this lane's request's first block that begins at or behind a unit
            auto block = [&](long long at) { return at <= first ? 0ll : quotient(at - first + len - 1, len); };
            const long long j0 = block(u0), j1 = block(u1);
            const bool mine = lane == 0 || !one;
            const uint32_t has0 = __ballot_sync(0xffffffffu, mine && j0 < n_rb);
            const uint32_t has1 = __ballot_sync(0xffffffffu, mine && j1 < n_rb);
            if (s0 < 0 && has0 != 0) {
                const int src = __ffs(has0) - 1;
                s0 = __shfl_sync(0xffffffffu, first + j0 * len, src);
                if (lane == src) {
                    out->b = b0 + lane;
                    out->r = r;
                    out->seg = out->at = 0;
                    out->rb = static_cast<int>(j0);
                    out->begin = static_cast<int>(first - s0);
                }
            }
            if (has1 != 0) {
                s1 = __shfl_sync(0xffffffffu, first + j1 * len, __ffs(has1) - 1);
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            out->count = s0 < 0 ? 0 : s1 - s0;
            out->seg_tiles = static_cast<int>(kTreeMaxRow);
        }
    }

    // One warp: this cluster's run; run length = ceil(units / clusters).
    static __device__ void find_work(const Params& p, int cluster, int lane, TreeWork* out) {
        auto request_of = [&](int b) {
            TreeRequest r{};
            if (b < p.batch) r = load_tree_request(p, b);
            return r;
        };
        auto units_of = [&](const TreeRequest& r) { return static_cast<long long>(blocks_of(p, r)) * tiles_of(r); };
        const bool one = p.batch == 1;                         // every lane has the one request
        TreeRequest r = request_of(one ? 0 : lane);            // requests 0 .. 31 stay in registers
        long long total = units_of(r);
        for (int b0 = 32; b0 < p.batch; b0 += 32) total += units_of(request_of(b0 + lane));
        if (!one) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        long long per = quotient(total + p.clusters - 1, p.clusters);
        if (per < 1) per = 1;
        bool whole = false;
        if (kByBlocks && total >= kTreeFewPieces && total < kTreeMaxRow) {
            const int own = units_of(r) > 0 ? tiles_of(r) : 0;
            const int longest = one ? own : __reduce_max_sync(0xffffffffu, own);
            const bool alike = one || __all_sync(0xffffffffu, own == 0 || own == longest);
            if (longest > 0 && (alike || longest <= 2 + 2 * p.clusters / kTreePieceRate))
                whole = keep_whole(p, r, longest, alike, lane, static_cast<uint32_t>(total), static_cast<uint32_t>(per));
        }
        const long long u0 = per * cluster;
        const long long count = u0 >= total ? 0 : (total - u0 < per ? total - u0 : per);
        const int seg_tiles = static_cast<int>(kByBlocks && per >= kTreeCutTiles ? min(per, kTreeMaxRow) : kTreeMaxRow);
        if (lane == 0) {
            out->per = per;
            out->count = count;
            out->seg_tiles = seg_tiles;
        }
        if (whole) {
            find_whole(p, r, one, u0, u0 + per, total, lane, out);
            return;
        }
        long long before = 0;
        for (int b0 = 0; b0 < p.batch && count > 0; b0 += 32) {
            if (b0 > 0) r = request_of(b0 + lane);
            const long long u = units_of(r);
            long long incl = u;
            if (!one) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
            }
            const long long first = before + incl - u;         // this lane's request is units [first, first + u)
            const bool here = u0 >= first && u0 < first + u && (lane == 0 || !one);
            if (here) {
                const int n_tiles = tiles_of(r), n_rb = blocks_of(p, r);
                TreeSegments sg;
                sg.set(n_tiles, n_rb, seg_tiles);
                long long at = u0 - first;                     // in the request, then in the segment
                int seg = 0;
                if (sg.full > 0) {
                    const long long each = static_cast<long long>(n_rb) * seg_tiles;
                    seg = static_cast<int>(min(quotient(at, each), static_cast<long long>(sg.full)));
                    at -= seg * each;
                }
                if (seg == sg.full && sg.b > 0 && at >= static_cast<long long>(n_rb) * sg.a) {
                    at -= static_cast<long long>(n_rb) * sg.a;
                    ++seg;
                }
                out->rb = static_cast<int>(quotient(at, sg.tiles(seg)));
                out->at = static_cast<int>(at - static_cast<long long>(out->rb) * sg.tiles(seg));
                out->seg = seg;
                out->begin = static_cast<int>(first - u0);
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
    CUtensorMap q_tail;                                    // queries, q_tail rows x 1 chunk
};

// Of the 64 query rows from `row` on, how many are loaded: those in the tensor, if boxes
// of q_tail rows make them up, and otherwise all.  (Rows that TMA fills with zeros cost
// nothing in one CTA, but 5 us where all of them ask for some at once: one token of 16
// heads over 16384 rows 22 us, without such rows 17.)  Rows that are not loaded hold
// anything; they are dead, and no row's result depends on another's.
__device__ __forceinline__ int query_rows(const TreeParams& p, int row) {
    const int there = min(max((p.batch * p.tokens * p.heads - row + 7) & ~7, 0), 64);
    return there % p.q_tail == 0 ? there : 64;
}
// `n` of them: kQChunks 64-column chunks from `chunk` on.
template <int kQChunks>
__device__ __forceinline__ void load_query_rows(uint8_t* dst, const TreeMaps& maps, int row, int n, int tail, int chunk,
                                                uint32_t bar, uint64_t policy) {
    if (n == 64) {
        tma_load_3d_pair(dst, &maps.q, 0, row, chunk, bar, policy);
        return;
    }
    for (int i = 0; i < n; i += tail)
#pragma unroll
        for (int k = 0; k < kQChunks; ++k)
            tma_load_3d_pair(dst + k * 8192 + i * 128, &maps.q_tail, 0, row + i, chunk + k, bar, policy);
}
cudaError_t tree_attend_prepare();
cudaError_t launch_tree_attend(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream);
// The pieces of row blocks that several runs share, joined.
cudaError_t launch_tree_merge(const TreeParams& p, bool pdl, cudaStream_t stream);
cudaError_t tree_weights_prepare();
cudaError_t launch_tree_weights(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream);

}  // namespace mla
