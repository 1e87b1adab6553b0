// mla_pages.cu -- the pages of a cache: forked, copied, reserved, freed and
// compacted on the device (include/mla_paged.h).
//
// fork.  A page's references follow from the new tables alone, so there is no list of
// free pages to keep: refs are counted anew, and the free pages are those without
// any.  Three launches: clear; every request's entries, counted with atomics (sums and
// minima of integers: the same in any order), by whose last block the pages are handed
// out (one block: its scan of refs ends as soon as it has found enough free pages);
// then the tables written and the shared last pages copied.  The new table waits in
// scratch, since a request's row may be another's parent.  Smaller forks are one block's.
//
// compact.  The k-th page in use behind the front goes to the k-th hole in it.  Pools of up to
// kBitsPages pages take one launch: every block counts all of them itself, which costs it
// less than a launch whose counts it would wait for (512 pages 4.3 us for 8.7, 65536
// 9.9 for 13.7); references in place take a second.  Larger pools, three: counts
// per 4096 pages; lists of holes and moving pages; moves, tables and references.
//
// Bound: bytes (tables and references, and the rows that are copied), below that the
// launches, each a chain of a few loads.  256 requests with 65300 entries, a pool of 65536: 13.8 us.
// 7700 pages of 26 KB moved by bulk copies: 74 us, 5.6 TB/s (by loads and stores of a thread's own, 82).
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_paged.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kPlaceThreads = 1024;
constexpr int kMostRequests = 4096;
constexpr int kChunk = 4096;                               // pages per block of the counts
constexpr int kNobody = 0x7fffffff;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct ForkParams {
    mla_pages_fork_args a;
    int shift;                                             // log2(page_rows)
    int blocks;                                            // of the counting launch
    int* table;                                            // [B][columns] the new table
    int* keeper;                                           // [n_pages] first request that ends in the page
    int* rows;                                             // [B] n
    int* src;                                              // [B] page to copy, or -1
    int* dst;                                              // [B]
    int* free;                                             // pages taken, in order
    int* ticket;
};

// Request b's parent (-1: it ends).
__device__ __forceinline__ int fork_parent(const ForkParams& p, int b) {
    const int parent = p.a.parent ? p.a.parent[b] : b;
    return parent >= 0 && parent < p.a.batch ? parent : -1;
}
// n rows, by a request's entries, or their full pages' where the page that they end in is missing.  (Not inlined: forks
// without a window do not call it, and four beams took 6.9 us for 6.7 with its code among theirs.)
__device__ __noinline__ int without_missing(const int* entries, int n_pages, int n, int shift) {
    const int part = n & ((1 << shift) - 1);
    return part && static_cast<unsigned>(entries[n >> shift]) >= static_cast<unsigned>(n_pages) ? n - part : n;
}
// Rows that request b goes on with.  Where they end in a page that is missing, the rows of that page are not there, and n
// falls to the full pages before it: here with a window, since n says what a window gives back, else in fork_place (one look-up
// less in a row).
__device__ __forceinline__ int fork_rows(const ForkParams& p, int b, int parent) {
    if (parent < 0) return 0;
    const int d = max(p.a.d_pos[parent], 0);
    const int n = min(min(d, p.a.rows ? max(p.a.rows[b], 0) : d), p.a.columns << p.shift);
    return p.a.window > 0 ? without_missing(p.a.page_table + static_cast<long long>(parent) * p.a.columns, p.a.n_pages, n, p.shift) : n;
}
// Column behind the last one that request b reserves, n rows kept.
__device__ __forceinline__ int fork_end(const ForkParams& p, int n) {
    const long long rows = static_cast<long long>(n) + p.a.reserve + (1 << p.shift) - 1;
    return static_cast<int>(min(rows >> p.shift, static_cast<long long>(p.a.columns)));
}

__global__ void __launch_bounds__(kThreads) mla_fork_clear_kernel(const __grid_constant__ ForkParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.a.n_pages; i += gridDim.x * kThreads) {
        p.a.refs[i] = 0;
        p.keeper[i] = kNobody;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
}

// Inclusive sum over the block; `total`: of all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();                                       // (the sums of the scan before have been read)
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return v + before;
}

// Hand out pages (one block).  All of its threads have passed a barrier behind the counts, which other blocks have made
// (kShared: this one, in its shared memory).
template <bool kShared>
__device__ __forceinline__ int counted(const int* at) {
    return kShared ? *at : __ldcg(at);
}
template <bool kShared>
__device__ void fork_place(const ForkParams& p) {
    __shared__ int sums[32];
    struct Request {
        int n, end;                                        // rows, column behind those reserved
        int page;                                          // that n ends in, or -1
        bool copied;                                       // it is not this request's to keep
        int at;                                            // its first page among those taken
    } mine[kMostRequests / kPlaceThreads];
    const int batch = p.a.batch, columns = p.a.columns, rows_mask = (1 << p.shift) - 1;
    // ---- what each request needs: a copy of its last page, pages behind it
    int needed = 0;
#pragma unroll 1
    for (int q = 0; q * kPlaceThreads < batch; ++q) {
        const int b = q * kPlaceThreads + threadIdx.x;
        Request r{0, 0, -1, false, 0};
        if (b < batch) {
            const bool goes_on = fork_parent(p, b) >= 0;
            r.n = counted<kShared>(p.rows + b);
            if (r.n & rows_mask) {
                r.page = counted<kShared>(p.table + static_cast<long long>(b) * columns + (r.n >> p.shift));
                if (r.page >= 0)
                    r.copied = counted<kShared>(p.a.refs + r.page) > 0 || counted<kShared>(p.keeper + r.page) != b;
                else
                    r.n &= ~rows_mask;
            }
            if (goes_on) r.end = fork_end(p, r.n);
            p.src[b] = r.copied ? r.page : -1;
        }
        const int need = max(0, r.end - (r.n >> p.shift)) - (r.page >= 0 && !r.copied);
        int total;
        r.at = needed + block_scan(need, sums, total) - need;
        needed += total;
        mine[q] = r;
    }
    // ---- last pages that stay  (all have looked at the references)
#pragma unroll 1
    for (int q = 0; q * kPlaceThreads + static_cast<int>(threadIdx.x) < batch; ++q)
        if (mine[q].page >= 0 && !mine[q].copied) p.a.refs[mine[q].page] = 1;
    __syncthreads();
    // ---- the first free pages
    int found = 0;
    for (int i0 = 0; i0 < p.a.n_pages && found < needed; i0 += 4 * kPlaceThreads) {
        const int i = i0 + 4 * threadIdx.x;
        bool is[4];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            is[k] = i + k < p.a.n_pages && counted<kShared>(p.a.refs + i + k) == 0;
            mine += is[k];
        }
        int total;
        int at = found + block_scan(mine, sums, total) - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (is[k]) {
                if (at < needed) p.free[at] = i + k;
                ++at;
            }
        found += total;
    }
    const int have = min(found, needed);
    __syncthreads();
    // ---- and who gets them
#pragma unroll 1
    for (int q = 0; q * kPlaceThreads + static_cast<int>(threadIdx.x) < batch; ++q) {
        const int b = q * kPlaceThreads + threadIdx.x;
        const Request r = mine[q];
        const int last = r.n >> p.shift;
        int* row = p.table + static_cast<long long>(b) * columns;
        int at = r.at, to = -1, rows = r.n;
        for (int c = last + (r.page >= 0 && !r.copied); c < r.end; ++c) {
            const int page = at < have ? p.free[at] : -1;
            ++at;
            if (page >= 0) p.a.refs[page] = 1;
            row[c] = page;
            if (c == last && r.copied) {
                to = page;
                if (page < 0) rows = r.n & ~rows_mask;
            }
        }
        p.dst[b] = to;
        p.rows[b] = rows;
    }
    if (threadIdx.x == 0) *p.a.missing = needed - have;
}

// Entry c of request b, which has n rows of its parent's: the page, or -1.
__device__ __forceinline__ int fork_page(const ForkParams& p, int c, int parent, int n) {
    const long long t0 = static_cast<long long>(c) << p.shift, t1 = t0 + (1 << p.shift);
    // (no later token attends rows up to n - window)
    if (t0 >= n || (p.a.window > 0 && t0 >= p.a.sink && t1 <= static_cast<long long>(n) + 1 - p.a.window)) return -1;
    const int page = p.a.page_table[static_cast<long long>(parent) * p.a.columns + c];
    return page >= p.a.n_pages ? -1 : max(page, -1);
}
// ... into the new table, and counted.
__device__ __forceinline__ void fork_entry(const ForkParams& p, int b, int c, int page, int n) {
    if (page >= 0) {
        if ((static_cast<long long>(c) + 1) << p.shift <= n)
            atomicAdd(p.a.refs + page, 1);
        else
            atomicMin(p.keeper + page, b);
    }
    p.table[static_cast<long long>(b) * p.a.columns + c] = page;
}

// A request's entries, kThreads * 4 columns a block; the last block hands out pages.
__global__ void __launch_bounds__(kPlaceThreads) mla_fork_count_kernel(const __grid_constant__ ForkParams p) {
    __shared__ int is_last;
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.y;
    const int parent = fork_parent(p, b), n = fork_rows(p, b, parent);
    for (int c = blockIdx.x * kPlaceThreads + threadIdx.x; c < p.a.columns; c += gridDim.x * kPlaceThreads)
        fork_entry(p, b, c, fork_page(p, c, parent, n), n);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.rows[b] = n;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) is_last = atomicAdd(p.ticket, 1) == p.blocks - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    fork_place<false>(p);
}

// Eight loads a thread on their way; thread `at` of `threads`.
__device__ __forceinline__ void copy_units(uint4* dst, const uint4* src, int units, int at, int threads) {
    for (int i = at; i < units; i += 8 * threads) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k * threads < units) v[k] = src[i + k * threads];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k * threads < units) dst[i + k * threads] = v[k];
    }
}
// Request b's copied page, if it has one.
__device__ __forceinline__ void fork_copy(const ForkParams& p, int b, int at, int threads) {
    const int n = p.rows[b], from = p.src[b], to = p.dst[b];
    if (to < 0) return;
    char* pages = static_cast<char*>(p.a.pages);
    const int rows = n & ((1 << p.shift) - 1);
    copy_units(reinterpret_cast<uint4*>(pages + to * p.a.page_stride),
               reinterpret_cast<const uint4*>(pages + from * p.a.page_stride),
               rows * (p.a.row_bytes / 16), at, threads);
}

// A block per request: its table, its rows, its copied page.
__global__ void __launch_bounds__(kThreads) mla_fork_write_kernel(const __grid_constant__ ForkParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x;
    const long long row = static_cast<long long>(b) * p.a.columns;
    for (int c = threadIdx.x; c < p.a.columns; c += kThreads) p.a.page_table_out[row + c] = p.table[row + c];
    if (threadIdx.x == 0) p.a.d_pos_out[b] = p.rows[b];
    fork_copy(p, b, threadIdx.x, kThreads);
}

// All of it in one block, counted in shared memory, but for large copies, which take a second launch.  Measured
// against the three launches, us (requests x columns, pages of the pool): 4.4 and 7.8 (1 x 40, 512), 8.4 and 10.5 (32 x 64,
// 2048), 9.6 and 13.1 (2 x 4096, 8192), 11.2 and 14.1 (4 x 3000, 12000); but 12.1 and 9.7 (200 x 100, 1000).
constexpr int kBlockBytes = 192 << 10, kBlockEntries = 16384, kOwnCopies = 128 << 10;
long long fork_block_bytes(const mla_pages_fork_args& a) {
    return 12ll * a.n_pages + 4ll * a.batch * a.columns + 12ll * a.batch;
}
template <bool kCopies>
__global__ void __launch_bounds__(kPlaceThreads) mla_fork_block_kernel(const __grid_constant__ ForkParams args) {
    extern __shared__ __align__(16) int smem[];
    constexpr int kAhead = 4;
    const int entries = args.a.batch * args.a.columns, batch = args.a.batch, columns = args.a.columns;
    ForkParams p = args;
    p.a.refs = smem;
    p.keeper = p.a.refs + p.a.n_pages;
    p.free = p.keeper + p.a.n_pages;
    p.table = p.free + p.a.n_pages;
    p.rows = p.table + entries;
    p.src = p.rows + batch;
    p.dst = p.src + batch;
    for (int i = threadIdx.x; i < p.a.n_pages; i += kPlaceThreads) {
        p.a.refs[i] = 0;
        p.keeper[i] = kNobody;
    }
    grid_dependency_wait();
    allow_dependent_launch();
    for (int b = threadIdx.x; b < batch; b += kPlaceThreads) {
        const int parent = fork_parent(p, b);
        p.dst[b] = parent;                                 // (so far)
        p.rows[b] = fork_rows(p, b, parent);
    }
    __syncthreads();
    for (int e0 = threadIdx.x; e0 < entries; e0 += kAhead * kPlaceThreads) {
        int page[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int e = e0 + k * kPlaceThreads, b = e / columns;
            page[k] = e < entries ? fork_page(p, e - b * columns, p.dst[b], p.rows[b]) : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int e = e0 + k * kPlaceThreads, b = e / columns;
            if (e < entries) fork_entry(p, b, e - b * columns, page[k], p.rows[b]);
        }
    }
    __syncthreads();
    fork_place<true>(p);
    __syncthreads();
    for (int e = threadIdx.x; e < entries; e += kPlaceThreads) p.a.page_table_out[e] = p.table[e];
    for (int i = threadIdx.x; i < p.a.n_pages; i += kPlaceThreads) args.a.refs[i] = p.a.refs[i];
    for (int b = threadIdx.x; b < batch; b += kPlaceThreads) {
        p.a.d_pos_out[b] = p.rows[b];
        if (!kCopies) {
            args.rows[b] = p.rows[b];
            args.src[b] = p.src[b];
            args.dst[b] = p.dst[b];
        }
    }
    // copies, kThreads threads a request
    if (kCopies)
        for (int b = threadIdx.x / kThreads; b < batch; b += kPlaceThreads / kThreads)
            fork_copy(p, b, threadIdx.x % kThreads, kThreads);
}
__global__ void __launch_bounds__(kThreads) mla_fork_copy_kernel(const __grid_constant__ ForkParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    fork_copy(p, blockIdx.x, threadIdx.x, kThreads);
}

// ---- compact --------------------------------------------------------------------
struct CompactParams {
    mla_pages_compact_args a;
    int chunks;
    int* counts;                                           // [chunks] pages in use
    int* place;                                            // [n_pages] -1: not in use; its rank among the moving
                                                           // pages, if it moves
    int* hole;                                             // [..] by rank: page to fill
    int* mover;                                            // ... and the page that goes there
    int* mover_refs;                                       // ... and its references
    int* moves;                                            // number of them; of pages in use
    uint32_t* bits;                                        // kept for the references in place: which pages are in use
};

// Whole pages moved by bulk copies through shared memory: one warp keeps kPartsAhead parts of pages on their way in and the
// rest of the ring on its way out.
constexpr int kPartBytes = 16384, kParts = 12, kPartsAhead = 7;
constexpr int kMoveThreads = 1024;
struct __align__(128) MoveRing {
    uint8_t part[kParts][kPartBytes];
    uint64_t full[kParts];
    char* to[kParts];
    int bytes[kParts];
};

__device__ __forceinline__ void bulk_copy_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void init_ring(MoveRing& r) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < kParts; ++i) mbar_init(&r.full[i], 1);
        mbar_init_fence();
    }
    __syncthreads();
}
// One warp.  places(k, from, to): the k-th moving page and where it goes.  A copy that does not arrive: `used` is -1.
template <class Places>
__device__ void move_pages(const CompactParams& p, MoveRing& r, int moves, int lane, const Places& places) {
    char* pages = static_cast<char*>(p.a.pages);
    const int page = p.a.page_rows * p.a.row_bytes, per = (page + kPartBytes - 1) / kPartBytes;
    const long long all = static_cast<long long>(moves) * per, first = blockIdx.x, step = gridDim.x;
    const long long mine = first < all ? (all - first + step - 1) / step : 0;
    const uint64_t policy = l2_policy_evict_first();
    volatile int never = 0;
    bool ok = true;
    int in = 0, out = 0;                                   // ring slots of the next part in and out
    uint32_t phase = 0;                                    // of `out`
    auto send = [&] {
        const bool there = mbar_wait_bounded(&r.full[out], phase, &never);
        if (there) bulk_copy_s2g(r.to[out], r.part[out], r.bytes[out]);
        if (++out == kParts) {
            out = 0;
            phase ^= 1;
        }
        return there;
    };
    for (long long base = 0; base < mine && ok; base += 32) {
        int from = 0, to = 0, offset = 0;
        if (base + lane < mine) {
            const long long t = first + (base + lane) * step;
            const int k = static_cast<int>(t / per);
            offset = static_cast<int>(t - static_cast<long long>(k) * per) * kPartBytes;
            places(k, from, to);
        }
        const int n = static_cast<int>(min(mine - base, 32ll));
        for (int j = 0; j < n; ++j) {
            const int f = __shfl_sync(0xffffffffu, from, j), t = __shfl_sync(0xffffffffu, to, j);
            const int o = __shfl_sync(0xffffffffu, offset, j);
            if (lane == 0 && ok) {
                if (base + j >= kPartsAhead) ok = send();
                // the part that was in this slot has left it
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kParts - kPartsAhead) : "memory");
                const int bytes = min(page - o, kPartBytes);
                r.to[in] = pages + t * p.a.page_stride + o;
                r.bytes[in] = bytes;
                if (ok) {
                    mbar_arrive_expect_tx(&r.full[in], bytes);
                    bulk_copy_g2s(r.part[in], pages + f * p.a.page_stride + o, bytes, &r.full[in], policy);
                }
                if (++in == kParts) in = 0;
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
        for (long long i = min(mine, static_cast<long long>(kPartsAhead)); i > 0 && ok; --i) ok = send();
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok) {
            // copies in flight get time to land before shared memory is given up
            const long long t0 = clock64();
            while (clock64() - t0 < 2000ll * 1000ll) {
            }
            *p.a.used = -1;
        }
    }
}

// Pools of up to kBitsPages pages: every block counts all of them itself, as bits in its shared memory with the set bits
// before each word, and finds the k-th hole and the k-th moving page there.
constexpr int kBitsPages = 65536, kBitsWords = kBitsPages / 32, kBitsThreads = kMoveThreads;
struct PageBits {
    uint32_t word[kBitsWords];
    int before[kBitsWords];
    int sums[32];
};

// Bits of the block's words to their ranks; returns the number of pages in use.  (words: up to kBitsWords.)
__device__ int rank_bits(PageBits& s, int words) {
    constexpr int kEach = kBitsWords / kBitsThreads;
    int mine[kEach], sum = 0, live;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int w = kEach * threadIdx.x + k;
        mine[k] = w < words ? __popc(s.word[w]) : 0;
        sum += mine[k];
    }
    int at = block_scan(sum, s.sums, live) - sum;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        s.before[kEach * threadIdx.x + k] = at;            // (behind the last word: all)
        at += mine[k];
    }
    __syncthreads();
    return live;
}
__device__ __forceinline__ int bit_rank(const PageBits& s, int i) {
    return s.before[i >> 5] + __popc(s.word[i >> 5] & ((1u << (i & 31)) - 1));
}
// The n-th bit (from 0) that is set, or with kZero that is not.
template <bool kZero>
__device__ __noinline__ int nth_bit(const PageBits& s, int words, int n) {
    int lo = 0, hi = words;                                // the word lies in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((kZero ? 32 * mid - s.before[mid] : s.before[mid]) <= n)
            lo = mid;
        else
            hi = mid;
    }
    n -= kZero ? 32 * lo - s.before[lo] : s.before[lo];
    uint32_t v = kZero ? ~s.word[lo] : s.word[lo];
    int bit = 0;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
        const int c = __popc(v & ((1u << step) - 1));
        if (n >= c) {
            n -= c;
            v >>= step;
            bit += step;
        }
    }
    return 32 * lo + bit;
}

__global__ void __launch_bounds__(kBitsThreads) mla_compact_bits_kernel(const __grid_constant__ CompactParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    MoveRing& ring = *reinterpret_cast<MoveRing*>(smem_raw);
    PageBits& s = *reinterpret_cast<PageBits*>(smem_raw + sizeof(MoveRing));
    init_ring(ring);
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, words = (p.a.n_pages + 31) >> 5;
    constexpr int kWarps = kBitsThreads / 32, kAhead = 8;
    for (int w0 = threadIdx.x >> 5; w0 < words; w0 += kAhead * kWarps) {
        int refs[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = 32 * (w0 + k * kWarps) + lane;
            refs[k] = i < p.a.n_pages ? p.a.refs[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t word = __ballot_sync(0xffffffffu, refs[k] > 0);
            if (lane == 0 && w0 + k * kWarps < words) s.word[w0 + k * kWarps] = word;
        }
    }
    const int live = rank_bits(s, words);
    const int front = live < 32 * words ? bit_rank(s, live) : live;   // pages in use among the first `live`
    const int moves = live - front;
    const bool in_place = p.a.refs_out == p.a.refs;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) {
            *p.a.used = live;
            p.moves[1] = live;
        }
        if (in_place)
            for (int w = threadIdx.x; w < words; w += kBitsThreads) p.bits[w] = s.word[w];
    }
    // ---- the pages, by one warp; the table and the references by the others
    if (threadIdx.x < 32) {
        move_pages(p, ring, moves, lane, [&](int k, int& from, int& to) {
            from = nth_bit<false>(s, words, front + k);
            to = nth_bit<true>(s, words, k);
        });
        return;
    }
    // ---- the table
    const long long at = static_cast<long long>(blockIdx.x) * (kBitsThreads - 32) + threadIdx.x - 32;
    const long long step = static_cast<long long>(gridDim.x) * (kBitsThreads - 32);
    const long long entries = static_cast<long long>(p.a.batch) * p.a.columns;
    for (long long e = at; e < entries; e += step) {
        int v = p.a.page_table[e];
        if (v < 0 || v >= p.a.n_pages || !(s.word[v >> 5] >> (v & 31) & 1))
            v = -1;
        else if (v >= live)
            v = nth_bit<true>(s, words, bit_rank(s, v) - front);
        p.a.page_table_out[e] = v;
    }
    if (in_place) return;                                  // (other blocks may still read the references)
    for (long long i = at; i < p.a.n_pages; i += step) {
        const int from = i >= live ? -1 : s.word[i >> 5] >> (i & 31) & 1 ? static_cast<int>(i)
                         : nth_bit<false>(s, words, front + static_cast<int>(i) - bit_rank(s, static_cast<int>(i)));
        p.a.refs_out[i] = from < 0 ? 0 : p.a.refs[from];
    }
}

// The references in place: the k-th moving page's go to the k-th hole.
__global__ void __launch_bounds__(kBitsThreads) mla_compact_refs_kernel(const __grid_constant__ CompactParams p) {
    __shared__ PageBits s;
    grid_dependency_wait();
    allow_dependent_launch();
    const int words = (p.a.n_pages + 31) >> 5, live = p.moves[1];
    for (int w = threadIdx.x; w < words; w += kBitsThreads) s.word[w] = p.bits[w];
    rank_bits(s, words);
    const int front = live < 32 * words ? bit_rank(s, live) : live;
    for (int i = live + blockIdx.x * kBitsThreads + threadIdx.x; i < p.a.n_pages; i += gridDim.x * kBitsThreads) {
        if (s.word[i >> 5] >> (i & 31) & 1)
            p.a.refs_out[nth_bit<true>(s, words, bit_rank(s, i) - front)] = p.a.refs_out[i];
        p.a.refs_out[i] = 0;
    }
}

__global__ void __launch_bounds__(kThreads) mla_compact_count_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int i0 = blockIdx.x * kChunk;
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kChunk / kThreads; ++k) {
        const int i = i0 + k * kThreads + threadIdx.x;
        if (i < p.a.n_pages) mine += p.a.refs[i] > 0;
    }
    int total;
    block_scan(mine, sums, total);
    if (threadIdx.x == 0) p.counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads) mla_compact_list_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int sums[32];
    grid_dependency_wait();
    allow_dependent_launch();
    int live = 0, before = 0;                              // pages in use: all, and in the chunks before
    for (int c0 = 0; c0 < p.chunks; c0 += kThreads) {
        const int c = c0 + threadIdx.x;
        const int v = c < p.chunks ? p.counts[c] : 0;
        int t;
        block_scan(v, sums, t);
        live += t;
        block_scan(c < static_cast<int>(blockIdx.x) ? v : 0, sums, t);
        before += t;
    }
    // pages in use among the first `live`
    int front = 0;
    const int edge = live / kChunk;                        // (the chunk that the front ends in)
    for (int c0 = 0; c0 < edge; c0 += kThreads) {
        int t;
        block_scan(c0 + static_cast<int>(threadIdx.x) < edge ? p.counts[c0 + threadIdx.x] : 0, sums, t);
        front += t;
    }
    {
        int mine = 0, t;
        for (int i = edge * kChunk + threadIdx.x; i < live; i += kThreads) mine += p.a.refs[i] > 0;
        block_scan(mine, sums, t);
        front += t;
    }
    // this chunk's pages, sixteen a thread
    constexpr int kEach = kChunk / kThreads;
    const int i0 = blockIdx.x * kChunk + threadIdx.x * kEach;
    int refs[kEach], mine = 0, t;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        refs[k] = i0 + k < p.a.n_pages ? p.a.refs[i0 + k] : 0;
        mine += refs[k] > 0;
    }
    int rank = before + block_scan(mine, sums, t) - mine;  // pages in use before i
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = i0 + k;
        if (i >= p.a.n_pages) break;
        if (refs[k] > 0) {
            p.place[i] = rank - front;                     // (used for i >= live alone)
            if (i >= live) {
                p.mover[rank - front] = i;
                p.mover_refs[rank - front] = refs[k];
            } else {
                p.place[i] = 0;
            }
            ++rank;
        } else {
            p.place[i] = -1;
            if (i < live) p.hole[i - rank] = i;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.a.used = live;
        p.moves[0] = live - front;
        p.moves[1] = live;
    }
}

__global__ void __launch_bounds__(kMoveThreads) mla_compact_move_kernel(const __grid_constant__ CompactParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    MoveRing& ring = *reinterpret_cast<MoveRing*>(smem_raw);
    init_ring(ring);
    grid_dependency_wait();
    allow_dependent_launch();
    const int moves = p.moves[0], live = p.moves[1];
    if (threadIdx.x < 32) {
        move_pages(p, ring, moves, threadIdx.x, [&](int k, int& from, int& to) {
            from = p.mover[k];
            to = p.hole[k];
        });
        return;
    }
    const long long at = static_cast<long long>(blockIdx.x) * (kMoveThreads - 32) + threadIdx.x - 32;
    const long long step = static_cast<long long>(gridDim.x) * (kMoveThreads - 32);
    const long long entries = static_cast<long long>(p.a.batch) * p.a.columns;
    for (long long e = at; e < entries; e += step) {
        int v = p.a.page_table[e];
        if (v < 0 || v >= p.a.n_pages) {
            v = -1;
        } else {
            const int place = p.place[v];
            if (place < 0)
                v = -1;
            else if (v >= live)
                v = p.hole[place];
        }
        p.a.page_table_out[e] = v;
    }
    // references: of a page that stays its own, of the k-th hole the k-th moving page's
    for (long long i = at; i < p.a.n_pages; i += step) {
        if (i >= live)
            p.a.refs_out[i] = 0;
        else if (p.place[i] >= 0 && p.a.refs_out != p.a.refs)
            p.a.refs_out[i] = p.a.refs[i];
    }
    for (long long k = at; k < moves; k += step) p.a.refs_out[p.hole[k]] = p.mover_refs[k];
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// Outputs may be their inputs, but not lie across them.
bool across(const void* in, const void* out, size_t ints) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
    return a != b && (a < b ? b - a : a - b) < 4 * ints;
}

bool sizes_ok(int batch, int columns, int n_pages) {
    return batch >= 1 && batch <= kMostRequests && columns >= 1 && n_pages >= 1 && n_pages <= (1 << 30) &&
           static_cast<long long>(batch) * columns < (1ll << 30);
}

int check(const void* pages, long long page_stride, int n_pages, int page_rows, int row_bytes, int batch, int columns) {
    if (!pages || !sizes_ok(batch, columns, n_pages)) return MLA_EINVAL;
    if (page_rows < 8 || page_rows > 1024 || (page_rows & (page_rows - 1)) != 0) return MLA_EINVAL;
    if (static_cast<long long>(columns) * page_rows > 0x7fffff00LL) return MLA_EINVAL;
    if (row_bytes < 16 || row_bytes > 65536 || page_stride < static_cast<long long>(page_rows) * row_bytes)
        return MLA_EINVAL;
    return row_bytes % 16 != 0 || page_stride % 16 != 0 || off(pages, 16) ? MLA_EALIGN : MLA_OK;
}

// Scratch: fork's and compact's arrays, whichever are more.
size_t fork_bytes(int batch, int columns, int n_pages) {
    const size_t entries = static_cast<size_t>(batch) * columns;
    return 256 + up256(4 * entries) + 2 * up256(4 * static_cast<size_t>(n_pages)) + 3 * up256(4 * static_cast<size_t>(batch));
}
size_t compact_bytes(int n_pages) {
    const size_t n = static_cast<size_t>(n_pages);
    return 256 + up256(4 * ((n + kChunk - 1) / kChunk)) + 4 * up256(4 * n);
}

struct Carver {
    char* at;
    int* take(size_t ints) {
        int* p = reinterpret_cast<int*>(at);
        at += up256(4 * ints);
        return p;
    }
};

template <class Params>
cudaError_t launch(void (*kernel)(Params), dim3 grid, int threads, const Params& p, void* stream, size_t smem = 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

constexpr size_t kBitsSmem = sizeof(MoveRing) + sizeof(PageBits);
static_assert(kBitsSmem <= 227 * 1024, "fits shared memory");
std::atomic<int> g_pages_prepared[kMaxDevices];

// The device's SMs, and once per device the kernels' shared memory.
int prepare_pages(int* sms) {
    int dev = 0;
    int rc = current_device(&dev);
    if (rc == MLA_OK) rc = device_sm_count(dev, sms);
    if (rc != MLA_OK || g_pages_prepared[dev].load(std::memory_order_acquire)) return rc;
    cudaError_t e = cudaFuncSetAttribute(mla_compact_bits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kBitsSmem));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mla_compact_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(sizeof(MoveRing)));
    for (auto kernel : {mla_fork_block_kernel<false>, mla_fork_block_kernel<true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockBytes);
    if (e == cudaSuccess) g_pages_prepared[dev].store(1, std::memory_order_release);
    return launch_status(e);
}

}  // namespace
}  // namespace mla

extern "C" {

size_t mla_pages_scratch_bytes(int batch, int columns, int n_pages) {
    if (!mla::sizes_ok(batch, columns, n_pages)) return 0;
    return std::max(mla::fork_bytes(batch, columns, n_pages), mla::compact_bytes(n_pages));
}

int mla_pages_fork(const mla_pages_fork_args* args, void* scratch, size_t scratch_bytes, void* stream) {
    using namespace mla;
    if (!args) return MLA_EINVAL;
    int rc = check(args->pages, args->page_stride, args->n_pages, args->page_rows, args->row_bytes, args->batch,
                   args->columns);
    if (rc != MLA_OK) return rc;
    if (!args->page_table || !args->d_pos || !args->page_table_out || !args->d_pos_out || !args->refs || !args->missing ||
        args->reserve < 0 || args->window < 0 || args->sink < 0)
        return MLA_EINVAL;
    if (off(args->page_table, 4) || off(args->d_pos, 4) || off(args->parent, 4) || off(args->rows, 4) ||
        off(args->page_table_out, 4) || off(args->d_pos_out, 4) || off(args->refs, 4) || off(args->missing, 4))
        return MLA_EALIGN;
    if (across(args->page_table, args->page_table_out, static_cast<size_t>(args->batch) * args->columns) ||
        across(args->d_pos, args->d_pos_out, args->batch))
        return MLA_EINVAL;
    if (!scratch || off(scratch, 256) || scratch_bytes < fork_bytes(args->batch, args->columns, args->n_pages))
        return MLA_ESCRATCH;
    ForkParams p{};
    p.a = *args;
    while ((1 << p.shift) < args->page_rows) ++p.shift;
    Carver c{static_cast<char*>(scratch)};
    p.ticket = c.take(64);
    p.table = c.take(static_cast<size_t>(args->batch) * args->columns);
    p.keeper = c.take(args->n_pages);
    p.free = c.take(args->n_pages);
    p.rows = c.take(args->batch);
    p.src = c.take(args->batch);
    p.dst = c.take(args->batch);
    if (fork_block_bytes(*args) <= kBlockBytes && args->batch * args->columns <= kBlockEntries) {
        int sms = 0;
        rc = prepare_pages(&sms);
        if (rc != MLA_OK) return rc;
        const size_t smem = static_cast<size_t>(fork_block_bytes(*args));
        if (static_cast<long long>(args->batch) * args->page_rows * args->row_bytes <= kOwnCopies)
            return launch_status(launch(mla_fork_block_kernel<true>, dim3(1), kPlaceThreads, p, stream, smem));
        cudaError_t e = launch(mla_fork_block_kernel<false>, dim3(1), kPlaceThreads, p, stream, smem);
        if (e == cudaSuccess) e = launch(mla_fork_copy_kernel, dim3(args->batch), kThreads, p, stream);
        return launch_status(e);
    }
    const dim3 count((args->columns + kPlaceThreads - 1) / kPlaceThreads, args->batch);
    p.blocks = static_cast<int>(count.x * count.y);
    const int clear = std::min((args->n_pages + kThreads - 1) / kThreads, 1024);
    cudaError_t e = launch(mla_fork_clear_kernel, dim3(clear), kThreads, p, stream);
    if (e == cudaSuccess) e = launch(mla_fork_count_kernel, count, kPlaceThreads, p, stream);
    if (e == cudaSuccess) e = launch(mla_fork_write_kernel, dim3(args->batch), kThreads, p, stream);
    return launch_status(e);
}

int mla_pages_compact(const mla_pages_compact_args* args, void* scratch, size_t scratch_bytes, void* stream) {
    using namespace mla;
    if (!args) return MLA_EINVAL;
    int rc = check(args->pages, args->page_stride, args->n_pages, args->page_rows, args->row_bytes, args->batch,
                   args->columns);
    if (rc != MLA_OK) return rc;
    if (!args->page_table || !args->refs || !args->page_table_out || !args->refs_out || !args->used) return MLA_EINVAL;
    if (off(args->page_table, 4) || off(args->refs, 4) || off(args->page_table_out, 4) || off(args->refs_out, 4) ||
        off(args->used, 4))
        return MLA_EALIGN;
    if (across(args->page_table, args->page_table_out, static_cast<size_t>(args->batch) * args->columns) ||
        across(args->refs, args->refs_out, args->n_pages))
        return MLA_EINVAL;
    if (!scratch || off(scratch, 256) || scratch_bytes < compact_bytes(args->n_pages)) return MLA_ESCRATCH;
    CompactParams p{};
    p.a = *args;
    p.chunks = (args->n_pages + kChunk - 1) / kChunk;
    Carver c{static_cast<char*>(scratch)};
    p.moves = c.take(64);
    p.counts = c.take(p.chunks);
    p.place = c.take(args->n_pages);
    p.hole = c.take(args->n_pages);
    p.mover = c.take(args->n_pages);
    p.mover_refs = c.take(args->n_pages);
    int sms = 0;
    rc = prepare_pages(&sms);
    if (rc != MLA_OK) return rc;
    if (args->n_pages <= kBitsPages) {
        p.bits = reinterpret_cast<uint32_t*>(p.hole);
        cudaError_t e = launch(mla_compact_bits_kernel, dim3(sms), kBitsThreads, p, stream, kBitsSmem);
        if (e == cudaSuccess && args->refs_out == args->refs)
            e = launch(mla_compact_refs_kernel, dim3(std::min((args->n_pages + kBitsThreads - 1) / kBitsThreads, sms)),
                       kBitsThreads, p, stream);
        return launch_status(e);
    }
    cudaError_t e = launch(mla_compact_count_kernel, dim3(p.chunks), kThreads, p, stream);
    if (e == cudaSuccess) e = launch(mla_compact_list_kernel, dim3(p.chunks), kThreads, p, stream);
    if (e == cudaSuccess) e = launch(mla_compact_move_kernel, dim3(sms), kMoveThreads, p, stream, sizeof(MoveRing));
    return launch_status(e);
}

}  // extern "C"
