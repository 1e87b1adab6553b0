// mla_evict.cu -- eviction from the latent cache by accumulated attention
// weight (include/mla_evict.h): select, then move.
//
// Select.  Each row's rank is a 32-bit key that orders as (protected, weight):
// the float's bits made monotonic, NaN as -infinity, -0 as +0, protected rows
// above everything.  The keep-th largest key K is found exactly by a radix
// descent over four digits of eight bits, histograms in shared memory, by a
// cluster of CTAs per request that read each other's histograms (distributed
// shared memory is slow: 2048 bins and three digits took three times as long);
// the keys stay in shared memory between the passes when they fit.
// Rows above K stay, and of the rows equal to K the first so many that `keep`
// is met; every warp counts over a contiguous run of rows, and prefix sums over
// warps and CTAs number the evicted rows below `keep` and the kept rows
// behind it in ascending order, which pairs them up.  Integers only: no order of
// execution shows in the result.  Bound: latency (barriers and passes over shared
// memory); 25 us for 16 requests of up to 131072 rows, 8 for one of 8192.
//
// Move.  A warp copies four bf16 rows (eight E4M3 rows) at a time, nine
// 16-byte loads in flight per lane; source rows lie at or behind `keep` and
// destinations below it, so the copy is safe in place.  Bound: the bytes of the
// moved rows, read and written once, in rows of 1152 bytes from anywhere: 116 us
// for 16 requests (0.58 GB in and out, 5 TB/s).
#include <atomic>
#include <cooperative_groups.h>
#include <cstdint>

#include "device_utils.cuh"
#include "mla_evict.h"
#include "mla_internal.h"

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kLoadBatch = 8;
constexpr int kCachedKeys = 32768;                         // keys a CTA holds in shared memory (128 KB)
constexpr int kMaxCluster = 8;
// One CTA up to this many rows per request, a cluster of eight above.  Calls that move
// next to nothing, one CTA / cluster: one request of 4096 rows 11.0 / 14.3 us, 8192 13.0 /
// 14.6, 12288 15.5 / 15.1, 16384 17.2 / 14.4, 32768 26 / 16; eight requests the same.  (From
// about 18 requests on the clusters take turns: 64 of 16384 rows 18 / 62 us.  The rule does
// not look at the batch.)
constexpr int kOneCtaRows = 8192;
constexpr int kMoveThreads = 256;
// Blocks of the move's launch: about four times what fits the GPU at once.  (16 requests of
// 131072 rows to 32768: 152 * 2 blocks 232 us, * 8 210, * 12 205, * 24 207, * 48 210; one
// request, 65536 rows moved: 36, 31.8, 31.9, 31.8, 31.8.)
constexpr int kMoveBlocks = 152 * 12;
constexpr int kMoveUnits = 288;                            // 16-byte units a warp moves at a time

struct EvictScratch {
    int* n_moves;                                          // [B]
    int* hole;                                             // [B][keep] evicted rows below keep, ascending
    int* moved;                                            // [B][keep] kept rows behind keep, ascending
};

// Rows above / equal to the threshold K, below `keep` and behind it.
struct __align__(16) Counts {
    uint32_t gt0, gt1, eq0, eq1;
};

struct SelShared {
    uint32_t hist[2][kBins];
    uint32_t sum[kBins];                                   // over the cluster
    uint32_t bin, above;                                   // the chosen digit, keys with a larger one
    Counts warp_counts[kSelWarps];
    Counts cta;                                            // the CTA's, read by the others of the cluster
};

__device__ __forceinline__ uint32_t rank_key(float w, int pos, int sink, long long recent_from) {
    if (pos < sink || pos >= recent_from) return 0xffffffffu;
    if (w != w) w = -INFINITY;
    if (w == 0.f) w = 0.f;                                 // -0 and +0 tie
    const uint32_t u = __float_as_uint(w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Rows of a request: [0, n) at off.
__device__ __forceinline__ int request_rows(const mla_evict_args& a, int b, long long* base) {
    const long long o = a.row_offset ? a.row_offset[b] : 0;
    *base = o;
    const long long room = o < 0 ? 0 : a.kv_rows - o;
    long long n = a.d_pos[b];
    if (n > room) n = room;
    return n < 0 ? 0 : static_cast<int>(n);
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

template <int CL>
__global__ void __launch_bounds__(kSelThreads) mla_evict_select_kernel(const mla_evict_args a, const EvictScratch s) {
    constexpr int kCache = CL == 1 ? kOneCtaRows : kCachedKeys;
    extern __shared__ __align__(16) uint32_t cached[];
    __shared__ SelShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = CL == 1 ? 0 : static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / CL;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto everyone = [&] {
        if constexpr (CL == 1)
            __syncthreads();
        else
            cluster.sync();
    };
    grid_dependency_wait();
    long long base;
    const int n = request_rows(a, b, &base);
    const int keep = min(n, a.keep);
    // this CTA's rows [r0, r1), in runs of `run` rows (a multiple of 32) per warp
    const int run = static_cast<int>((static_cast<long long>(n) + CL * kSelThreads - 1) / (CL * kSelThreads)) * 32;
    const long long per = static_cast<long long>(run) * kSelWarps;
    const int r0 = static_cast<int>(min(static_cast<long long>(n), rank * per));
    const int r1 = static_cast<int>(min(static_cast<long long>(n), r0 + per));
    if (n <= a.keep) {                                     // uniform over the cluster
        for (int r = r0 + tid; r < r1; r += kSelThreads) {
            a.weights_out[base + r] = a.weights[base + r];
            a.positions_out[base + r] = a.positions[base + r];
        }
        if (rank == 0 && tid == 0) {
            s.n_moves[b] = 0;
            a.d_pos_out[b] = n;
        }
        allow_dependent_launch();
        return;
    }
    const long long recent_from = static_cast<long long>(a.next_pos[b]) - a.recent;
    auto compute_key = [&](int r) {
        return rank_key(a.weights[base + r], a.positions[base + r], a.sink, recent_from);
    };
    auto key_of = [&](int r) { return r - r0 < kCache ? cached[r - r0] : compute_key(r); };
    auto with_keys = [&](auto&& f) {
        if (r1 - r0 <= kCache)
            f([&](int r) { return cached[r - r0]; });
        else
            f(key_of);
    };
    // keys into shared memory, eight loads of each array in flight per thread; the
    // rows below keep get their own weight and position in the outputs (the move
    // overwrites those of the evicted ones)
    const bool copy_w = a.weights_out != a.weights, copy_p = a.positions_out != a.positions;
    auto load = [&](int r, int end, float (&w)[kLoadBatch], int (&pos)[kLoadBatch]) {
#pragma unroll
        for (int i = 0; i < kLoadBatch; ++i) {
            const int row = min(r + i * kSelThreads, end - 1);   // (no branch: all loads at once)
            w[i] = a.weights[base + row];
            pos[i] = a.positions[base + row];
        }
    };
    auto copy = [&](int r, int end, const float (&w)[kLoadBatch], const int (&pos)[kLoadBatch]) {
#pragma unroll
        for (int i = 0; i < kLoadBatch; ++i) {
            const int row = r + i * kSelThreads;
            if (row < end) {
                if (copy_w) a.weights_out[base + row] = w[i];
                if (copy_p) a.positions_out[base + row] = pos[i];
            }
        }
    };
    float w[kLoadBatch];
    int pos[kLoadBatch];
    for (int r = r0 + tid; r < r1; r += kLoadBatch * kSelThreads) {
        load(r, r1, w, pos);
#pragma unroll
        for (int i = 0; i < kLoadBatch; ++i) {
            const int row = r + i * kSelThreads;
            if (row < r1 && row - r0 < kCache) cached[row - r0] = rank_key(w[i], pos[i], a.sink, recent_from);
        }
        if (CL == 1) copy(r, min(r1, keep), w, pos);
    }
    if (CL > 1 && (copy_w || copy_p)) {
        // (the first CTAs have all the rows below keep: shared out over the cluster)
        const int per_cta = (keep + CL - 1) / CL, c0 = min(keep, rank * per_cta), c1 = min(keep, c0 + per_cta);
        for (int r = c0 + tid; r < c1; r += kLoadBatch * kSelThreads) {
            load(r, c1, w, pos);
            copy(r, c1, w, pos);
        }
    }

    // ---- the keep-th largest key
    uint32_t prefix = 0, need = static_cast<uint32_t>(keep);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t high_mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
        uint32_t* hist = sh.hist[pass & 1];
        if (tid < kBins) hist[tid] = 0;
        __syncthreads();
        auto count_key = [&](uint32_t k) {
            if ((k & high_mask) == prefix) atomicAdd(&hist[k >> shift & 255u], 1u);
        };
        with_keys([&](auto key) {
#pragma unroll 4
            for (int r = r0 + tid; r < r1; r += kSelThreads) count_key(key(r));
        });
        everyone();
        // every CTA sums all histograms (the next pass writes the other one; this one
        // is written again only after every CTA has passed the next pass's barrier)
        if (tid < kBins) {
            uint32_t c = 0;
#pragma unroll
            for (int q = 0; q < CL; ++q) c += (CL == 1 ? hist : cluster.map_shared_rank(hist, q))[tid];
            sh.sum[tid] = c;
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: digits 255 - 8 l and the seven below it
            uint32_t c[8], all = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = sh.sum[kBins - 1 - 8 * lane - i];
                all += c[i];
            }
            uint32_t before = warp_incl_scan(all, lane) - all;
            if (before < need && before + all >= need) {   // one lane
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && before + c[i] >= need) {
                        sh.bin = kBins - 1 - 8 * lane - i;
                        sh.above = before;
                    }
                    before += c[i];
                }
            }
        }
        __syncthreads();
        prefix |= sh.bin << shift;
        need -= sh.above;
    }
    const uint32_t K = prefix;                             // `need` rows equal to K stay, the first ones

    // ---- the warp's rows above and equal to K, below keep and behind it
    auto run_from = [&](int w) { return static_cast<int>(min(static_cast<long long>(r1), r0 + static_cast<long long>(w) * run)); };
    const int from = run_from(warp), to = run_from(warp + 1);
    const int low_to = min(max(keep, from), to);           // rows below keep, then the others
    {
        uint32_t gt = 0, eq = 0;
        auto count_rows = [&](int r0, int r1) {
            with_keys([&](auto key) {
#pragma unroll 4
                for (int r = r0 + lane; r < r1; r += 32) {
                    const uint32_t k = key(r);
                    gt += k > K;
                    eq += k == K;
                }
            });
        };
        count_rows(from, low_to);
        const uint32_t gt0 = gt, eq0 = eq;
        count_rows(low_to, to);
        const Counts c{__reduce_add_sync(0xffffffffu, gt0), __reduce_add_sync(0xffffffffu, gt - gt0),
                       __reduce_add_sync(0xffffffffu, eq0), __reduce_add_sync(0xffffffffu, eq - eq0)};
        if (lane == 0) sh.warp_counts[warp] = c;
    }
    // Of the rows equal to K that follow `before` others, min(count, need - before)
    // stay, the first ones: from the counts follow the evicted rows below keep and
    // the kept rows behind it, which prefix sums number.
    auto stay_of = [&](const Counts& c, uint32_t before) {
        return before < need ? min(c.eq0 + c.eq1, need - before) : 0u;
    };
    auto holes_of = [&](const Counts& c, uint32_t before, uint32_t below) {
        return below - c.gt0 - min(c.eq0, stay_of(c, before));
    };
    auto moves_of = [&](const Counts& c, uint32_t before) {
        const uint32_t stay = stay_of(c, before);
        return c.gt1 + (stay > c.eq0 ? stay - c.eq0 : 0u);
    };
    auto rows_below = [&](long long from, long long to) {  // of [from, to): rows below keep
        const long long end = to < keep ? to : keep;
        return static_cast<uint32_t>(end > from ? end - from : 0);
    };
    __syncthreads();
    // every warp: lane l has warp l's counts, of this CTA
    const Counts mine = sh.warp_counts[lane];
    const uint32_t eq_mine = mine.eq0 + mine.eq1;
    const uint32_t eq_incl = warp_incl_scan(eq_mine, lane);
    uint32_t eq = 0, hole0 = 0, moved0 = 0, all_moves = 0;
    if (CL > 1) {
        // what lies in the CTAs before this one: lane q has CTA q's counts
        const Counts sum{__reduce_add_sync(0xffffffffu, mine.gt0), __reduce_add_sync(0xffffffffu, mine.gt1),
                         __reduce_add_sync(0xffffffffu, mine.eq0), __reduce_add_sync(0xffffffffu, mine.eq1)};
        if (tid == 0) sh.cta = sum;
        everyone();
        Counts c{0, 0, 0, 0};
        if (lane < CL) c = *cluster.map_shared_rank(&sh.cta, lane);
        const uint32_t before = warp_incl_scan(c.eq0 + c.eq1, lane) - (c.eq0 + c.eq1);
        const long long c0 = min(static_cast<long long>(n), lane * per), c1 = min(static_cast<long long>(n), c0 + per);
        const uint32_t m = moves_of(c, before), h = lane < CL ? holes_of(c, before, rows_below(c0, c1)) : 0u;
        eq = __shfl_sync(0xffffffffu, before, rank);
        hole0 = __reduce_add_sync(0xffffffffu, lane < rank ? h : 0u);
        moved0 = __reduce_add_sync(0xffffffffu, lane < rank ? m : 0u);
        all_moves = __reduce_add_sync(0xffffffffu, m);
    }
    {
        const uint32_t before = eq + eq_incl - eq_mine;
        const uint32_t h = holes_of(mine, before, rows_below(run_from(lane), run_from(lane + 1)));
        const uint32_t m = moves_of(mine, before);
        const uint32_t hi = warp_incl_scan(h, lane), mi = warp_incl_scan(m, lane);
        eq = __shfl_sync(0xffffffffu, before, warp);
        hole0 += __shfl_sync(0xffffffffu, hi - h, warp);
        moved0 += __shfl_sync(0xffffffffu, mi - m, warp);
        if (CL == 1) all_moves = __shfl_sync(0xffffffffu, mi, 31);
    }
    if (rank == 0 && tid == 0) {
        s.n_moves[b] = static_cast<int>(all_moves);        // as many as evicted rows below keep
        a.d_pos_out[b] = keep;                             // every CTA read d_pos before its first barrier
    }
    int* hole_list = s.hole + static_cast<long long>(b) * a.keep;
    int* moved_list = s.moved + static_cast<long long>(b) * a.keep;
    // the warp's rows again, 32 at a time, so that the lists are written in runs
    // (a thread's own rows one by one: scattered stores, three times the time)
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t eq_warp = __shfl_sync(0xffffffffu, eq_mine, warp);
    auto list_rows = [&](int r0, int r1, bool kept_ones, int* list, uint32_t at, auto&& kept) {
#pragma unroll 4
        for (int r = r0; r < r1; r += 32) {
            const int row = r + lane;
            const bool listed = kept(row, r1) == kept_ones && row < r1;
            const uint32_t who = __ballot_sync(0xffffffffu, listed);
            if (listed) list[at + __popc(who & lower)] = row;
            at += __popc(who);
        }
    };
    auto list_both = [&](auto&& kept) {
        list_rows(from, low_to, false, hole_list, hole0, kept);
        list_rows(low_to, to, true, moved_list, moved0, kept);
    };
    if (eq + eq_warp <= need || (eq >= need && K != 0xffffffffu)) {
        // all or none of the warp's rows equal to K stay
        const uint32_t least = eq + eq_warp <= need ? K : K + 1;
        with_keys([&](auto key) { list_both([&](int row, int end) { return row < end && key(row) >= least; }); });
    } else {
        list_both([&](int row, int end) {
            const uint32_t k = row < end ? key_of(row) : 0u;
            const bool equal = row < end && k == K;
            const uint32_t e = __ballot_sync(0xffffffffu, equal);
            const bool stays = (row < end && k > K) || (equal && eq + __popc(e & lower) < need);
            eq += __popc(e);
            return stays;
        });
    }
    allow_dependent_launch();
    everyone();                                            // no CTA leaves while others read its shared memory
}

template <int UNITS>                                       // 16-byte units per row: 72 (bf16) or 36 (E4M3)
__global__ void __launch_bounds__(kMoveThreads) mla_evict_move_kernel(const mla_evict_args a, const EvictScratch s) {
    constexpr int kRows = kMoveUnits / UNITS;              // rows a warp moves at a time
    constexpr int kPer = kMoveUnits / 32;                  // 16-byte units per lane
    grid_dependency_wait();
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    const int n = s.n_moves[b];
    const int* hole = s.hole + static_cast<long long>(b) * a.keep;
    const int* moved = s.moved + static_cast<long long>(b) * a.keep;
    const long long base = a.row_offset ? a.row_offset[b] : 0;
    const long long stride = a.row_stride * (UNITS == 72 ? 2 : 1);
    char* kv = static_cast<char*>(a.kv) + base * stride;
    const int step = gridDim.x * (kMoveThreads / 32) * kRows;
    long long k0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * static_cast<long long>(kRows);
    // the list entries of the next rows are on their way while rows move
    int src = 0, dst = 0;
    if (lane < kRows && k0 + lane < n) {
        src = moved[k0 + lane];
        dst = hole[k0 + lane];
    }
    for (; k0 < n; k0 += step) {
        uint4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int w = lane + 32 * i, row = w / UNITS;
            const int from = __shfl_sync(0xffffffffu, src, row);
            if (k0 + row < n) v[i] = reinterpret_cast<const uint4*>(kv + from * stride)[w - row * UNITS];
        }
        const bool entry = lane < kRows && k0 + lane < n;
        float weight = 0.f;
        int pos = 0;
        if (entry) {
            weight = a.weights[base + src];
            pos = a.positions[base + src];
        }
        const int to_row = dst;
        if (lane < kRows && k0 + step + lane < n) {
            src = moved[k0 + step + lane];
            dst = hole[k0 + step + lane];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int w = lane + 32 * i, row = w / UNITS;
            const int to = __shfl_sync(0xffffffffu, to_row, row);
            if (k0 + row < n) reinterpret_cast<uint4*>(kv + to * stride)[w - row * UNITS] = v[i];
        }
        if (entry) {
            a.weights_out[base + to_row] = weight;
            a.positions_out[base + to_row] = pos;
        }
    }
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

template <int CL>
cudaError_t launch_select(const mla_evict_args& a, const EvictScratch& s, cudaStream_t st) {
    const size_t smem = CL == 1 ? kOneCtaRows * sizeof(uint32_t) : kCachedKeys * sizeof(uint32_t);
    // (the attribute of the larger form is set once per device)
    static std::atomic<int> prepared[kMaxDevices];
    if (smem > 48 * 1024 - sizeof(SelShared)) {
        int dev = 0;
        if (current_device(&dev) != MLA_OK) return cudaErrorInvalidDevice;
        if (!prepared[dev].load(std::memory_order_acquire)) {
            const cudaError_t e = cudaFuncSetAttribute(
                mla_evict_select_kernel<CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
            prepared[dev].store(1, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * CL);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mla_evict_select_kernel<CL>, a, s);
}

template <int UNITS>
cudaError_t launch_move(const mla_evict_args& a, const EvictScratch& s, cudaStream_t st) {
    // at most `keep` rows move, and no more than lie behind it; a longer request than
    // expected only makes the warps loop
    long long moves = a.max_rows - a.keep;
    if (moves > a.keep) moves = a.keep;
    const long long per = kMoveThreads / 32 * (kMoveUnits / UNITS);
    long long grid = (moves + per - 1) / per;
    if (grid < 1) grid = 1;
    // a few rounds per warp, so that the lists' latency is paid once
    const long long fill = (kMoveBlocks + a.batch - 1) / a.batch;
    if (grid > fill) grid = fill;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), a.batch);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_evict_move_kernel<UNITS>, a, s);
}

}  // namespace
}  // namespace mla

extern "C" size_t mla_evict_scratch_bytes(int batch, int keep) {
    if (batch < 1 || batch > 65535 || keep < 1) return 0;
    return mla::up256(static_cast<size_t>(batch) * 4) + 2 * mla::up256(static_cast<size_t>(batch) * keep * 4);
}

extern "C" int mla_evict(const mla_evict_args* a, void* scratch, size_t scratch_bytes, void* stream) {
    if (!a || !a->kv || !a->weights || !a->positions || !a->d_pos || !a->next_pos || !a->weights_out ||
        !a->positions_out || !a->d_pos_out)
        return MLA_EINVAL;
    if (a->batch < 1 || a->batch > 65535 || a->keep < 1 || a->sink < 0 || a->recent < 0 || a->max_rows < 1)
        return MLA_EINVAL;
    if (a->kv_fp8 != 0 && a->kv_fp8 != 1) return MLA_EINVAL;
    if (a->kv_rows < 1 || a->row_stride < MLA_D_ROW || (a->batch > 1 && !a->row_offset)) return MLA_EINVAL;
    if (a->row_stride % (a->kv_fp8 ? 16 : 8) != 0 || mla::off(a->kv, 16) || mla::off(a->weights, 4) ||
        mla::off(a->positions, 4) || mla::off(a->d_pos, 4) || mla::off(a->next_pos, 4) ||
        mla::off(a->row_offset, 8) || mla::off(a->weights_out, 4) || mla::off(a->positions_out, 4) ||
        mla::off(a->d_pos_out, 4))
        return MLA_EALIGN;
    if (!scratch || mla::off(scratch, 256) || scratch_bytes < mla_evict_scratch_bytes(a->batch, a->keep))
        return MLA_ESCRATCH;
    char* base = static_cast<char*>(scratch);
    const size_t list = mla::up256(static_cast<size_t>(a->batch) * a->keep * 4);
    mla::EvictScratch s{};
    s.n_moves = reinterpret_cast<int*>(base);
    s.hole = reinterpret_cast<int*>(base + mla::up256(static_cast<size_t>(a->batch) * 4));
    s.moved = reinterpret_cast<int*>(reinterpret_cast<char*>(s.hole) + list);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = a->max_rows <= mla::kOneCtaRows ? mla::launch_select<1>(*a, s, st)
                                                    : mla::launch_select<mla::kMaxCluster>(*a, s, st);
    if (e == cudaSuccess)
        e = a->kv_fp8 ? mla::launch_move<36>(*a, s, st) : mla::launch_move<72>(*a, s, st);
    return mla::launch_status(e);
}
