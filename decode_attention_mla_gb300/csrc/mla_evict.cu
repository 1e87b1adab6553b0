// mla_evict.cu -- eviction from the latent cache by accumulated attention
// weight (include/mla_evict.h): select, then move.
//
// Select.  Each row's rank is a 32-bit key that orders as (protected, weight):
// the float's bits made monotonic, NaN as -infinity, -0 as +0, protected rows
// above everything.  The keep-th largest key K is found exactly by a radix
// descent over 11 + 11 + 10 bits with histograms in shared memory, by a cluster
// of CTAs per request that read each other's histograms (distributed shared
// memory); the keys stay in shared memory between the passes when they fit.
// Rows above K stay, and of the rows equal to K the first so many that `keep`
// is met; counts by ballots, summed over warps, CTA and cluster, number the
// evicted rows below `keep` and the kept rows behind it in ascending order,
// which pairs them up.  Integers only: no order of execution shows in the result.
//
// Move.  A warp copies four bf16 rows (eight E4M3 rows) at a time, nine
// 16-byte loads in flight per lane; source rows lie at or behind `keep` and
// destinations below it, so the copy is safe in place.  Bound: the bytes of the
// moved rows, read and written once.
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
constexpr int kBins = 2048;
constexpr int kLoadBatch = 8;
constexpr int kCachedKeys = 32768;                         // keys a CTA holds in shared memory (128 KB)
constexpr int kMaxCluster = 8;
// One CTA up to this many rows per request, a cluster of eight above.
constexpr int kOneCtaRows = 8192;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 288;                            // 16-byte units a warp moves at a time

struct EvictScratch {
    int* n_moves;                                          // [B]
    int* hole;                                             // [B][keep] evicted rows below keep, ascending
    int* moved;                                            // [B][keep] kept rows behind keep, ascending
};

struct SelShared {
    uint32_t hist[2][kBins];
    uint32_t scan[kSelWarps];
    uint32_t bin, above;                                   // the chosen digit, keys with a larger one
    uint32_t warp_gt[2][kSelWarps], warp_eq[2][kSelWarps]; // rows above / equal to K, below keep and behind it
    uint32_t cta_gt[2], cta_eq[2];                         // the CTA's, read by the others of the cluster
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

// Exclusive prefix of this warp's count over the CTA's warps, and the CTA's
// total (counts[] written by lane 0 of every warp before the barrier).
__device__ __forceinline__ uint32_t warp_base(const uint32_t* counts, int warp, int lane, uint32_t* total) {
    const uint32_t v = counts[lane];
    const uint32_t incl = warp_incl_scan(v, lane);
    *total = __shfl_sync(0xffffffffu, incl, 31);
    return __shfl_sync(0xffffffffu, incl - v, warp);
}

template <int CL>
__global__ void __launch_bounds__(kSelThreads) mla_evict_select_kernel(const mla_evict_args a, const EvictScratch s) {
    constexpr int kCache = CL == 1 ? kOneCtaRows : kCachedKeys;
    extern __shared__ uint32_t cached[];
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
    // this CTA's rows [r0, r1), this warp's rows [w0, w1)
    const int per = static_cast<int>(((static_cast<long long>(n) + CL * 1024 - 1) / (CL * 1024)) * 1024);
    const int r0 = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(rank) * per));
    const int r1 = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(r0) + per));
    const int w_per = per / kSelWarps;                     // a multiple of 32
    const int w0 = min(r1, r0 + warp * w_per), w1 = min(r1, w0 + w_per);
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
    // keys into shared memory, eight loads of each array in flight per thread; the
    // rows below keep get their own weight and position in the outputs (the move
    // overwrites those of the evicted ones)
    const bool copy_w = a.weights_out != a.weights, copy_p = a.positions_out != a.positions;
    for (int r = r0 + tid; r < r1; r += kLoadBatch * kSelThreads) {
        float w[kLoadBatch];
        int pos[kLoadBatch];
#pragma unroll
        for (int i = 0; i < kLoadBatch; ++i) {
            const int row = r + i * kSelThreads;
            if (row < r1) {
                w[i] = a.weights[base + row];
                pos[i] = a.positions[base + row];
            }
        }
#pragma unroll
        for (int i = 0; i < kLoadBatch; ++i) {
            const int row = r + i * kSelThreads;
            if (row < r1) {
                if (row - r0 < kCache) cached[row - r0] = rank_key(w[i], pos[i], a.sink, recent_from);
                if (row < keep) {
                    if (copy_w) a.weights_out[base + row] = w[i];
                    if (copy_p) a.positions_out[base + row] = pos[i];
                }
            }
        }
    }

    // ---- the keep-th largest key
    uint32_t prefix = 0, need = static_cast<uint32_t>(keep);
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
        const uint32_t high_mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
        uint32_t* hist = sh.hist[pass & 1];
        hist[tid] = 0;
        hist[tid + kSelThreads] = 0;
        __syncthreads();
        for (int r = r0 + tid; r < r1; r += kSelThreads) {
            const uint32_t k = key_of(r);
            if ((k & high_mask) == prefix) atomicAdd(&hist[(k >> shift) & digit_mask], 1u);
        }
        everyone();
        // every CTA sums all histograms: thread t takes the bins 2047 - 2t, 2046 - 2t (descending)
        uint32_t c0 = 0, c1 = 0;
        const int bin0 = kBins - 1 - 2 * tid;
#pragma unroll
        for (int q = 0; q < CL; ++q) {
            const uint32_t* h = CL == 1 ? hist : cluster.map_shared_rank(hist, q);
            c0 += h[bin0];
            c1 += h[bin0 - 1];
        }
        const uint32_t incl = warp_incl_scan(c0 + c1, lane);
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        uint32_t total;
        const uint32_t before = warp_base(sh.scan, warp, lane, &total) + incl - (c0 + c1);
        if (before < need && before + c0 >= need) {
            sh.bin = bin0;
            sh.above = before;
        } else if (before + c0 < need && before + c0 + c1 >= need) {
            sh.bin = bin0 - 1;
            sh.above = before + c0;
        }
        __syncthreads();
        prefix |= sh.bin << shift;
        need -= sh.above;
        // the next pass writes the other histogram; this one is not written again
        // before every CTA has passed the next pass's cluster barrier
    }
    const uint32_t K = prefix;                             // `need` rows equal to K stay, the first ones

    // ---- this warp's rows above and equal to K, below keep and behind it
    uint32_t gt[2] = {0, 0}, eqs[2] = {0, 0};
    for (int r = w0; r < w1; r += 32) {
        const int row = r + lane;
        const uint32_t k = row < w1 ? key_of(row) : 0u;
        const uint32_t g = __ballot_sync(0xffffffffu, row < w1 && k > K);
        const uint32_t e = __ballot_sync(0xffffffffu, row < w1 && k == K);
        const uint32_t low = keep - r >= 32 ? 0xffffffffu : keep > r ? (1u << (keep - r)) - 1u : 0u;
        gt[0] += __popc(g & low);
        gt[1] += __popc(g & ~low);
        eqs[0] += __popc(e & low);
        eqs[1] += __popc(e & ~low);
    }
    if (lane == 0) {
        sh.warp_gt[0][warp] = gt[0];
        sh.warp_gt[1][warp] = gt[1];
        sh.warp_eq[0][warp] = eqs[0];
        sh.warp_eq[1][warp] = eqs[1];
    }
    __syncthreads();
    // every warp: the CTA's totals and, for lane w, what lies before warp w of the CTA
    const uint32_t my_gt0 = sh.warp_gt[0][lane], my_gt1 = sh.warp_gt[1][lane];
    const uint32_t my_eq0 = sh.warp_eq[0][lane], my_eq1 = sh.warp_eq[1][lane];
    const uint32_t eq_incl = warp_incl_scan(my_eq0 + my_eq1, lane);
    if (CL > 1) {
        if (warp == 0) {
            const uint32_t t[4] = {warp_incl_scan(my_gt0, lane), warp_incl_scan(my_gt1, lane),
                                   warp_incl_scan(my_eq0, lane), warp_incl_scan(my_eq1, lane)};
            if (lane == 31) {
                sh.cta_gt[0] = t[0];
                sh.cta_gt[1] = t[1];
                sh.cta_eq[0] = t[2];
                sh.cta_eq[1] = t[3];
            }
        }
        everyone();
    }
    // Of `e` rows equal to K with `before` such rows in front, min(e, need - before)
    // stay, the first ones; so the evicted rows below keep and the kept ones behind
    // it follow from the counts.
    auto holes_of = [&](uint32_t below, uint32_t g0, uint32_t e0, uint32_t before) {
        const uint32_t stay = before < need ? min(e0, need - before) : 0u;
        return below - g0 - stay;
    };
    auto moves_of = [&](uint32_t g1, uint32_t e0, uint32_t e1, uint32_t before) {
        const uint32_t stay = before < need ? min(e0 + e1, need - before) : 0u;
        return g1 + (stay > e0 ? stay - e0 : 0u);
    };
    auto rows_below = [&](long long from, long long to) {  // of [from, to): rows below keep
        const long long end = to < keep ? to : keep;
        return static_cast<uint32_t>(end > from ? end - from : 0);
    };
    uint32_t eq0 = 0, hole0 = 0, moved0 = 0, all_moves = 0;
    if (CL > 1) {
        uint32_t before = 0;
#pragma unroll
        for (int q = 0; q < CL; ++q) {
            const uint32_t* g = cluster.map_shared_rank(sh.cta_gt, q);
            const uint32_t* e = cluster.map_shared_rank(sh.cta_eq, q);
            const uint32_t e0 = e[0], e1 = e[1], mv = moves_of(g[1], e0, e1, before);
            const long long from = min(static_cast<long long>(n), static_cast<long long>(q) * per);
            const long long to = min(static_cast<long long>(n), from + per);
            if (q < rank) {
                eq0 += e0 + e1;
                hole0 += holes_of(rows_below(from, to), g[0], e0, before);
                moved0 += mv;
            }
            all_moves += mv;
            before += e0 + e1;
        }
    }
    {
        // lane w: warp w's counts, then the exclusive prefix at this warp
        const long long from = min(static_cast<long long>(r1), static_cast<long long>(r0) + lane * w_per);
        const long long to = min(static_cast<long long>(r1), from + w_per);
        const uint32_t before = eq0 + eq_incl - (my_eq0 + my_eq1);
        const uint32_t h = holes_of(rows_below(from, to), my_gt0, my_eq0, before);
        const uint32_t m = moves_of(my_gt1, my_eq0, my_eq1, before);
        const uint32_t h_incl = warp_incl_scan(h, lane), m_incl = warp_incl_scan(m, lane);
        if (CL == 1) all_moves = __shfl_sync(0xffffffffu, m_incl, 31);
        eq0 = __shfl_sync(0xffffffffu, before, warp);
        hole0 += __shfl_sync(0xffffffffu, h_incl - h, warp);
        moved0 += __shfl_sync(0xffffffffu, m_incl - m, warp);
    }
    if (rank == 0 && tid == 0) {
        s.n_moves[b] = static_cast<int>(all_moves);        // as many as evicted rows below keep
        a.d_pos_out[b] = keep;                             // every CTA read d_pos before its first barrier
    }
    int* hole_list = s.hole + static_cast<long long>(b) * a.keep;
    int* moved_list = s.moved + static_cast<long long>(b) * a.keep;
    uint32_t eq = eq0;
    const uint32_t lower = (1u << lane) - 1u;
    for (int r = w0; r < w1; r += 32) {
        const int row = r + lane;
        const uint32_t k = row < w1 ? key_of(row) : 0u;
        const bool is_eq = row < w1 && k == K;
        const uint32_t bal = __ballot_sync(0xffffffffu, is_eq);
        const bool kept = row < w1 && (k > K || (is_eq && eq + __popc(bal & lower) < need));
        eq += __popc(bal);
        const bool hole = row < w1 && row < keep && !kept, moved = row >= keep && kept;
        const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, moved);
        if (hole) hole_list[hole0 + __popc(hb & lower)] = row;
        if (moved) moved_list[moved0 + __popc(mb & lower)] = row;
        hole0 += __popc(hb);
        moved0 += __popc(mb);
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
    const int warps = gridDim.x * (kMoveThreads / 32);
    const int step = warps * kRows;
    for (long long k0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * static_cast<long long>(kRows); k0 < n;
         k0 += step) {
        int src = 0, dst = 0;
        if (lane < kRows && k0 + lane < n) {
            src = moved[k0 + lane];
            dst = hole[k0 + lane];
            a.weights_out[base + dst] = a.weights[base + src];
            a.positions_out[base + dst] = a.positions[base + src];
        }
        uint4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int w = lane + 32 * i, row = w / UNITS;
            const int from = __shfl_sync(0xffffffffu, src, row);
            if (k0 + row < n) v[i] = reinterpret_cast<const uint4*>(kv + from * stride)[w - row * UNITS];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int w = lane + 32 * i, row = w / UNITS;
            const int to = __shfl_sync(0xffffffffu, dst, row);
            if (k0 + row < n) reinterpret_cast<uint4*>(kv + to * stride)[w - row * UNITS] = v[i];
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
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 1 : 0;
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
    if (grid > 4096) grid = 4096;
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
