// mla_tree_attend.cu -- attention of drafted tokens over the latent cache on
// pairs of SMs (tcgen05 cta_group::2, tensor memory, TMA).
//
// Rows and tiles.  All (token, head) query rows of a request share its cache
// rows, so they are one matrix: row r = token * heads + head, in blocks of 128
// rows, and
//     S = Q K^T * scale,   P = exp2(S - m),   O += P V,   V = the latent part of K
// is taken for 128 cache rows (a tile) at a time.  A pair of CTAs owns a row
// block, 64 rows each: O is 64 x 512 fp32 per CTA and fits tensor memory (256
// columns) beside two score buffers, and every operand is read from shared
// memory half per SM, which one SM alone could not do: with 128 rows O would
// fill tensor memory, with 64 rows the MMA would run at half rate.
//
//   QK: M = 128 (64 rows per CTA), N = 128 keys (64 per CTA),   K = 576: 36 MMAs
//   PV: M = 128,                   N = 256 features (128 per CTA), K = 128 keys: 2 x 8 MMAs
//
// In tensor memory a row's 128 scores lie in two lanes (row, row + 64), 64 keys
// each; O likewise, so two threads own a row and share only its reference m.
//
// Work split.  The units (request, row block, tile), in this order, are cut
// into equal runs, one per pair, from the lengths on the device: no pair idles
// however ragged the batch.  A run that holds a whole row block writes the
// result; otherwise it leaves a normalised fp32 piece and its log-sum-exp, and
// a second kernel merges the pieces of a block in ascending order.
//
// Staging.  Ring of eight 16 KB slots (64 keys x 128 columns) filled by TMA in
// the order the MMAs take them: four slots with this CTA's 64 keys for QK, four
// with its 256 features of all 128 keys for PV (keys of the other CTA's half are
// L2 hits).  QK of tile g + 1 is issued before PV of tile g, so the softmax of a
// tile runs under the next tile's QK.
//
// Warps of a CTA: 0-3 softmax and epilogue (thread = tensor-memory lane), 4
// TMA producer, 5 MMA issue (even CTA only) and tensor memory.  Barriers that
// the MMA thread waits on live in the even CTA and take arrivals of both.
//
// Rounding: P is rounded to bf16 for the product (relative 2^-8 at most per
// probability, sums use the unrounded values), O and the statistics are fp32.
//
// What a token does not attend must not reach it although the product runs over
// whole tiles: masked scores become -infinity and P = 0, and in the tiles that
// hold drafted rows or rows behind them the softmax threads clear, in the staged
// V, the rows behind the end and every non-finite value of a drafted row (a
// token that attends such a row has a NaN score, unless the score is -infinity).
//
// Every wait is bounded; a wait that runs out raises MLA_EDEVICE in the status
// word, both CTAs leave their loops and meet at a cluster barrier, and copies
// still in flight get time to land before shared memory is given up.
#include <cfloat>
#include <cmath>

#include "mla_tree.cuh"
#include "tc_pair_utils.cuh"

namespace mla {
namespace {

constexpr int kSlots = 8;
constexpr uint32_t kSlotBytes = 16384;                     // 2 column chunks of 64 rows x 128 bytes
constexpr uint32_t kChunkBytes = 8192;
constexpr uint32_t kQBytes = 9 * kChunkBytes;
constexpr int kThreads = 192;
constexpr int kSoftmaxThreads = 128;
constexpr int kProducerWarp = 4, kMmaWarp = 5;
constexpr int kBarSoftmax = 1;                             // hardware barrier of the softmax warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0, kTmemS = 256;               // O: 2 x 128 columns, S: 2 x 64 columns
constexpr float kRescaleLog2 = 8.0f;                       // move the reference when a max grows past 2^8
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kDrainCycles = 2000ll * 1000ll;        // about 1 ms: time for copies in flight after an abort

struct Work {                                              // this cluster's run of units
    int b;
    long long rel, count, per;                             // first unit of the run within request b, units, run length
};

struct __align__(1024) Shared {
    uint8_t ring[kSlots][kSlotBytes];
    uint8_t rope[kChunkBytes];                             // this CTA's 64 keys, rope columns
    uint8_t q[kQBytes];                                    // 9 chunks of 64 query rows
    uint8_t p[2][kChunkBytes];                             // P, 64 rows x 128 keys, two key atoms
    float red_max[kSoftmaxThreads], red_sum[kSoftmaxThreads];
    uint64_t ready[kSlots], rope_ready, q_ready, p_ready, o_free;   // used in the even CTA, arrivals of both
    uint64_t empty[kSlots], rope_empty, q_empty, s_full[2], o_done; // in each CTA, arrivals of the MMA thread
    uint64_t v_local[2];                                   // V of a tile with drafted rows has landed in this CTA
    uint64_t stall_bar;
    Work work;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Shared) + 1024 <= 227 * 1024, "fits shared memory");

__device__ __forceinline__ int row_blocks(const TreeParams& p, const TreeRequest& r) {
    return (r.n_tok * p.heads + kTreeBlockRows - 1) / kTreeBlockRows;
}
__device__ __forceinline__ int tiles_of(const TreeRequest& r) { return (r.hi + kTreeTileKeys - 1) / kTreeTileKeys; }

// Walks the tiles of a run.
struct Cursor {
    TreeRequest r;
    int b, rb, n_rb, tile, n_tiles;
    long long left;                                        // tiles of the run from here on, this one included
    int g;                                                 // tiles of the run before this one
    int item;                                              // row blocks (or parts) before this one
    bool first;                                            // first tile of its item

    __device__ __forceinline__ void request(const TreeParams& p) {
        r = load_tree_request(p, b);
        n_rb = row_blocks(p, r);
        n_tiles = tiles_of(r);
    }
    __device__ __forceinline__ void start(const TreeParams& p, const Work& w) {
        b = w.b;
        left = w.count;
        g = item = 0;
        first = true;
        if (left <= 0) return;
        request(p);
        rb = static_cast<int>(w.rel / n_tiles);
        tile = static_cast<int>(w.rel - static_cast<long long>(rb) * n_tiles);
    }
    __device__ __forceinline__ bool last() const { return left == 1 || tile == n_tiles - 1; }
    __device__ __forceinline__ void next(const TreeParams& p) {
        first = last();
        if (first) ++item;
        ++g;
        --left;
        if (++tile < n_tiles) return;
        tile = 0;
        if (++rb < n_rb || left <= 0) return;
        rb = 0;
        do {
            ++b;
            request(p);
        } while (n_rb == 0 || n_tiles == 0);
    }
    // the tile holds drafted rows or rows behind them
    __device__ __forceinline__ bool special() const { return (tile + 1) * kTreeTileKeys > r.d_pos; }
};

// Tell both CTAs of the pair to leave their loops (neither exits before both
// have reached the closing cluster barrier).
__device__ __forceinline__ void raise_error(Shared& sh, int* status) {
    st_cluster_s32(map_to_rank(&sh.abort_flag, 0), 1);
    st_cluster_s32(map_to_rank(&sh.abort_flag, 1), 1);
    if (status) atomicCAS(status, 0, static_cast<int>(MLA_EDEVICE));
}

// One warp: this cluster's run.  All units in order of (request, row block,
// tile); run length = ceil(units / clusters), at least min_tiles.
__device__ void find_work(const TreeParams& p, int cluster, int lane, Work* out) {
    auto units_of = [&](int b) -> long long {
        if (b >= p.batch) return 0;
        const TreeRequest r = load_tree_request(p, b);
        return static_cast<long long>(row_blocks(p, r)) * tiles_of(r);
    };
    const long long mine = units_of(lane);                 // requests 0 .. 31 stay in registers
    long long total = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) total += b0 == 0 ? mine : units_of(b0 + lane);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    long long per = (total + p.clusters - 1) / p.clusters;
    if (per < p.min_tiles) per = p.min_tiles;
    const long long u0 = per * cluster;
    Work w;
    w.per = per;
    w.b = 0;
    w.rel = 0;
    w.count = u0 >= total ? 0 : (total - u0 < per ? total - u0 : per);
    long long before = 0;
    for (int b0 = 0; b0 < p.batch && w.count > 0; b0 += 32) {
        const long long u = b0 == 0 ? mine : units_of(b0 + lane);
        long long incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const bool here = u0 >= before + incl - u && u0 < before + incl;
        const uint32_t at = __ballot_sync(0xffffffffu, here);
        if (at) {
            const int src = __ffs(at) - 1;
            w.b = b0 + src;
            w.rel = u0 - before - __shfl_sync(0xffffffffu, incl - u, src);
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *out = w;
}

// ============================== producer ==================================
struct Producer {
    const TreeMaps& maps;
    const TreeParams& p;
    Shared& sh;
    uint32_t rank;
    uint64_t pol_kv, pol_q;
    uint32_t n = 0;                                        // ring slots filled so far
    uint32_t specials = 0;

    __device__ __forceinline__ bool slot_free() {
        return n < kSlots || mbar_wait_bounded_cluster(&sh.empty[n % kSlots], ((n / kSlots) - 1) & 1, &sh.abort_flag);
    }
    __device__ bool load_q(const Cursor& c) {
        if (c.item > 0 && !mbar_wait_bounded_cluster(&sh.q_empty, (c.item - 1) & 1, &sh.abort_flag)) return false;
        const uint32_t bar = map_to_rank(&sh.q_ready, 0);
        mbar_arrive_expect_tx_cluster(bar, kQBytes);
        const int row = c.b * p.tokens * p.heads + c.rb * kTreeBlockRows + static_cast<int>(rank) * 64;
        tma_load_3d_pair(sh.q, &maps.q, 0, row, 0, bar, pol_q);
        return true;
    }
    // QK operands: this CTA's 64 keys, 128 columns a slot, then the rope columns
    __device__ bool load_k(const Cursor& c) {
        const int y = static_cast<int>(c.r.base) + c.tile * kTreeTileKeys + static_cast<int>(rank) * 64;
#pragma unroll 1
        for (int s = 0; s < 4; ++s, ++n) {
            if (!slot_free()) return false;
            const uint32_t bar = map_to_rank(&sh.ready[n % kSlots], 0);
            mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
            tma_load_3d_pair(sh.ring[n % kSlots], &maps.kv, 0, y, 2 * s, bar, pol_kv);
        }
        if (c.g > 0 && !mbar_wait_bounded_cluster(&sh.rope_empty, (c.g - 1) & 1, &sh.abort_flag)) return false;
        const uint32_t bar = map_to_rank(&sh.rope_ready, 0);
        mbar_arrive_expect_tx_cluster(bar, kChunkBytes);
        tma_load_3d_pair(sh.rope, &maps.rope, 0, y, 8, bar, pol_kv);
        return true;
    }
    // PV operands: features 256 i + 128 rank .. + 127 of the keys of half kb
    __device__ bool load_v(const Cursor& c) {
        const int y = static_cast<int>(c.r.base) + c.tile * kTreeTileKeys;
        const bool special = c.special();
        // two barriers: V of two such tiles may be staged at once, of three not
        // (V of tile g + 2 takes the slots of V of tile g)
        uint64_t* local = &sh.v_local[specials & 1];
        if (special) {
            mbar_arrive_expect_tx(local, 4 * kSlotBytes);
            ++specials;
        }
#pragma unroll 1
        for (int s = 0; s < 4; ++s, ++n) {
            if (!slot_free()) return false;
            const uint32_t bar = map_to_rank(&sh.ready[n % kSlots], 0);
            const int i = s >> 1, kb = s & 1;
            if (special) {
                // the softmax threads wait for these bytes and vouch for them with P
                tma_load_3d(sh.ring[n % kSlots], &maps.kv, 0, y + 64 * kb, 4 * i + 2 * static_cast<int>(rank),
                            local, pol_kv);
                mbar_arrive_cluster(bar);
            } else {
                mbar_arrive_expect_tx_cluster(bar, kSlotBytes);
                tma_load_3d_pair(sh.ring[n % kSlots], &maps.kv, 0, y + 64 * kb, 4 * i + 2 * static_cast<int>(rank),
                                 bar, pol_kv);
            }
        }
        return true;
    }
};

__device__ void produce(const TreeMaps& maps, const TreeParams& p, Shared& sh, uint32_t rank) {
    Producer pr{maps, p, sh, rank, l2_policy_evict_normal(), l2_policy_evict_normal()};
    Cursor c;
    c.start(p, sh.work);
    if (c.left <= 0) return;
    bool ok = pr.load_q(c) && pr.load_k(c);
    while (ok) {
        Cursor nx = c;
        const bool more = c.left > 1;
        if (more) nx.next(p);
        // the order in which the MMA thread takes them
        if (more && !nx.first) ok = pr.load_k(nx);
        ok = ok && pr.load_v(c);
        if (ok && more && nx.first) ok = pr.load_q(nx) && pr.load_k(nx);
        if (!more) break;
        c = nx;
    }
    if (!ok) raise_error(sh, p.status);
}

// ============================== MMA issue ==================================
struct Issuer {
    const TreeParams& p;
    Shared& sh;
    uint32_t tmem;
    uint64_t ring_k, ring_v, rope, q, pd;
    uint32_t n = 0;

    __device__ __forceinline__ bool slot_ready() {
        const bool ok = mbar_wait_bounded_cluster(&sh.ready[n % kSlots], (n / kSlots) & 1, &sh.abort_flag);
        tc_fence_after_sync();
        return ok;
    }
    __device__ bool qk(const Cursor& c) {
        constexpr uint32_t idesc = make_idesc_bf16(128, 128, 0, 0);
        const uint32_t d = tmem + kTmemS + 64 * (c.g & 1);
        if (c.first && !mbar_wait_bounded_cluster(&sh.q_ready, c.item & 1, &sh.abort_flag)) return false;
#pragma unroll 1
        for (int s = 0; s < 4; ++s, ++n) {
            if (!slot_ready()) return false;
            const uint64_t kb = ring_k + ((n % kSlots) * kSlotBytes >> 4);
            const uint64_t qb = q + (2 * s * kChunkBytes >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t off = ((k >> 2) * kChunkBytes + (k & 3) * 32u) >> 4;
                umma_pair_bf16(d, qb + off, kb + off, idesc, (s | k) ? 1u : 0u);
            }
            umma_commit_pair(&sh.empty[n % kSlots]);
        }
        if (!mbar_wait_bounded_cluster(&sh.rope_ready, c.g & 1, &sh.abort_flag)) return false;
        tc_fence_after_sync();
#pragma unroll
        for (int k = 0; k < 4; ++k)
            umma_pair_bf16(d, q + ((8 * kChunkBytes + k * 32u) >> 4), rope + (k * 32u >> 4), idesc, 1u);
        umma_commit_pair(&sh.rope_empty);
        umma_commit_pair(&sh.s_full[c.g & 1]);
        if (c.last()) umma_commit_pair(&sh.q_empty);
        return true;
    }
    __device__ bool pv(const Cursor& c) {
        constexpr uint32_t idesc = make_idesc_bf16(128, 256, 0, 1);
        if (!mbar_wait_bounded_cluster(&sh.p_ready, c.g & 1, &sh.abort_flag)) return false;
        if (c.first && c.item > 0 && !mbar_wait_bounded_cluster(&sh.o_free, (c.item - 1) & 1, &sh.abort_flag))
            return false;
        tc_fence_after_sync();
#pragma unroll 1
        for (int s = 0; s < 4; ++s, ++n) {
            if (!slot_ready()) return false;
            const uint64_t vb = ring_v + ((n % kSlots) * kSlotBytes >> 4);
            const uint64_t pb = pd + ((s & 1) * kChunkBytes >> 4);
            const uint32_t d = tmem + kTmemO + 128 * (s >> 1);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                umma_pair_bf16(d, pb + (k * 32u >> 4), vb + (k * 2048u >> 4), idesc,
                               (c.first && (s & 1) == 0 && k == 0) ? 0u : 1u);
            umma_commit_pair(&sh.empty[n % kSlots]);
        }
        umma_commit_pair(&sh.o_done);
        return true;
    }
};

__device__ void issue(const TreeParams& p, Shared& sh, uint32_t tmem) {
    Issuer is{p, sh, tmem, make_sdesc(smem_u32(sh.ring), 16, 1024, kLayoutSw128),
              make_sdesc(smem_u32(sh.ring), kChunkBytes, 1024, kLayoutSw128),
              make_sdesc(smem_u32(sh.rope), 16, 1024, kLayoutSw128), make_sdesc(smem_u32(sh.q), 16, 1024, kLayoutSw128),
              make_sdesc(smem_u32(sh.p), 16, 1024, kLayoutSw128)};
    Cursor c;
    c.start(p, sh.work);
    if (c.left <= 0) return;
    bool ok = is.qk(c);
    while (ok) {
        Cursor nx = c;
        const bool more = c.left > 1;
        if (more) nx.next(p);
        if (more && !nx.first) ok = is.qk(nx);
        ok = ok && is.pv(c);
        if (ok && more && nx.first) ok = is.qk(nx);
        if (!more) break;
        c = nx;
    }
    if (!ok) raise_error(sh, p.status);
}

// ============================== softmax ====================================
__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Clear what must not meet P = 0 in the staged V of a tile: rows behind the
// end, and non-finite values of drafted rows.  Slots n0 .. n0 + 3 of the ring.
__device__ void clean_v(Shared& sh, const Cursor& c, uint32_t n0, int tid) {
    const int t0 = c.tile * kTreeTileKeys;
    const int from = max(0, c.r.d_pos - t0);
    const int end = min(kTreeTileKeys, c.r.d_pos + c.r.n_tok - t0);   // rows from here on are behind the drafts
    // unit w of a row: 2 feature halves x 2 chunks x 8 units of 16 bytes
    for (int e = tid; e < (kTreeTileKeys - from) * 32; e += kSoftmaxThreads) {
        const int key = from + (e >> 5), w = e & 31;
        uint8_t* slot = sh.ring[(n0 + 2 * (w >> 4) + (key >> 6)) % kSlots];
        uint4* at = reinterpret_cast<uint4*>(slot + ((w >> 3) & 1) * kChunkBytes + (key & 63) * 128 +
                                             (((w & 7) ^ (key & 7)) << 4));
        if (key >= end) {
            *at = make_uint4(0, 0, 0, 0);
        } else {
            uint4 v = *at;
            if (has_nonfinite(v.x) || has_nonfinite(v.y) || has_nonfinite(v.z) || has_nonfinite(v.w)) {
                uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((x[i] & 0x7f80u) == 0x7f80u) x[i] &= 0xffff0000u;
                    if ((x[i] & 0x7f800000u) == 0x7f800000u) x[i] &= 0x0000ffffu;
                }
                *at = make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
    }
}

// out[0 .. 127] of a row's feature run, in the output's type
__device__ __forceinline__ void store32(const TreeParams& p, bool whole, long long at, const uint32_t (&o)[32],
                                        float inv, float* part) {
    if (!whole || p.a.out_fp32) {
        float4* dst = reinterpret_cast<float4*>((whole ? static_cast<float*>(p.a.out) : part) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                 __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * j]) * inv, __uint_as_float(o[8 * i + 2 * j + 1]) * inv);
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__device__ void softmax(const TreeParams& p, Shared& sh, uint32_t tmem, uint32_t rank, int cluster, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const int row = tid & 63, half = tid >> 6;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t p_bar = map_to_rank(&sh.p_ready, 0), o_bar = map_to_rank(&sh.o_free, 0);
    const uint32_t p_line = smem_u32(sh.p[half]) + row * 128;
    const float c2 = p.scale_log2;
    TreeMerge merge{0, 0, 0, 0};
    uint32_t n_v = 4;                                      // ring number of the tile's first V slot, see below
    uint32_t specials = 0;
    bool ok = true, bad = false;
    Cursor c;
    c.start(p, sh.work);
    while (c.left > 0 && ok) {
        // ---- one item: tiles of one row block
        const int r = c.rb * kTreeBlockRows + static_cast<int>(rank) * 64 + row;
        const int live_rows = c.r.n_tok * p.heads;
        const unsigned long long mask = r < live_rows ? tree_mask(p, c.b, r / p.heads, c.r.n_tok) : 0ull;
        const int b = c.b, rb = c.rb, tile0 = c.tile, n_tiles = c.n_tiles;
        float m_ref = -INFINITY, l = 0.f;
        int done = 0;
        bool last;
        do {
            const int g = c.g, buf = g & 1;
            last = c.last();
            bool w = mbar_wait_bounded_cluster(&sh.s_full[buf], (g >> 1) & 1, &sh.abort_flag);
            w = __all_sync(0xffffffffu, w);
            tc_fence_after_sync();
            uint32_t s[2][32];
            if (w) {
                tmem_ld32_async(tmem + lanes + kTmemS + 64 * buf, s[0]);
                tmem_ld32_async(tmem + lanes + kTmemS + 64 * buf + 32, s[1]);
                tmem_wait_ld32(s[0]);
                tmem_wait_ld32(s[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[0][i] = s[1][i] = 0;
            }
            const int t0 = c.tile * kTreeTileKeys;
            if (t0 + kTreeTileKeys > c.r.d_pos || t0 < c.r.lo || t0 + kTreeTileKeys > c.r.hi) {
                const unsigned long long v = visible64(c.r, mask, t0 + 64 * half);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (!(v >> i & 1)) s[0][i] = 0xff800000u;
                    if (!(v >> (i + 32) & 1)) s[1][i] = 0xff800000u;
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                mx[i & 1] = fmaxf(mx[i & 1], __uint_as_float(s[0][i]));
                mx[2 + (i & 1)] = fmaxf(mx[2 + (i & 1)], __uint_as_float(s[1][i]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
            float alpha = 1.f;
            bad |= !w;
            if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad || top > m_ref + kRescaleLog2)) {
                // rare after the first tile: the row's maximum moves the reference
                sh.red_max[tid] = top;
                if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad)) {
                    ok = false;
                    break;
                }
                const float tm = fmaxf(top, sh.red_max[tid ^ 64]);
                if (tm > m_ref + kRescaleLog2) {
                    if (m_ref > -INFINITY) alpha = ex2_approx(m_ref - tm);
                    m_ref = tm;
                }
                l *= alpha;
            }
            // P of the tile before has been read, O holds all tiles before
            w = g == 0 || mbar_wait_bounded_cluster(&sh.o_done, (g - 1) & 1, &sh.abort_flag);
            w = __all_sync(0xffffffffu, w);
            if (w && __any_sync(0xffffffffu, alpha != 1.f)) {
                // O of this item (tiles before this one; alpha is 1 on the first)
                tc_fence_after_sync();
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {
                    float o[16];
                    tmem_ld16(tmem + lanes + kTmemO + 16 * j, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= alpha;
                    tmem_st16(tmem + lanes + kTmemO + 16 * j, o);
                }
            }
            // ---- probabilities, bf16, K-major lines of 64 keys
            const float base = m_ref > -INFINITY ? m_ref : 0.f;
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t pk[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = ex2_approx(fmaf(__uint_as_float(s[h][8 * u + 2 * i]), c2, -base));
                        const float y = ex2_approx(fmaf(__uint_as_float(s[h][8 * u + 2 * i + 1]), c2, -base));
                        sum[0] += x;
                        sum[1] += y;
                        pk[i] = pack_bf16x2(x, y);
                    }
                    st_shared_v4(p_line + (((4 * h + u) ^ (row & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
                }
            l += sum[0] + sum[1];
            if (c.special()) {
                // this tile's V was loaded for this CTA's own eyes: its ring slots
                // follow the next tile's K slots unless the item ends here
                const uint32_t n0 = n_v + (last ? 0u : 4u);
                bool v = w && mbar_wait_bounded(&sh.v_local[specials & 1], (specials >> 1) & 1, &sh.abort_flag);
                ++specials;
                if (__all_sync(0xffffffffu, v))
                    clean_v(sh, c, n0, tid);
                else
                    w = false;
            }
            fence_proxy_async_all();
            tc_fence_before_sync();
            __syncwarp();
            bad |= !w;                                     // the threads leave together at the next barrier
            if (lane == 0 && !bad) mbar_arrive_cluster(p_bar);
            ++done;
            n_v += 8;
            c.next(p);
        } while (!last);
        if (!ok) break;

        // ---- epilogue: l of both halves, O / l, log-sum-exp
        sh.red_sum[tid] = l;
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad)) {
            ok = false;
            break;
        }
        const float lt = half == 0 ? l + sh.red_sum[tid ^ 64] : sh.red_sum[tid ^ 64] + l;
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const float lse2 = lt == 0.f ? -INFINITY : m_ref + log2f(lt);
        const bool whole = tile0 == 0 && done == n_tiles;
        const int slot = 2 * cluster + (tile0 == 0 ? 1 : 0);
        const int block_row = static_cast<int>(rank) * 64 + row;
        const long long out_row =
            whole ? static_cast<long long>(b) * p.tokens * p.heads + r : static_cast<long long>(slot) * kTreeBlockRows + block_row;
        if (half == 0 && r < live_rows) {
            if (whole)
                p.a.lse[out_row] = lse2 * kLn2;
            else
                p.lse_part[out_row] = lse2;
        }
        if (!whole && tile0 == 0) {
            merge.b = b;
            merge.rb = rb;
            merge.rows = min(kTreeBlockRows, live_rows - rb * kTreeBlockRows);
            merge.pieces = 1 + static_cast<int>((n_tiles - done + sh.work.per - 1) / sh.work.per);
        }
        bool w = mbar_wait_bounded_cluster(&sh.o_done, (c.g - 1) & 1, &sh.abort_flag);
        w = __all_sync(0xffffffffu, w);
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, !w)) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            uint32_t o[32];
            tmem_ld32_async(tmem + lanes + kTmemO + 32 * j, o);
            tmem_wait_ld32(o);
            const int feature = 256 * (j >> 2) + 128 * half + 32 * (j & 3);
            if (r < live_rows) store32(p, whole, out_row * kDLatent + feature, o, inv, p.part);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(o_bar);
    }
    if (!ok && lane == 0) raise_error(sh, p.status);
    if (rank == 0 && tid == 0) p.merge[cluster] = merge;
}

// Requests without rows: their tokens' outputs, by the softmax threads of all CTAs.
__device__ void write_empty(const TreeParams& p, int cta, int ctas, int tid) {
    for (int b = cta; b < p.batch; b += ctas) {
        const TreeRequest r = load_tree_request(p, b);
        if (r.hi > 0 || r.n_tok == 0) continue;
        const long long row0 = static_cast<long long>(b) * p.tokens * p.heads;
        const int rows = r.n_tok * p.heads;
        for (int i = tid; i < rows; i += kSoftmaxThreads) p.a.lse[row0 + i] = -INFINITY;
        const int per = p.a.out_fp32 ? 128 : 64;           // 16-byte units per row
        uint4* o = reinterpret_cast<uint4*>(p.a.out) + row0 * per;
        for (int i = tid; i < rows * per; i += kSoftmaxThreads) o[i] = make_uint4(0, 0, 0, 0);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_tree_attend_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    if (tid == 0) {
        prefetch_tensormap(&maps.kv);
        prefetch_tensormap(&maps.rope);
        prefetch_tensormap(&maps.q);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.ready[i], 2);
            mbar_init(&sh.empty[i], 1);
        }
        mbar_init(&sh.rope_ready, 2);
        mbar_init(&sh.q_ready, 2);
        mbar_init(&sh.p_ready, 8);
        mbar_init(&sh.o_free, 8);
        mbar_init(&sh.rope_empty, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.v_local[0], 1);
        mbar_init(&sh.v_local[1], 1);
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == kProducerWarp) find_work(p, cluster, lane, &sh.work);
    tc_fence_before_sync();
    __syncthreads();
    cluster_barrier();                                     // both CTAs' barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    if (p.stall_test && blockIdx.x == 0 && tid == 32 * kProducerWarp) {
        // test hook: a wait that runs out, so the abort path runs for real
        volatile int never = 0;
        if (!mbar_wait_bounded(&sh.stall_bar, 0, &never, kStallTestCycles)) raise_error(sh, p.status);
    }
    if (warp == kProducerWarp) {
        if (lane == 0) produce(maps, p, sh, rank);
    } else if (warp == kMmaWarp) {
        if (rank == 0 && lane == 0) issue(p, sh, tmem);
    } else {
        softmax(p, sh, tmem, rank, cluster, tid);
        write_empty(p, blockIdx.x, gridDim.x, tid);
    }
    __syncthreads();
    if (*static_cast<volatile int*>(&sh.abort_flag)) {
        // nothing more is issued by this CTA: let its copies and MMAs end
        const long long t0 = clock64();
        while (clock64() - t0 < kDrainCycles) {
        }
    }
    tc_fence_before_sync();
    cluster_barrier();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ============================== merge ======================================
// A warp per row: weights exp2(lse_i - lse) of the pieces, ascending.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;

__global__ void __launch_bounds__(kMergeThreads) mla_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int c0 = blockIdx.x;
    const TreeMerge m = p.merge[c0];
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
    if (m.pieces == 0 || row >= m.rows) return;
    // piece 0 is the owner's second slot, the others are the first slots of the clusters behind it
    auto slot = [&](int i) { return static_cast<long long>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * kTreeBlockRows + row; };
    float top = -INFINITY;
    for (int i = lane; i < m.pieces; i += 32) top = fmaxf(top, p.lse_part[slot(i)]);
    top = warp_max_f32(top);
    const float base = top > -INFINITY ? top : 0.f;
    float sum = 0.f;
    float4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < m.pieces; ++i) {
        const long long s = slot(i);
        const float w = exp2f(p.lse_part[s] - base);       // NaN stays NaN
        const float4* src = reinterpret_cast<const float4*>(p.part + s * kDLatent);
        sum += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = src[lane + 32 * j];
            acc[j].x = fmaf(w, v.x, acc[j].x);
            acc[j].y = fmaf(w, v.y, acc[j].y);
            acc[j].z = fmaf(w, v.z, acc[j].z);
            acc[j].w = fmaf(w, v.w, acc[j].w);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long out_row =
        static_cast<long long>(m.b) * p.tokens * p.heads + static_cast<long long>(m.rb) * kTreeBlockRows + row;
    if (lane == 0) p.a.lse[out_row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 v = make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
        const long long at = out_row * kDLatent + 4 * (lane + 32 * j);
        if (p.a.out_fp32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) = v;
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

}  // namespace

size_t tree_attend_smem_bytes() { return sizeof(Shared) + 1024; }

cudaError_t tree_attend_prepare() {
    return cudaFuncSetAttribute(mla_tree_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(tree_attend_smem_bytes()));
}

cudaError_t launch_tree_attend(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = tree_attend_smem_bytes();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, mla_tree_attend_kernel, maps, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(p.clusters, kTreeBlockRows / kMergeRows);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, mla_tree_merge_kernel, p);
}

}  // namespace mla
