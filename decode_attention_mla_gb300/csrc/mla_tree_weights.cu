// mla_tree_weights.cu -- attention weight that each cache row gets from a
// call's tokens and heads (mla_tree_weights in include/mla_tree.h):
//   w[t] = decay w[t] + sum_r exp(s_rt - lse_r),     s = Q K^T * scale
//
// The log-sum-exps are known, so one pass over the cache is enough.  The scores
// are taken with the cache rows on M, on pairs of SMs (tcgen05 cta_group::2):
//   S^T[256 cache rows x 128 query rows] = K Q^T: 36 MMAs, 128 cache rows and
//   64 query rows from each CTA's shared memory
// so a cache row is one tensor-memory lane, its weight a sum over the lane's
// columns, and no sum crosses threads but that of the two column halves.
//
// Bound: the cache's bytes for up to 256 query rows, the tensor cores above.
// Staging by TMA, in one of three forms chosen by the most query rows a request
// can have:
//   up to 128   queries resident (72 KB), K in 9 slots of 16 KB
//   up to 256   queries resident (144 KB), K in 5 slots (with 4, 7% slower), where the cache
//               has more rows than one tile per pair
//   otherwise   K of the tile resident (9 slots), the query blocks streamed past
//               it from L2 through 9 slots of 8 KB: each cache row is read once
//               however many query rows there are
// (256 query rows, resident / streamed: over 4000 cache rows 9.9 / 8.9 us, 19400 11.7 / 10.4,
// 24000 13.8 / 14.3, 38000 15.3 / 15.8, 131072 31.4 / 39.5; 64 requests of 1000 rows 21 / 25.)
// The units (request, tile of 256 cache rows) are cut into equal runs, one per
// pair, from the lengths on the device.
//
// The tensor cores' sums drop what does not fit, towards zero: over one chain of 36 MMAs a
// score of normal values loses 4.4e-7 of itself.  So there are two chains of half the length,
// added in fp32 (weights over 5164 rows: 1.6e-7 of their norm off with one chain, 0.5e-7 with
// two, as with plain fp32 products).  One block's two partial scores lie side by side in a score
// buffer; of two blocks each chain has a buffer to itself, and the first chain's scores wait in
// registers (with both in one, tensor memory has no room for the next tile's: 30% slower), both
// blocks by one MMA with N = 256 (by two with N = 128, 4% slower).
//
// Measured, back to back in long rows of calls: one query block over 131072 rows 26.5 us, 5.7
// TB/s of cache; 8 requests of 8192 .. 131072 rows with 256 query rows 137 .. 144 us, 5.4 TB/s
// and 1380 TFLOP/s at once; 1024 query rows over 131072 108 us, 1430 TFLOP/s; 16 query rows
// over 8192 rows 7.3 us, most of it launch and set-up.
//
// Warps of a CTA: 0-7 weights (warps w and w + 4 share cache rows and split the
// columns), 8 TMA of K, 9 MMA issue (even CTA) and tensor memory, 10 TMA of Q.
// Waits are bounded as in the attention kernel.
#include <cmath>

#include "mla_tree.cuh"

namespace mla {
namespace {

constexpr int kTileKeys = 256;                             // cache rows per tile of a pair
using Cursor = TreeCursor<kTileKeys, false>;

constexpr int kChunks = 9;                                 // 64-column chunks of a row
constexpr uint32_t kKChunkBytes = 16384;                   // 128 cache rows
constexpr uint32_t kQChunkBytes = 8192;                    // 64 query rows
constexpr int kSumWarps = 8;
constexpr int kSumThreads = 32 * kSumWarps;
constexpr int kKWarp = 8, kMmaWarp = 9, kQWarp = 10;
constexpr int kThreads = 352;
constexpr int kBarSum = 1;
constexpr uint32_t kTmemCols = 512;
// Score buffers, 256 columns each: two blocks' scores, or one block's in two partial sums
// (128 columns each), of the chunks before kSecond and from there on.
constexpr uint32_t kBuffers = 2, kScoreCols = kTmemCols / kBuffers;
constexpr int kSecond = (kChunks + 1) / 2;
constexpr long long kDrainCycles = 2000ll * 1000ll;

// Form of the staging: kBlocks query blocks resident, or (0) streamed.
template <int kBlocks>
struct Cfg {
    static constexpr bool kStream = kBlocks == 0;
    static constexpr int kKSlots = kBlocks == 2 ? 5 : 9;
    static constexpr int kQBuffers = kBlocks == 2 ? 2 : 1;
    // The partial sums: side by side in a score buffer, or (two blocks) in a buffer each
    static constexpr bool kBeside = kBlocks != 2;
    static constexpr bool opens_buffer(int chunk) { return chunk == 0 || (!kBeside && chunk == kSecond); }
    static constexpr bool ends_buffer(int chunk) { return chunk == kChunks - 1 || (!kBeside && chunk == kSecond - 1); }
};

template <int kBlocks>
struct __align__(1024) Shared {
    using C = Cfg<kBlocks>;
    uint8_t k[C::kKSlots][kKChunkBytes];
    uint8_t q[C::kQBuffers * kChunks][kQChunkBytes];       // resident blocks, or a ring of 9 chunks
    __align__(16) float lse2[2][128];                      // base 2, negative; -inf: the row adds nothing
    uint32_t adds[2][4];                                   // bit per row: it adds something
    float half_sum[2][128];
    // used in the even CTA
    uint64_t k_ready[C::kKSlots], q_ready[kChunks], s_free[kBuffers];
    // in each CTA
    uint64_t k_empty[C::kKSlots], q_empty[kChunks], s_full[kBuffers];
    uint64_t stall_bar;
    TreeWork work;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Shared<0>) <= 227 * 1024 && sizeof(Shared<1>) <= 227 * 1024 && sizeof(Shared<2>) <= 227 * 1024,
              "fits shared memory");

// Query blocks of a request (one, of rows that all add nothing, if it has no tokens).
__device__ __forceinline__ int query_blocks(const TreeParams& p, const TreeRequest& r) {
    return max(1, (r.n_tok * p.heads + kTreeBlockRows - 1) / kTreeBlockRows);
}

template <int kBlocks>
__device__ __forceinline__ uint32_t expect(Shared<kBlocks>&, uint64_t* bar, uint32_t bytes, uint32_t rank) {
    if (rank == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
    return map_to_rank(bar, 0);
}

template <int kBlocks>
__device__ void produce_k(const TreeMaps& maps, const TreeParams& p, Shared<kBlocks>& sh, uint32_t rank) {
    using C = Cfg<kBlocks>;
    const uint64_t policy = l2_policy_evict_first();
    uint32_t slot = 0, round = 0;
    bool ok = true;
    Cursor c;
    for (c.start(p, sh.work); c.left > 0 && ok; c.next(p)) {
        const int y = static_cast<int>(c.r.base) + c.tile * kTileKeys + static_cast<int>(rank) * 128;
#pragma unroll 1
        for (int s = 0; s < kChunks && ok; ++s) {
            ok = round == 0 || mbar_wait_bounded(&sh.k_empty[slot], (round - 1) & 1, &sh.abort_flag);
            if (ok)
                tma_load_3d_pair(sh.k[slot], &maps.k, 0, y, s, expect(sh, &sh.k_ready[slot], kKChunkBytes, rank),
                                 policy);
            if (++slot == C::kKSlots) {
                slot = 0;
                ++round;
            }
        }
    }
    if (!ok) raise_tree_error(&sh.abort_flag, p.status);
}

template <int kBlocks>
__device__ void produce_q(const TreeMaps& maps, const TreeParams& p, Shared<kBlocks>& sh, uint32_t rank) {
    using C = Cfg<kBlocks>;
    const uint64_t policy = l2_policy_evict_normal();
    uint32_t round = 0;                                    // times the query buffers were filled
    bool ok = true;
    Cursor c;
    for (c.start(p, sh.work); c.left > 0 && ok; c.next(p)) {
        const int row0 = c.b * p.tokens * p.heads, row = row0 + static_cast<int>(rank) * 64;
        const int blocks = query_blocks(p, c.r);
        const int last0 = query_rows(p, row0 + (blocks - 1) * kTreeBlockRows),
                  last1 = query_rows(p, row0 + (blocks - 1) * kTreeBlockRows + 64);   // (the blocks before it are whole)
        if constexpr (C::kStream) {
            // (a loop of its own for a last block that is not loaded whole: this one keeps
            // pace with the MMAs only while it is short)
            const int whole = last0 + last1 == kTreeBlockRows ? blocks : blocks - 1;
            for (int rb = 0; rb < whole && ok; ++rb, ++round) {
#pragma unroll 1
                for (int s = 0; s < kChunks && ok; ++s) {
                    ok = round == 0 || mbar_wait_bounded(&sh.q_empty[s], (round - 1) & 1, &sh.abort_flag);
                    if (ok)
                        tma_load_3d_pair(sh.q[s], &maps.q, 0, row + rb * kTreeBlockRows, s,
                                         expect(sh, &sh.q_ready[s], kQChunkBytes, rank), policy);
                }
            }
            if (whole < blocks && ok) {
#pragma unroll 1
                for (int s = 0; s < kChunks && ok; ++s) {
                    ok = round == 0 || mbar_wait_bounded(&sh.q_empty[s], (round - 1) & 1, &sh.abort_flag);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&sh.q_ready[s], (last0 + last1) * 128);
                    load_query_rows<1>(sh.q[s], maps, row + whole * kTreeBlockRows, rank == 0 ? last0 : last1, p.q_tail,
                                       s, map_to_rank(&sh.q_ready[s], 0), policy);
                }
                ++round;
            }
        } else if (c.first) {
            // a request's blocks stay for its part of the run
            ok = round == 0 || mbar_wait_bounded(&sh.q_empty[0], (round - 1) & 1, &sh.abort_flag);
            if (ok) {
                if (rank == 0)
                    mbar_arrive_expect_tx(&sh.q_ready[0], ((blocks - 1) * kTreeBlockRows + last0 + last1) * (kChunks * 128));
                for (int i = 0; i < blocks * kChunks; ++i) {
                    const int rb = i / kChunks;
                    load_query_rows<1>(sh.q[i % kChunks * C::kQBuffers + rb], maps, row + rb * kTreeBlockRows,
                                       rb < blocks - 1 ? 64 : rank == 0 ? last0 : last1, p.q_tail, i % kChunks,
                                       map_to_rank(&sh.q_ready[0], 0), policy);
                }
            }
            ++round;
        }
    }
    if (!ok) raise_tree_error(&sh.abort_flag, p.status);
}

// The whole warp walks and waits, one lane issues; barriers are looked at ahead
// of the MMAs before their use (a look never blocks).  A buffer is announced as free only
// to a load that will wait for it: the closing barrier orders what threads did, not the
// arrival of a commit, and the odd CTA may be gone by then.
template <int kBlocks>
__device__ void issue(const TreeParams& p, Shared<kBlocks>& sh, uint32_t tmem) {
    using C = Cfg<kBlocks>;
    constexpr uint32_t idesc = make_idesc_bf16(256, 128 * C::kQBuffers, 0, 0);
    const bool lead = elect_one();
    const uint64_t kd = make_sdesc(smem_u32(sh.k), 16, 1024, kLayoutSw128);
    const uint64_t qd = make_sdesc(smem_u32(sh.q), 16, 1024, kLayoutSw128);
    bool ok = true;
    auto need = [&](bool seen, uint64_t* bar, uint32_t parity) {
        if (!seen) ok = wait_slowly(bar, parity, &sh.abort_flag) && ok;
    };
    uint32_t slot = 0, k_par = 0;
    uint32_t n = 0;                                        // score buffers filled so far
    uint32_t q_round = 0;
    bool see_k = false, see_q = false;
    Cursor c;
    for (c.start(p, sh.work); c.left > 0 && ok; c.next(p)) {
        const int blocks = query_blocks(p, c.r);
        const bool more = c.left > 1;                      // tiles of the run
        if constexpr (C::kStream) {
            for (int rb = 0; rb < blocks && ok; ++rb, ++n) {
                const uint32_t buf = n % kBuffers, q_par = n & 1;
                const uint32_t d = tmem + kScoreCols * buf;
                if (n >= kBuffers) need(false, &sh.s_free[buf], (n / kBuffers - 1) & 1);
                tc_fence_after_sync();
#pragma unroll
                for (int s = 0; s < kChunks; ++s) {
                    if (rb == 0) need(false, &sh.k_ready[s], c.g & 1);
                    need(see_q, &sh.q_ready[s], q_par);
                    if (s + 1 < kChunks) see_q = mbar_test(&sh.q_ready[s + 1], q_par);
                    if (lead && ok) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_pair_bf16(d + (s < kSecond ? 0 : 128), kd + ((s * kKChunkBytes + k * 32u) >> 4),
                                           qd + ((s * kQChunkBytes + k * 32u) >> 4), idesc, (s % kSecond | k) ? 1u : 0u);
                        if (more || rb < blocks - 1) umma_commit_pair(&sh.q_empty[s]);
                        if (more && rb == blocks - 1) umma_commit_pair(&sh.k_empty[s]);
                    }
                }
                see_q = false;
                if (lead && ok) umma_commit_pair(&sh.s_full[buf]);
            }
        } else {
            uint32_t buf = 0, d = 0;
            if (c.first) need(false, &sh.q_ready[0], q_round & 1);
#pragma unroll
            for (int s = 0; s < kChunks; ++s) {
                if (C::opens_buffer(s)) {
                    buf = n % kBuffers;
                    d = tmem + kScoreCols * buf;
                    if (n >= kBuffers) {
                        const uint32_t par = (n / kBuffers - 1) & 1;
                        need(mbar_test(&sh.s_free[buf], par), &sh.s_free[buf], par);
                    }
                    tc_fence_after_sync();
                }
                const uint32_t at = slot;
                need(see_k, &sh.k_ready[at], k_par);
                if (++slot == C::kKSlots) {
                    slot = 0;
                    k_par ^= 1;
                }
                see_k = mbar_test(&sh.k_ready[slot], k_par);
                if (lead && ok) {
                    const uint64_t ka = kd + (at * kKChunkBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_pair_bf16(d + (C::kBeside && s >= kSecond ? 128 : 0), ka + (k * 32u >> 4),
                                       qd + ((s * C::kQBuffers * kQChunkBytes + k * 32u) >> 4), idesc,
                                       (s % kSecond | k) ? 1u : 0u);
                    // (the slot's next load is kKSlots loads on)
                    if (kChunks * c.left - 1 - s >= C::kKSlots) umma_commit_pair(&sh.k_empty[at]);
                }
                if (C::ends_buffer(s)) {
                    if (lead && ok) umma_commit_pair(&sh.s_full[buf]);
                    ++n;
                }
            }
            if (c.last()) {
                if (lead && ok && more) umma_commit_pair(&sh.q_empty[0]);
                ++q_round;
            }
        }
    }
    if (!ok && lead) raise_tree_error(&sh.abort_flag, p.status);
}

// Two fp32 numbers in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ float first(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float second(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ uint64_t add_pairs(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pairs(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// x += y, y of 16 or 32 numbers, x from its number `from` on
template <int N, typename T>
__device__ __forceinline__ void add_to(uint32_t (&x)[32], int from, const T (&y)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t r = add_pairs(pair(x[from + i], x[from + i + 1]), pair(y[i], y[i + 1]));
        x[from + i] = static_cast<uint32_t>(r);
        x[from + i + 1] = static_cast<uint32_t>(r >> 32);
    }
}

template <int kBlocks>
__device__ void add_weights(const TreeParams& p, Shared<kBlocks>& sh, uint32_t tmem, uint32_t rank, int tid) {
    using C = Cfg<kBlocks>;
    const int lane = tid & 31, warp = tid >> 5;
    const int sub = warp >> 2;                             // columns 64 sub .. of a block
    const int key = 32 * (warp & 3) + lane;                // of this CTA's 128
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_bar = map_to_rank(&sh.s_free[0], 0);
    const float c2 = p.scale_log2;
    const uint64_t c2c2 = pair(c2, c2);
    // (of two blocks, the even CTA's 64 + 64 query rows are columns 0 .., the odd one's 128 ..)
    const uint32_t d0 = tmem + lanes + 64 * C::kQBuffers * sub;
    uint32_t n = 0;                                        // score buffers taken so far
    bool bad = false;
    bool careful[2] = {false, false};                      // the block has rows that add nothing
    auto take = [&] { bad |= !warp_wait(&sh.abort_flag, &sh.s_full[n % kBuffers], n / kBuffers & 1); };
    auto release = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0 && !bad) mbar_arrive_peer(s_bar + 8 * (n % kBuffers));   // the score buffer is free
        ++n;
    };
    Cursor c;
    c.start(p, sh.work);
    for (; c.left > 0; c.next(p)) {
        const int live = c.r.n_tok * p.heads;
        const int blocks = query_blocks(p, c.r);
        const int t = c.tile * kTileKeys + static_cast<int>(rank) * 128 + key;
        const bool mine = sub == 0 && t >= c.r.lo && t < c.r.hi;
        float* dst = p.weights + c.r.base + t;
        const float old = mine && p.decay != 0.f ? *dst : 0.f;
        const bool special = c.special();
        // which tokens attend a drafted row (bit per token)
        const bool draft = special && t >= c.r.d_pos;
        unsigned long long seen_by = 0;
        if (draft) {
            const int j = t - c.r.d_pos;
            if (j < c.r.n_tok)
                for (int i = 0; i < c.r.n_tok; ++i) seen_by |= (tree_mask(p, c.b, i, c.r.n_tok) >> j & 1ull) << i;
        }
        uint64_t sum[2] = {0, 0};
        // log-sum-exps of a block to place `at`
        auto stage = [&](int rb, int at) {
            // (their last readers have passed a barrier since: the one of the block or
            // tile before)
            bool none = false;
            if (tid < 128) {
                const int r = rb * kTreeBlockRows + tid;
                float l = -INFINITY;
                if (r < live) l = p.a.lse[static_cast<long long>(c.b) * p.tokens * p.heads + r];
                none = l == -INFINITY;
                sh.lse2[at][tid] = none ? -INFINITY : -l * kLog2e;
                const uint32_t adds = __ballot_sync(0xffffffffu, !none);
                if (lane == 0) sh.adds[at][warp] = adds;
            }
            careful[at] = named_barrier_or(kBarSum, kSumThreads, none);
        };
        // which of a block's columns 64 sub .. count for this row (bit per column)
        auto count = [&](int rb, int at) {
            unsigned long long counts = sh.adds[at][2 * sub] | static_cast<unsigned long long>(sh.adds[at][2 * sub + 1]) << 32;
            if (draft) {
                const int c0 = rb * kTreeBlockRows + 64 * sub;
                unsigned long long seen = 0;
                for (int i = c0 / p.heads; i < c.r.n_tok && i * p.heads < c0 + 64; ++i)
                    if (seen_by >> i & 1ull) seen |= low_bits((i + 1) * p.heads - c0) & ~low_bits(i * p.heads - c0);
                counts &= seen;
            }
            return counts;
        };
        // the weights of 32 columns: all, or those whose bits are set
        auto add = [&](const uint32_t (&s)[32], int at, int col, bool all, uint32_t counts) {
            const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(&sh.lse2[at][col]);
            if (all) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const ulonglong2 l = l4[i];
                    const uint64_t x = fma_pairs(pair(s[4 * i], s[4 * i + 1]), c2c2, l.x);
                    const uint64_t y = fma_pairs(pair(s[4 * i + 2], s[4 * i + 3]), c2c2, l.y);
                    sum[0] = add_pairs(sum[0], pair(ex2_approx(first(x)), ex2_approx(second(x))));
                    sum[1] = add_pairs(sum[1], pair(ex2_approx(first(y)), ex2_approx(second(y))));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = ex2_approx(fmaf(__uint_as_float(s[2 * i]), c2, sh.lse2[at][col + 2 * i]));
                    const float y = ex2_approx(fmaf(__uint_as_float(s[2 * i + 1]), c2, sh.lse2[at][col + 2 * i + 1]));
                    sum[i & 1] = add_pairs(sum[i & 1], pair(counts >> (2 * i) & 1u ? x : 0.f,
                                                            counts >> (2 * i + 1) & 1u ? y : 0.f));
                }
            }
        };
        if constexpr (C::kBeside) {
            for (int rb = 0; rb < blocks; ++rb) {
                const int at = C::kStream ? n & 1 : 0;     // place of the block's log-sum-exps
                if (C::kStream || c.first) stage(rb, at);
                take();
                const int columns = min(kTreeBlockRows, max(live - rb * kTreeBlockRows, 0)) - 64 * sub;
                const uint32_t d = d0 + kScoreCols * (n % kBuffers);
                const bool all = !special && !careful[at];
                const unsigned long long counts = all ? 0 : count(rb, at);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    if (32 * j >= columns || bad) break;   // warp-uniform
                    uint32_t s[32], more[32];
                    tmem_ld32_async(d + 32 * j, s);
                    tmem_ld32_async(d + 128 + 32 * j, more);
                    tmem_wait_ld32(s);
                    tmem_wait_ld32(more);
                    add_to(s, 0, more);
                    add(s, at, 64 * sub + 32 * j, all, static_cast<uint32_t>(counts >> (32 * j)));
                }
                release();
            }
        } else {
            // the first partial scores wait in registers for the second ones (those of rows
            // that do not exist are taken along and not added)
            uint32_t s[2][2][32];
            if (c.first) {
                stage(0, 0);
                stage(1, 1);
            }
            take();
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                for (int j = 0; j < 2; ++j) tmem_ld32_async(d0 + kScoreCols * (n % kBuffers) + 64 * rb + 32 * j, s[rb][j]);
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                for (int j = 0; j < 2; ++j) tmem_wait_ld32(s[rb][j]);
            release();
            take();
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // (16 at a time: there are no registers for more)
                    float more[16];
                    tmem_ld16(d0 + kScoreCols * (n % kBuffers) + 64 * rb + 16 * k, more);
                    add_to(s[rb][k >> 1], 16 * (k & 1), more);
                }
            release();
#pragma unroll
            for (int rb = 0; rb < 2; ++rb) {
                const bool all = !special && !careful[rb];
                const unsigned long long counts = all ? 0 : count(rb, rb);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    add(s[rb][j], rb, 64 * sub + 32 * j, all, static_cast<uint32_t>(counts >> (32 * j)));
            }
        }
        const float total = (first(sum[0]) + second(sum[0])) + (first(sum[1]) + second(sum[1]));
        if (sub == 1) sh.half_sum[c.g & 1][key] = total;
        if (named_barrier_or(kBarSum, kSumThreads, bad)) break;
        if (mine) *dst = (p.decay != 0.f ? p.decay * old : 0.f) + (total + sh.half_sum[c.g & 1][key]);
    }
    if (bad && lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

template <int kBlocks>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_tree_weights_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeParams p) {
    using C = Cfg<kBlocks>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared<kBlocks>& sh = *reinterpret_cast<Shared<kBlocks>*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    if (tid == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.q);
        if (p.q_tail < 64) prefetch_tensormap(&maps.q_tail);
        for (int i = 0; i < C::kKSlots; ++i) {
            mbar_init(&sh.k_ready[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&sh.q_ready[i], 1);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (uint32_t i = 0; i < kBuffers; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 2 * kSumWarps);
        }
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    __syncwarp();
    cluster_arrive();
    if (warp == kMmaWarp) tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == kKWarp) Cursor::find_work(p, cluster, lane, &sh.work);
    tc_fence_before_sync();
    __syncthreads();
    cluster_wait();                                        // both CTAs' barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    if (p.stall_test && blockIdx.x == 0 && tid == 32 * kKWarp) {
        // test hook: a wait that runs out, so the abort path runs for real
        volatile int never = 0;
        if (!mbar_wait_bounded(&sh.stall_bar, 0, &never, kStallTestCycles)) raise_tree_error(&sh.abort_flag, p.status);
    }
    // the dynamic window starts 1024-byte aligned (the 128-byte swizzle needs it)
    if ((smem_u32(smem_raw) & 1023u) != 0 && tid == 0) raise_tree_error(&sh.abort_flag, p.status);
    if (warp == kKWarp) {
        if (lane == 0) produce_k(maps, p, sh, rank);
    } else if (warp == kQWarp) {
        if (lane == 0) produce_q(maps, p, sh, rank);
    } else if (warp == kMmaWarp) {
        if (rank == 0) issue(p, sh, tmem);
    } else {
        add_weights(p, sh, tmem, rank, tid);
    }
    __syncthreads();
    if (*static_cast<volatile int*>(&sh.abort_flag)) {
        // nothing more is issued by this CTA: let its copies and MMAs end
        const long long t0 = clock64();
        while (clock64() - t0 < kDrainCycles) {
        }
    }
    tc_fence_before_sync();
    cluster_barrier();                                     // orders the threads' last arrivals (s_free), too
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

template <int kBlocks>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(mla_tree_weights_kernel<kBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(Shared<kBlocks>)));
}
template <int kBlocks>
cudaError_t launch_one(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared<kBlocks>);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mla_tree_weights_kernel<kBlocks>, maps, p);
}

}  // namespace

cudaError_t tree_weights_prepare() {
    cudaError_t e = prepare_one<0>();
    if (e == cudaSuccess) e = prepare_one<1>();
    if (e == cudaSuccess) e = prepare_one<2>();
    return e;
}

cudaError_t launch_tree_weights(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream) {
    const int blocks = (p.tokens * p.heads + kTreeBlockRows - 1) / kTreeBlockRows;
    if (blocks == 1) return launch_one<1>(maps, p, pdl, stream);
    if (blocks == 2 && p.a.kv_rows > kTileKeys * p.clusters) return launch_one<2>(maps, p, pdl, stream);
    return launch_one<0>(maps, p, pdl, stream);
}

}  // namespace mla
