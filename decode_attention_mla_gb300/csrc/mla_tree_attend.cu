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
// each, and warps w and w + 4 share lanes: four threads own a row, 32 keys each.  They
// share the row's reference m (its maximum goes through shared memory when it moves)
// and, at a block's end, its sum.
//
// Work split.  The units (request, row block, tile) are cut into equal runs, one
// per pair, from the lengths on the device: no pair idles however ragged the batch.
// Tiles of a run go in an order that keeps the pairs of a request at the same cache
// rows at the same time (TreeCursor).  A run that holds a whole row block writes the
// result; otherwise it leaves a normalised fp32 piece and its log-sum-exp, and
// a second kernel merges the pieces of a block in a fixed order.
//
// Staging, all by TMA: the queries of the row block (72 KB per CTA); K of a tile
// whole (this CTA's 64 keys: four slots of 128 columns, the rope columns beside the
// last), V of a tile whole (this CTA's 256 features of all 128 keys: two halves of
// two slots; the keys of the other CTA's half are L2 hits); P 16 KB.  QK of tile g
// goes before PV of tile g - 1, so the softmax of a tile runs under the next
// tile's QK and the PV before it; at a block's end PV goes first, since the next
// block's QK waits for its queries.
//
// Bound: the tensor cores (an M128 N128 K16 MMA of a pair takes 32 cycles, N256 64;
// a tile 2200), fed at 140 KB per tile and CTA.  Measured in long rows of calls, bf16
// outputs: 64 drafts x 128 heads over 65536 rows 740 us, 1590 TFLOP/s, under the power cap
// (in short rows 647 us, 1810 TFLOP/s or 0.93 of cuBLAS's burst rate); 16 ragged requests
// of 5 x 128 281 us, 1310 TFLOP/s (251 us; DRAM re-reads of row blocks that drift apart);
// 16 x 16 over 131072 rows 65 us; 8 x 16 over 248 rows 11.7 us, of which the two
// kernels' launches, set-up and merge are 10.
//
// Warps of a CTA: 0-7 softmax and epilogue, 8 TMA of Q and K, 9 MMA issue (even
// CTA; the odd one's writes empty requests) and tensor memory, 10 TMA of V.
// Barriers that the MMA warp waits on live in the even CTA and take arrivals of both.
//
// Rounding: O and the statistics are fp32, sums use the unrounded probabilities.  For
// bf16 outputs P enters the product as one bf16: 2^-8 of a probability at most, and on
// average over a row's keys no more than the rounding of the output.  For fp32 outputs
// (kFp32) it enters as a pair, P_hi + P_lo, within 2^-16, as in the decode: a single bf16
// leaves errors of up to 4e-3 over 2 .. 16 rows of normal values.  There is no room for a
// second P, so P_lo takes the buffer once the product with P_hi has read it, and V stays
// until both are done (bf16 / fp32 outputs: 8 x 16 query rows over 248 cache rows 11.9 / 12.8
// us, 1 x 16 over 16384 16.9 / 18.8, 16 x 16 over 131072 63.5 / 82, 16 requests of 5 x 128
// over 16384 240 / 367, 64 x 128 over 65536 650 / 1090).
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
#include <algorithm>
#include <cmath>

#include "mla_tree.cuh"
#include "tc_pair_utils.cuh"

namespace mla {
namespace {

using Cursor = TreeCursor<kTreeTileKeys, true>;

constexpr int kSlots = 4;                                  // of K and of V: a tile each
constexpr uint32_t kSlotBytes = 16384;                     // 2 column chunks of 64 rows x 128 bytes
constexpr uint32_t kChunkBytes = 8192;
constexpr uint32_t kQBytes = 9 * kChunkBytes;
constexpr int kThreads = 352;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kValueWarp = 10;
constexpr int kBarSoftmax = 1;                             // hardware barrier of the softmax warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0, kTmemS = 256;               // O: 2 x 128 columns, S: 2 x 64 columns
constexpr float kRescaleLog2 = 8.0f;                       // move the reference when a max grows past 2^8
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kDrainCycles = 2000ll * 1000ll;        // about 1 ms: time for copies in flight after an abort

struct __align__(1024) Shared {
    uint8_t k[kSlots][kSlotBytes];                         // this CTA's 64 keys x 128 columns, QK operand
    uint8_t v[kSlots][kSlotBytes];                         // (feature half i, key half kb) at 2 i + kb, PV operand
    uint8_t rope[kChunkBytes];                             // this CTA's 64 keys, rope columns
    uint8_t q[kQBytes];                                    // 9 chunks of 64 query rows
    uint8_t p[2][kChunkBytes];                             // P, 64 rows x 128 keys in two key atoms
    float red_max[4][64], red_sum[4][64];                  // by quarter of the tile's keys, row
    // used in the even CTA, arrivals of both
    uint64_t k_ready[kSlots], v_ready[2], q_ready, p_ready, o_free;
    // in each CTA, arrivals of the MMA thread
    uint64_t k_empty[kSlots], v_empty[2], q_empty, s_full[2], o_done;
    uint64_t v_local[2];                                   // V of a tile with drafted rows has landed in this CTA
    uint64_t stall_bar;
    TreeWork work;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Shared) <= 227 * 1024, "fits shared memory");

// ============================== producer ==================================
struct Producer {
    const TreeMaps& maps;
    const TreeParams& p;
    Shared& sh;
    uint32_t rank;
    uint64_t pol_kv, pol_q;
    uint32_t leader;                                       // what turns this CTA's addresses into the even CTA's
    uint32_t specials = 0;

    // The even CTA's barrier of a load; that CTA announces both CTAs' bytes (the odd
    // CTA's may land first: the phase is open until the announcement arrives).
    __device__ __forceinline__ uint32_t expect(uint64_t* bar, uint32_t bytes) {
        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
        return smem_u32(bar) + leader;
    }
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
        return mbar_try_wait(bar, parity) || wait_slowly(bar, parity, &sh.abort_flag);
    }
    __device__ bool load_q(const Cursor& c) {
        if (c.item > 0 && !mbar_wait_bounded(&sh.q_empty, (c.item - 1) & 1, &sh.abort_flag)) return false;
        const int row = c.b * p.tokens * p.heads + c.rb * kTreeBlockRows;
        const int n0 = query_rows(p, row), n1 = query_rows(p, row + 64);
        if (rank == 0) mbar_arrive_expect_tx(&sh.q_ready, (n0 + n1) * (kQBytes / 64));
        load_query_rows<9>(sh.q, maps, row + 64 * static_cast<int>(rank), rank == 0 ? n0 : n1, p.q_tail, 0,
                           smem_u32(&sh.q_ready) + leader, pol_q);
        return true;
    }
    // QK operands: this CTA's 64 keys, 128 columns a slot, the rope columns with the last
    __device__ bool load_k(const Cursor& c) {
        const int y = static_cast<int>(c.r.base) + c.tile * kTreeTileKeys + static_cast<int>(rank) * 64;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            if (c.g > 0 && !wait(&sh.k_empty[s], (c.g - 1) & 1)) return false;
            const uint32_t bar = expect(&sh.k_ready[s], kSlotBytes + (s == 3 ? kChunkBytes : 0));
            tma_load_3d_pair(sh.k[s], &maps.kv, 0, y, 2 * s, bar, pol_kv);
            if (s == 3) tma_load_3d_pair(sh.rope, &maps.rope, 0, y, 8, bar, pol_kv);
        }
        return true;
    }
    // PV operands: features 256 i + 128 rank .. + 127 of the keys of half kb
    __device__ bool load_v(const Cursor& c) {
        const int y = static_cast<int>(c.r.base) + c.tile * kTreeTileKeys;
        const bool special = c.special();
        // (two barriers: the bytes of the next such tile are announced here while the
        // softmax threads may still be waiting for this one's)
        uint64_t* local = &sh.v_local[specials & 1];
        if (special) {
            mbar_arrive_expect_tx(local, 4 * kSlotBytes);
            ++specials;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c.g > 0 && !wait(&sh.v_empty[i], (c.g - 1) & 1)) return false;
            const int z = 4 * i + 2 * static_cast<int>(rank);
            if (special) {
                // the softmax threads wait for these bytes and vouch for them with P
                tma_load_3d(sh.v[2 * i], &maps.kv, 0, y, z, local, pol_kv);
                tma_load_3d(sh.v[2 * i + 1], &maps.kv, 0, y + 64, z, local, pol_kv);
                if (rank == 0) mbar_arrive(&sh.v_ready[i]);
            } else {
                const uint32_t bar = expect(&sh.v_ready[i], 2 * kSlotBytes);
                tma_load_3d_pair(sh.v[2 * i], &maps.kv, 0, y, z, bar, pol_kv);
                tma_load_3d_pair(sh.v[2 * i + 1], &maps.kv, 0, y + 64, z, bar, pol_kv);
            }
        }
        return true;
    }
};

// One thread for the query rows and K, one for V: K of a tile is taken before V
// of the tile before it, so neither waits in the other's queue.
__device__ void produce(const TreeMaps& maps, const TreeParams& p, Shared& sh, uint32_t rank, bool values) {
    Producer pr{maps, p, sh, rank, l2_policy_evict_normal(), l2_policy_evict_normal(),
                map_to_rank(&sh, 0) - smem_u32(&sh)};
    Cursor c;
    bool ok = true;
    for (c.start(p, sh.work); c.left > 0 && ok; c.next(p)) {
        if (values)
            ok = pr.load_v(c);
        else
            ok = (!c.first || pr.load_q(c)) && pr.load_k(c);
    }
    if (!ok) raise_tree_error(&sh.abort_flag, p.status);
}

// ============================== MMA issue ==================================
// One warp issues everything: the tensor pipe takes the MMAs in order, and QK and
// PV interleaved from two warps ran at half the rate.  Its queue is short, so what
// the warp does between two MMAs costs tensor time.  Hence: the whole warp walks
// the tiles and waits, one lane issues (with a single thread doing all of it an
// MMA took 100 cycles to issue, instead of the 32 or 64 that it runs); each
// barrier is looked at once before the MMAs that precede its use, so a phase
// that is over by then costs nothing; and PV is a tile behind QK, so its
// probabilities have had a tile's time.  A buffer is announced as free only to a load that
// will wait for it: no barrier orders the arrival of a commit with the end of the other CTA.
//
// Phases of p_ready and o_done: one per tile, or (kFp32) two, of which P_hi's has
// parity 0 and P_lo's parity 1.
template <bool kFp32>
constexpr int kParts = kFp32 ? 2 : 1;
struct Issue {
    Shared& sh;
    bool lead, ok;

    // after `seen` (an earlier look at the barrier): the phase is over
    __device__ __forceinline__ void need(bool seen, uint64_t* bar, uint32_t parity) {
        if (!seen) ok = wait_slowly(bar, parity, &sh.abort_flag) && ok;
    }
};

template <bool kFp32>
__device__ void issue(const TreeParams& p, Shared& sh, uint32_t tmem) {
    constexpr uint32_t idesc_qk = make_idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idesc_pv = make_idesc_bf16(128, 256, 0, 1);
    Issue is{sh, elect_one(), true};
    const uint64_t kd = make_sdesc(smem_u32(sh.k), 16, 1024, kLayoutSw128);
    const uint64_t vd = make_sdesc(smem_u32(sh.v), kChunkBytes, 1024, kLayoutSw128);
    const uint64_t rope = make_sdesc(smem_u32(sh.rope), 16, 1024, kLayoutSw128);
    const uint64_t q = make_sdesc(smem_u32(sh.q), 16, 1024, kLayoutSw128);
    const uint64_t pd = make_sdesc(smem_u32(sh.p), 16, 1024, kLayoutSw128);
    int item = 0, pv_item = -1;
    Cursor c;                                              // moves from item to item here
    c.start(p, sh.work);
    const int total = c.left;
    int in_item = c.item_left;                             // tiles of the item still to come
    bool first = true;
    uint32_t pv_first = 0;                                 // the tile before this QK's was the first of its item
    // what an early look has shown of the next QK's first barrier and the next PV's
    // (false: not looked at, or not over yet; a look must not block, as try_wait may)
    bool see_k = false, see_p = false, see_v = false;
    for (int g = 0; g <= total && is.ok; ++g) {
        const uint32_t buf = g & 1, par = g & 1;           // of QK(g); PV(g - 1) has the other parity
        const uint32_t qk_first = first;
        // PV of a block's last tile goes first: the next block's QK waits for its queries
        const int pv_turn = first ? 0 : 1;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            if (turn == pv_turn) {
                if (g == 0) continue;
#pragma unroll
                for (int part = 0; part < kParts<kFp32>; ++part) {   // P, or P_hi and P_lo
                    constexpr int kLast = kParts<kFp32> - 1;
                    is.need(see_p, &sh.p_ready, kFp32 ? part : par ^ 1);
                    if (part == 0 && pv_first && ++pv_item > 0) is.need(false, &sh.o_free, (pv_item - 1) & 1);
                    tc_fence_after_sync();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (part == 0) is.need(see_v, &sh.v_ready[i], par ^ 1);
                        if (part == 0 && i == 0)
                            see_v = mbar_test(&sh.v_ready[1], par ^ 1);
                        else if (part == kLast && i == 1)
                            see_k = mbar_test(&sh.k_ready[0], par ^ pv_turn);   // of the QK that comes next
                        if (is.lead && is.ok) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                umma_pair_bf16(tmem + kTmemO + 128 * i,
                                               pd + (((k >> 2) * kChunkBytes + (k & 3) * 32u) >> 4),
                                               vd + (((2 * i + (k >> 2)) * kSlotBytes + (k & 3) * 2048u) >> 4), idesc_pv,
                                               part == 0 && k == 0 ? pv_first ^ 1u : 1u);
                            if (part == kLast && g < total) umma_commit_pair(&sh.v_empty[i]);
                        }
                    }
                    if (is.lead && is.ok) umma_commit_pair(&sh.o_done);
                    see_p = false;
                }
                see_v = false;
            } else {
                if (g == total) continue;
                const uint32_t d = tmem + kTmemS + 64 * buf;
                const bool last = in_item == 1;
                if (first) is.need(false, &sh.q_ready, item & 1);
                // (the scores of tile g - 2 have been read: PV(g - 2) waited for their P)
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    is.need(see_k, &sh.k_ready[s], par);
                    if (s < kSlots - 1) {
                        see_k = mbar_test(&sh.k_ready[s + 1], par);
                    } else if (pv_turn == 1 && g >= 1) {
                        see_p = mbar_test(&sh.p_ready, kFp32 ? 0 : par ^ 1);
                        see_v = mbar_test(&sh.v_ready[0], par ^ 1);
                    }
                    if (is.lead && is.ok) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = ((k >> 2) * kChunkBytes + (k & 3) * 32u) >> 4;
                            umma_pair_bf16(d, q + (2 * s * kChunkBytes >> 4) + off, kd + (s * kSlotBytes >> 4) + off,
                                           idesc_qk, (s | k) ? 1u : 0u);
                        }
                        if (s == 3) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_pair_bf16(d, q + ((8 * kChunkBytes + k * 32u) >> 4), rope + (k * 32u >> 4), idesc_qk,
                                               1u);
                        }
                        if (g + 1 < total) umma_commit_pair(&sh.k_empty[s]);
                    }
                }
                if (is.lead && is.ok) {
                    umma_commit_pair(&sh.s_full[buf]);
                    if (last && g + 1 < total) umma_commit_pair(&sh.q_empty);
                }
                see_k = false;
                first = last;
                if (--in_item == 0 && g + 1 < total) {
                    c.g = g + 1;
                    c.left = total - c.g;
                    c.next_item(p);
                    ++item;
                    in_item = c.item_left;
                }
            }
        }
        pv_first = qk_first;
    }
    if (!is.ok && is.lead) raise_tree_error(&sh.abort_flag, p.status);
}

// ============================== softmax ====================================
__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Clear what must not meet P = 0 in the staged V of a tile: rows behind the
// end, and non-finite values of drafted rows.
__device__ void clean_v(Shared& sh, const Cursor& c, int tid) {
    const int t0 = c.tile * kTreeTileKeys;
    const int from = max(0, c.r.d_pos - t0);
    const int end = min(kTreeTileKeys, c.r.d_pos + c.r.n_tok - t0);   // rows from here on are behind the drafts
    // unit w of a row: 2 feature halves x 2 chunks x 8 units of 16 bytes
    for (int e = tid; e < (kTreeTileKeys - from) * 32; e += kSoftmaxThreads) {
        const int key = from + (e >> 5), w = e & 31;
        uint8_t* slot = sh.v[2 * (w >> 4) + (key >> 6)];
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

// Place of a piece's feature quad: [slot][32-row group][quad][row], so that the
// epilogue's and the merge's warps (a row per lane) touch 512 consecutive bytes.
// (Rows of 2 KB, staged through shared memory, took 6300 cycles per row block.)
__device__ __forceinline__ long long piece_quad(int slot, int row, int quad, int groups = kTreeBlockRows / 32) {
    return ((static_cast<long long>(slot) * groups + (row >> 5)) * (kDLatent / 4) + quad) * 32 + (row & 31);
}

// 64 bytes of each of a warp's 32 rows (32 features in bf16, 16 in fp32),
// through its 2 KB of shared memory so that the stores of a row run along its
// features (16-byte units, swizzled by row pair).  `dst`: row 0's first
// feature, rows 512 elements apart; rows at or past n_rows are not written.
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t (&w)[16], char* dst, int row_bytes,
                                           int n_rows, int lane) {
    __syncwarp();                                          // the reads of the block before are done
#pragma unroll
    for (int u = 0; u < 4; ++u)
        st_shared_v4(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4), w[4 * u], w[4 * u + 1], w[4 * u + 2],
                     w[4 * u + 3]);
    __syncwarp();
    const int u = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
        const uint4 v = ld_shared_v4(stage + row * 64 + ((u ^ ((row >> 1) & 3)) << 4));
        if (row < n_rows) reinterpret_cast<uint4*>(dst + static_cast<long long>(row) * row_bytes)[u] = v;
    }
}

// Thread: 32 keys of one row.  Warps w and w + 4 share tensor-memory lanes 32 (w mod 4) ..
// and split their columns.
template <bool kFp32>
__device__ void softmax(const TreeParams& p, Shared& sh, uint32_t tmem, uint32_t rank, int cluster, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const int sub = warp >> 2, half = (warp >> 1) & 1;     // keys 64 half + 32 sub ..; features 256 sub + 128 half ..
    const int quarter = 2 * half + sub;
    const int row = 32 * (warp & 1) + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t p_bar = map_to_rank(&sh.p_ready, 0), o_bar = map_to_rank(&sh.o_free, 0);
    const uint32_t p_line = smem_u32(sh.p[half]) + row * 128;
    const float c2 = p.scale_log2;
    uint32_t specials = 0;
    bool ok = true, bad = false;
    const bool notes = rank == 0 && tid == 0;
    if (notes)
        for (int i = 0; i < kTreePieces; ++i) p.merge[i * p.clusters + cluster].pieces = 0;
    Cursor c;
    c.start(p, sh.work);
    while (c.left > 0 && ok) {
        // ---- one item: tiles of one row block
        const int r = c.rb * kTreeBlockRows + static_cast<int>(rank) * 64 + row;
        const int live_rows = c.r.n_tok * p.heads;
        const unsigned long long mask = r < live_rows ? tree_mask(p, c.b, r / p.heads, c.r.n_tok) : 0ull;
        const int b = c.b, rb = c.rb;
        const bool whole = c.whole(), run_first = c.g == 0;
        const bool opens = !whole && c.seg == 0 && c.opens(), cut = c.sg.count() > 1;
        const TreeCut of{c.n_rb, c.n_tiles, static_cast<int>(sh.work.per), c.begin};
        float m_ref = -INFINITY, l = 0.f;
        bool last;
        do {
            const int g = c.g, buf = g & 1;
            last = c.last();
            bool w = warp_wait(&sh.abort_flag, &sh.s_full[buf], (g >> 1) & 1);
            uint32_t s[32];
            if (w) {
                tmem_ld32_async(tmem + lanes + kTmemS + 64 * buf + 32 * sub, s);
                tmem_wait_ld32(s);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = 0;
            }
            const int t0 = c.tile * kTreeTileKeys;
            if (t0 + kTreeTileKeys > c.r.d_pos || t0 < c.r.lo || t0 + kTreeTileKeys > c.r.hi) {
                const uint32_t v = static_cast<uint32_t>(visible64(c.r, mask, t0 + 64 * half) >> (32 * sub));
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!(v >> i & 1)) s[i] = 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
            float alpha = 1.f;
            bad |= !w;
            if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad || top > m_ref + kRescaleLog2)) {
                // rare after the first tile: the row's maximum moves the reference
                sh.red_max[quarter][row] = top;
                if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad)) {
                    ok = false;
                    break;
                }
                const float tm = fmaxf(fmaxf(sh.red_max[0][row], sh.red_max[1][row]),
                                       fmaxf(sh.red_max[2][row], sh.red_max[3][row]));
                if (tm > m_ref + kRescaleLog2) {
                    if (m_ref > -INFINITY) alpha = ex2_approx(m_ref - tm);
                    m_ref = tm;
                }
                l *= alpha;
            }
            const float base = m_ref > -INFINITY ? m_ref : 0.f;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pk[16], rest[16];                     // (rest: kFp32 alone)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = ex2_approx(fmaf(__uint_as_float(s[2 * i]), c2, -base));
                const float y = ex2_approx(fmaf(__uint_as_float(s[2 * i + 1]), c2, -base));
                sum[i & 1] += x;
                sum[2 + (i & 1)] += y;
                if constexpr (kFp32)
                    split_bf16x2(x, y, pk[i], rest[i]);
                else
                    pk[i] = pack_bf16x2(x, y);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            // P of the tile before has been read, and O holds all tiles before this one
            w = g == 0 || warp_wait(&sh.abort_flag, &sh.o_done, kFp32 ? 1 : (g - 1) & 1);
            if (w && __any_sync(0xffffffffu, alpha != 1.f)) {   // (never on an item's first tile)
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    float o[16];
                    const uint32_t at = tmem + lanes + kTmemO + 128 * sub + 16 * j;
                    tmem_ld16(at, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] *= alpha;
                    tmem_st16(at, o);
                }
            }
            // ---- probabilities, bf16, K-major lines of 64 keys
            auto store_p = [&](const uint32_t (&v)[16]) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    st_shared_v4(p_line + (((4 * sub + u) ^ (row & 7)) << 4), v[4 * u], v[4 * u + 1], v[4 * u + 2],
                                 v[4 * u + 3]);
            };
            auto hand_over = [&] {
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                bad |= !w;                                 // the threads leave together at the next barrier
                if (lane == 0 && !bad) mbar_arrive_peer(p_bar);
            };
            store_p(pk);
            if (c.special()) {
                // V was loaded for this CTA's own eyes
                w = w && warp_wait(&sh.abort_flag, &sh.v_local[specials & 1], (specials >> 1) & 1);
                ++specials;
                if (w) clean_v(sh, c, tid);
            }
            hand_over();
            if (kFp32 && !bad) {
                w = warp_wait(&sh.abort_flag, &sh.o_done, 0);   // P_hi has been read
                store_p(rest);
                hand_over();
            }
            c.next(p);
        } while (!last);
        if (!ok) break;

        // ---- epilogue: l of the four quarters, O / l, log-sum-exp
        sh.red_sum[quarter][row] = l;
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad)) {
            ok = false;
            break;
        }
        const float lt = (sh.red_sum[0][row] + sh.red_sum[1][row]) + (sh.red_sum[2][row] + sh.red_sum[3][row]);
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        const float lse2 = lt == 0.f ? -INFINITY : m_ref + log2f(lt);
        // place of the piece: the run's first item, one that ends with the run's length, another
        const int place = run_first ? 0 : c.g == sh.work.per ? 2 : 1, slot = kTreePieces * cluster + place;
        if (quarter == 0 && r < live_rows) {
            if (whole)
                p.a.lse[static_cast<long long>(b) * p.tokens * p.heads + r] = lse2 * kLn2;
            else
                p.lse_part[slot * kTreeBlockRows + static_cast<int>(rank) * 64 + row] = lse2;
        }
        if (notes && opens) {
            const int rows = min(kTreeBlockRows, live_rows - rb * kTreeBlockRows);
            // (an uncut job's pieces lie in the runs from this one to that of its last unit)
            const int pieces = cut ? -1 : (of.begin + (rb + 1) * of.n_tiles - 1) / of.per + 1;
            const int at = (cut ? place : 0) * p.clusters + cluster;
            p.merge[at] = TreeMerge{b, rb, rows | place << 16, pieces};
            if (cut) p.cut[at] = of;
        }
        const bool w = warp_wait(&sh.abort_flag, &sh.o_done, kFp32 ? 1 : (c.g - 1) & 1);
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, !w)) {
            ok = false;
            break;
        }
        // (P's buffer is free: the last product is done)
        const uint32_t stage = smem_u32(sh.p) + warp * 2048;
        const int row_w = 32 * (warp & 1);                 // this warp's first row of the 64
        const int n_rows = live_rows - (r - row) - row_w;
        const int f0 = 256 * sub + 128 * half;             // its first feature
        float4* piece = reinterpret_cast<float4*>(p.part) +
                        piece_quad(slot, static_cast<int>(rank) * 64 + row_w, f0 / 4) + lane;
        char* out = static_cast<char*>(p.a.out) +
                    ((static_cast<long long>(b) * p.tokens * p.heads + r - row + row_w) * kDLatent + f0) *
                        (kFp32 ? 4 : 2);
#pragma unroll 1
        for (int j = 0; j < 4 && n_rows > 0; ++j) {        // (the merge reads groups with live rows only)
            uint32_t o[32];
            tmem_ld32_async(tmem + lanes + kTmemO + 128 * sub + 32 * j, o);
            tmem_wait_ld32(o);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    piece[(8 * j + i) * 32] =
                        make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                    __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                continue;
            }
            uint32_t x[16];
            if constexpr (!kFp32) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                store_rows(stage, x, out + 64 * j, 2 * kDLatent, n_rows, lane);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(o[16 * h + i]) * inv);
                    store_rows(stage, x, out + 128 * j + 64 * h, 4 * kDLatent, n_rows, lane);
                }
            }
        }
        tc_fence_before_sync();
        __syncwarp();
        // O may be overwritten.  (Only if something will wait for it, as for the buffers: the
        // closing barrier orders no arrival.)
        if (lane == 0 && c.left > 0) mbar_arrive_peer(o_bar);
    }
    if (!ok && lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

// Requests without rows: their tokens' outputs, by the odd CTAs' otherwise idle warp.
__device__ void write_empty(const TreeParams& p, int cluster, int clusters, int lane) {
    for (int b = cluster; b < p.batch; b += clusters) {
        const TreeRequest r = load_tree_request(p, b);
        if (r.hi > 0 || r.n_tok == 0) continue;
        const long long row0 = static_cast<long long>(b) * p.tokens * p.heads;
        const int rows = r.n_tok * p.heads;
        for (int i = lane; i < rows; i += 32) p.a.lse[row0 + i] = -INFINITY;
        const int per = p.a.out_fp32 ? 128 : 64;           // 16-byte units per row
        uint4* o = reinterpret_cast<uint4*>(p.a.out) + row0 * per;
        for (int i = lane; i < rows * per; i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
}

template <bool kFp32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_tree_attend_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    if (tid == 0) {
        prefetch_tensormap(&maps.kv);
        prefetch_tensormap(&maps.rope);
        prefetch_tensormap(&maps.q);
        if (p.q_tail < 64) prefetch_tensormap(&maps.q_tail);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.k_ready[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.v_ready[i], 1);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.v_local[i], 1);
        }
        mbar_init(&sh.p_ready, 2 * kSoftmaxWarps);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.q_ready, 1);
        mbar_init(&sh.o_free, 2 * kSoftmaxWarps);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    __syncwarp();
    cluster_arrive();                                      // (after this thread's barrier initialisation)
    if (warp == kMmaWarp) tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == kProducerWarp) Cursor::find_work(p, cluster, lane, &sh.work);
    tc_fence_before_sync();
    __syncthreads();
    cluster_wait();                                        // both CTAs' barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    if (p.stall_test && blockIdx.x == 0 && tid == 32 * kProducerWarp) {
        // test hook: a wait that runs out, so the abort path runs for real
        volatile int never = 0;
        if (!mbar_wait_bounded(&sh.stall_bar, 0, &never, kStallTestCycles)) raise_tree_error(&sh.abort_flag, p.status);
    }
    // the dynamic window starts 1024-byte aligned (the 128-byte swizzle needs it)
    if ((smem_u32(smem_raw) & 1023u) != 0 && tid == 0) raise_tree_error(&sh.abort_flag, p.status);
    if (warp == kProducerWarp) {
        if (lane == 0) produce(maps, p, sh, rank, false);
    } else if (warp == kValueWarp) {
        if (lane == 0) produce(maps, p, sh, rank, true);
    } else if (warp == kMmaWarp) {
        if (rank == 0)
            issue<kFp32>(p, sh, tmem);
        else
            write_empty(p, cluster, p.clusters, lane);
    } else {
        softmax<kFp32>(p, sh, tmem, rank, cluster, tid);
    }
    __syncthreads();
    if (*static_cast<volatile int*>(&sh.abort_flag)) {
        // nothing more is issued by this CTA: let its copies and MMAs end
        const long long t0 = clock64();
        while (clock64() - t0 < kDrainCycles) {
        }
    }
    tc_fence_before_sync();
    cluster_barrier_relaxed();                             // neither CTA's shared memory goes before both are done
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ============================== merge ======================================
// Out of the clusters' notes, block x takes the x-th row block that several runs
// share.  A warp: 32 rows (one per lane) and QUADS feature quads; the pieces in a
// fixed order, a batch of loads in flight at a time, with a running maximum of
// their log-sum-exps.  With few pieces a warp takes four quads (a lane's output is
// a whole sector); with many, one quad, and four warps share the pieces and join
// their sums in order (the pieces come from L2: 76 of them in one warp's hands
// took three times as long).
constexpr int kMergeWarps = 8;
// Up to about so many pieces per block: four quads per warp.  Measured on whole calls,
// four quads / shared pieces: 8 blocks (10 pieces) 22.5 / 27.1 us, 6 blocks (13) 28.6 /
// 30.2, 5 blocks (15) 40.8 / 40.6, 4 blocks (19) 27.8 / 26.0, 2 blocks (38) 28.9 / 20.8.
constexpr int kFewPieces = 15;

constexpr int kMergeList = 256;

// Candidates for the pieces of row block rb in segments: part c mod 3 of segment c / 3.
__device__ __forceinline__ int cut_candidates(const TreeCut& m) {
    TreeSegments sg;
    sg.set(m.n_tiles, m.n_rb, m.per);
    return 3 * sg.count();
}
// One warp: the slots of the pieces among candidates c0 .. c0 + kMergeList - 1.
__device__ __noinline__ int list_cut_pieces(const TreeCut& m, int rb, int cluster, int c0, int lane, int* list) {
    TreeSegments sg;
    sg.set(m.n_tiles, m.n_rb, m.per);
    const int all = min(3 * sg.count(), c0 + kMergeList);
    int n = 0;
    for (int c = c0; c < all; c += 32) {
        const int at = c + lane, seg = at / 3, part = at - 3 * seg;
        // units of the job, relative to the first of the run that opens the row block
        const int s0 = m.begin + m.n_rb * sg.start(seg) + rb * sg.tiles(seg), s1 = s0 + sg.tiles(seg);
        const int run = s0 / m.per, run_end = (run + 1) * m.per;
        const bool is = at < all && s1 > run_end + (part - 1) * m.per;
        const uint32_t bal = __ballot_sync(0xffffffffu, is);
        if (is)
            list[n + __popc(bal & ((1u << lane) - 1u))] =
                kTreePieces * (cluster + run + part) + (part > 0 || s0 == run * m.per ? 0 : s1 >= run_end ? 2 : 1);
        n += __popc(bal);
    }
    return n;
}

template <int QUADS, int PARTS>
__global__ void __launch_bounds__(32 * kMergeWarps) mla_tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kBatch = QUADS == 1 ? 10 : 4;
    __shared__ TreeMerge note;
    __shared__ int owner;
    __shared__ int list[kMergeList];                       // slots of pieces in segments, in order
    __shared__ int listed;
    __shared__ float joined[PARTS > 1 ? kMergeWarps : 1][6][32];   // maximum, sum, four features
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) {
        const int notes = kTreePieces * p.clusters;
        int seen = 0;
        bool found = false;
        for (int c = 0; c < notes && !found; c += 128) {
            TreeMerge n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = c + 32 * i + lane;
                n[i] = p.merge[min(at, notes - 1)];
                if (at >= notes) n[i].pieces = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bal = __ballot_sync(0xffffffffu, n[i].pieces != 0);
                const int rank = seen + __popc(bal & ((1u << lane) - 1u));
                if (n[i].pieces != 0 && rank == static_cast<int>(blockIdx.x)) {
                    note = n[i];
                    owner = c + 32 * i + lane;
                }
                seen += __popc(bal);
            }
            found = seen > static_cast<int>(blockIdx.x);
        }
        if (!found && lane == 0) owner = -1;
    }
    __syncthreads();
    if (owner < 0) return;
    const TreeMerge m = note;
    const int rows = m.rows & 0xffff;
    const bool cut = m.pieces < 0;
    int cluster = owner;                                   // whose run opens the row block
    while (cluster >= p.clusters) cluster -= p.clusters;
    // slot of a piece; pieces in segments are listed, kMergeList candidates at a time
    auto slot = [&](int i) {
        return cut ? list[i] : kTreePieces * (cluster + i) + (i == 0 ? m.rows >> 16 : 0);
    };
    auto list_pieces = [&](int c0) {
        if (warp == 0) {
            const int n = list_cut_pieces(p.cut[owner], m.rb, cluster, c0, lane, list);
            if (lane == 0) listed = n;
        }
        __syncthreads();
    };
    const int candidates = cut ? cut_candidates(p.cut[owner]) : 0;
    if (cut) list_pieces(0);
    constexpr int kQuadWarps = kMergeWarps / PARTS;        // warps of a block with quads of their own
    constexpr int kTasks = kDLatent / 4 / QUADS / kQuadWarps;   // blocks per 32 rows
    const int group = static_cast<int>(blockIdx.y) / kTasks;
    const int part_of = warp / kQuadWarps;                 // share of the pieces
    const int quad = ((static_cast<int>(blockIdx.y) % kTasks) * kQuadWarps + warp % kQuadWarps) * QUADS;
    const int row = 32 * group + lane;
    const bool live = row < rows;
    const int groups = (p.block_rows + 31) >> 5;           // of 32 rows, per piece
    if (32 * group >= rows) return;                      // uniform over the block
    const float4* part = reinterpret_cast<const float4*>(p.part);
    float4 acc[QUADS];
#pragma unroll
    for (int k = 0; k < QUADS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, top = -INFINITY, base = 0.f;
    for (int c0 = 0;; c0 += kMergeList) {
        const int n = cut ? listed : m.pieces;
        const int share = (n + PARTS - 1) / PARTS;
        const int end = min(n, (part_of + 1) * share);
        for (int i0 = part_of * share; i0 < end; i0 += kBatch) {
            float l[kBatch];
            float4 v[kBatch][QUADS];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = slot(min(i0 + i, end - 1));     // (no branch: all loads at once)
                l[i] = live ? p.lse_part[at * (32 * groups) + row] : -INFINITY;
                const float4* src = part + piece_quad(at, row, quad, groups);
#pragma unroll
                for (int k = 0; k < QUADS; ++k) v[i][k] = src[32 * k];
            }
            const float before = top;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) top = fmaxf(top, l[i]);   // (the repeated last piece changes nothing)
            if (top > before) {
                const float scale = before > -INFINITY ? exp2f(before - top) : 0.f;
                base = top;
                // (a NaN stays: a product with 0 only drops sums of nothing)
                if (before > -INFINITY || sum != 0.f) {
                    sum *= scale;
#pragma unroll
                    for (int k = 0; k < QUADS; ++k)
                        acc[k] = make_float4(acc[k].x * scale, acc[k].y * scale, acc[k].z * scale, acc[k].w * scale);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < end) {
                    const float w = exp2f(l[i] - base);        // NaN stays NaN
                    sum += w;
#pragma unroll
                    for (int k = 0; k < QUADS; ++k) {
                        acc[k].x = fmaf(w, v[i][k].x, acc[k].x);
                        acc[k].y = fmaf(w, v[i][k].y, acc[k].y);
                        acc[k].z = fmaf(w, v[i][k].z, acc[k].z);
                        acc[k].w = fmaf(w, v[i][k].w, acc[k].w);
                    }
                }
        }
        if (c0 + kMergeList >= candidates) break;          // (uniform)
        __syncthreads();
        list_pieces(c0 + kMergeList);
    }
    if constexpr (PARTS > 1) {
        static_assert(QUADS == 1, "one quad per warp where warps share pieces");
        const float mine[6] = {top, sum, acc[0].x, acc[0].y, acc[0].z, acc[0].w};
#pragma unroll
        for (int k = 0; k < 6; ++k) joined[warp][k][lane] = mine[k];
        __syncthreads();
        if (part_of != 0) return;
        float t[PARTS];
        top = -INFINITY;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            t[q] = joined[warp + q * kQuadWarps][0][lane];
            top = fmaxf(top, t[q]);
        }
        base = top > -INFINITY ? top : 0.f;
        sum = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            const float(&from)[6][32] = joined[warp + q * kQuadWarps];
            // (a share whose maximum is -infinity has the sum 0, or a NaN)
            const float w = t[q] > -INFINITY ? exp2f(t[q] - base) : 1.f;
            sum = fmaf(w, from[1][lane], sum);
            acc[0].x = fmaf(w, from[2][lane], acc[0].x);
            acc[0].y = fmaf(w, from[3][lane], acc[0].y);
            acc[0].z = fmaf(w, from[4][lane], acc[0].z);
            acc[0].w = fmaf(w, from[5][lane], acc[0].w);
        }
    }
    if (!live) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long out_row =
        static_cast<long long>(m.b) * p.tokens * p.heads + static_cast<long long>(m.rb) * p.block_rows + row;
    if (quad == 0) p.a.lse[out_row] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
#pragma unroll
    for (int k = 0; k < QUADS; ++k) {
        const float4 v = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
        const long long at = out_row * kDLatent + 4 * (quad + k);
        if (p.a.out_fp32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) = v;
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

}  // namespace

cudaError_t tree_attend_prepare() {
    for (auto kernel : {mla_tree_attend_kernel<false>, mla_tree_attend_kernel<true>}) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared)));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_tree_attend(const TreeMaps& maps, const TreeParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cudaError_t e =
        cudaLaunchKernelEx(&cfg, p.a.out_fp32 ? mla_tree_attend_kernel<true> : mla_tree_attend_kernel<false>, maps, p);
    if (e != cudaSuccess) return e;
    return launch_tree_merge(p, pdl, stream);
}

cudaError_t launch_tree_merge(const TreeParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    // shared row blocks: no more than there are row blocks or notes, and without
    // segments (one block per request) at most one per run
    const int per_request = (p.tokens * p.heads + p.block_rows - 1) / p.block_rows;
    const long long blocks = static_cast<long long>(p.batch) * per_request;
    const unsigned items =
        static_cast<unsigned>(std::min<long long>((per_request > 1 ? kTreePieces : 1) * p.clusters, blocks));
    const int groups = (std::min(p.tokens * p.heads, p.block_rows) + 31) / 32;
    cfg.blockDim = dim3(32 * kMergeWarps);
    // a row block has about clusters / blocks pieces
    if (p.clusters > kFewPieces * blocks) {
        cfg.gridDim = dim3(items, groups * (kDLatent / 4 / (kMergeWarps / 4)));
        return cudaLaunchKernelEx(&cfg, mla_tree_merge_kernel<1, 4>, p);
    }
    cfg.gridDim = dim3(items, groups * (kDLatent / 16 / kMergeWarps));
    return cudaLaunchKernelEx(&cfg, mla_tree_merge_kernel<4, 1>, p);
}

}  // namespace mla
