// mla_paged_attend.cu -- attention over the 4-bit paged cache on pairs of SMs
// (tcgen05 cta_group::2, tensor memory), rows widened on their way to the tensor
// cores (include/mla_paged.h).
//
// The matrices, the split into runs of tiles, the pieces and their merge are those of
// mla_tree_attend.cu: query rows (token * heads + head) in blocks of 128, 64 per CTA
// of a pair; tiles of 128 cache rows; S = Q K^T in two tensor-memory buffers, O (64 x
// 512 fp32 per CTA) in 256 columns; a run of tiles per pair.  What differs:
//
// Operands.  A latent value is code * scale * kv_scale; code * scale has six
// significant bits and lies between 2^-10 and 2688, so it is exact in f16.  Eight warps
// per CTA write the tiles' operands in the swizzled layout, slots of 64 rows x 128 columns: K (this CTA's rows,
// four slots) and V (the tile's rows, this CTA's 256 features, four slots).  The rows' bytes come by TMA
// into the slot itself, pass through registers, and go back widened (one conversion and one product per two
// values): there is no room for them beside the operands.  (Through registers alone, by loads of 16 bytes a
// lane a tile ahead: 507 us where this form takes 326 for 16 requests of 4 x 128; the loads in flight do not
// fit what shared memory leaves of L1.)  The key values stay bf16 and are multiplied with bf16
// queries, into the same accumulators; they land in their place, and rows are called to L2 three tiles ahead.
// q_lat goes to f16, the whole query row times a power of two that brings its largest value to
// 2^14 .. 2^15 (values down to 2^-31 of it stay exact); the scores' factor takes it back.
//
// Rounding: P enters the product as one f16 of 2^7 times the probability (relative to the reference,
// which lags the maximum by 2^8 at most: at most 2^15), off by up to 2^-11 each (below 2^-21 of the reference,
// where f16 is subnormal, by up to 2^-32 of it); bf16 and fp32 outputs are the same product, so an fp32 output is not closer than
// that.  O and the statistics are fp32, sums use the unrounded probabilities.
//
// What a token does not attend must not reach it: masked scores become -infinity and P = 0; the
// only value of V that is not finite, an E4M3 scale's NaN, becomes 0 there (a token that attends such
// a row has a NaN score from K, where it stays).  Rows without a page are zeros, and masked: the
// softmax warps read the tile's page numbers themselves.
//
// Bound: shared memory.  A tile takes 4100 .. 4400 cycles.  Its products are 2200 on the tensor cores; what passes through
// a CTA's shared memory for it is 470 KB, 3650 cycles at 128 bytes: 240 KB of operands that the MMAs read, 128 of widened
// values written, 48 by TMA, 36 read to be widened, 16 of P.  16 requests of 4 x 128 rows over 4096 .. 32768 rows 312 us, 1140
// TFLOP/s; 16 of up to 2 x 128 rows that see 4096 rows 63 us, of which 12 pass before the first scores (the run is found,
// queries and first rows arrive) and 10 behind the last ones (epilogue, merge).
//
// Every wait is bounded; a wait that runs out raises MLA_EDEVICE in the status word, both CTAs
// leave their loops and meet at a cluster barrier.
//
// Warps of a CTA: 0 MMA issue (even CTA; the odd one's writes empty requests) and tensor memory, 1 TMA of K, 2 TMA of V,
// 3 the items of the run, 4-11 softmax and epilogue, 12-19 operands and queries.  Barriers that the MMA warp waits
// on live in the even CTA and take arrivals of both.
#include <cmath>

#include "mla_paged.cuh"
#include "tc_pair_utils.cuh"

namespace mla {
namespace {

using Cursor = TreeCursor<kTreeTileKeys, true, PagedParams>;

constexpr int kSlots = 4;                                  // of K and of V: a tile each
constexpr uint32_t kSlotBytes = 16384;                     // 2 column chunks of 64 rows x 128 bytes
constexpr uint32_t kChunkBytes = 8192;
constexpr uint32_t kQBytes = 9 * kChunkBytes;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = 0, kKeyWarp = 1, kValueWarp = 2, kScoutWarp = 3;
constexpr int kSoftmaxWarp = 4, kFillWarp = 12, kFillWarps = 8;
constexpr int kItemReaders = kSoftmaxWarps + kFillWarps + 2;   // and the even CTA's MMA warp
constexpr int kThreads = 640;
constexpr int kBarSoftmax = 1;                             // hardware barrier of the softmax warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0, kTmemS = 256;               // O: 2 x 128 columns, S: 2 x 64 columns
constexpr float kRescaleLog2 = 8.0f;                       // move the reference when a max grows past 2^8
constexpr float kProbLog2 = 7.0f;                          // P is held times 2^7
constexpr float kLn2 = 0.6931471805599453f;
constexpr long long kDrainCycles = 2000ll * 1000ll;        // about 1 ms: time for copies and MMAs in flight after an abort

// What one run does of a job (see TreeCursor), for the warps that work on it.
struct __align__(16) Item {
    int b, lo, hi, tile;                                   // tiles lo .. hi - 1, from `tile` on and round
    int near, skip, d_pos, n_tok;                          // as r.lo, r.base of the request, and its own
    int rb, flags, n_rb, n_tiles;
    int begin, unused[3];
};
constexpr int kWhole = 1, kOpens = 2, kCut = 4;
constexpr int kItems = 4;

struct __align__(1024) Shared {
    uint8_t k[kSlots][kSlotBytes];                         // this CTA's 64 keys x 128 columns, QK operand
    uint8_t v[kSlots][kSlotBytes];                         // (feature half i, key half kb) at 2 i + kb, PV operand
    uint8_t rope[kChunkBytes];                             // this CTA's 64 keys, rope columns (bf16)
    uint8_t q[kQBytes];                                    // 9 chunks of 64 query rows (f16, the last bf16)
    uint8_t p[2][kChunkBytes];                             // P, 64 rows x 128 keys in two key atoms
    float red_max[4][64], red_sum[4][64];                  // by quarter of the tile's keys, row
    Item items[kItems];                                    // by item mod kItems
    int8_t factor_exp[4][64];                              // by item mod 4: of a query row's scores, as of factor_exp()
    // used in the even CTA, arrivals of both
    uint64_t k_ready[kSlots], rope_ready, v_ready[2], q_ready, p_ready, o_free;
    // in each CTA, arrivals of the MMA thread
    uint64_t k_empty[kSlots], v_empty[2], q_empty, s_full[2], o_done;
    uint64_t k_raw[kSlots], v_raw[kSlots];                 // a slot's bytes have landed in it
    // this CTA's query rows are there, by item mod 2 (those of an item may be there before the softmax
    // warps have come to the one before)
    uint64_t q_local[2];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t stall_bar;
    TreeWork work;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Shared) <= 227 * 1024, "fits shared memory");

// ============================== items ====================================
// One warp walks the run and lays its items out, a few ahead; the others need
// few registers for their place in it.
__device__ void scout(const PagedParams& p, Shared& sh, int lane) {
    Cursor c;
    c.start(p, sh.work);
    while (c.left > 0) {
        if (c.item >= kItems &&
            !warp_wait(&sh.abort_flag, &sh.item_empty[c.item % kItems], (c.item / kItems - 1) & 1)) {
            if (lane == 0) raise_tree_error(&sh.abort_flag, p.status);
            return;
        }
        if (lane == 0) {
            Item& i = sh.items[c.item % kItems];
            i.b = c.b;
            i.lo = c.lo;
            i.hi = c.hi;
            i.tile = c.tile;
            i.near = c.r.lo;
            i.skip = static_cast<int>(c.r.base);
            i.d_pos = c.r.d_pos;
            i.n_tok = c.r.n_tok;
            i.rb = c.rb;
            i.flags = (c.whole() ? kWhole : 0) | (!c.whole() && c.seg == 0 && c.opens() ? kOpens : 0) |
                      (c.sg.count() > 1 ? kCut : 0);
            i.n_rb = c.n_rb;
            i.n_tiles = c.n_tiles;
            i.begin = c.begin;
            mbar_arrive(&sh.item_full[c.item % kItems]);
        }
        __syncwarp();
        const int n = c.item_left;
        c.g += n;
        c.left -= n;
        ++c.item;
        if (c.left > 0) c.next_item(p);
    }
}

// A warp's place in the run: tile `tile` of item `item`, the g-th of the run.
struct Walk {
    int g, left;                                           // tiles before it, and from it on
    int item, in_item;                                     // tiles of the item from it on
    int tile, lo, hi, near, skip, b;
    bool first;                                            // first tile of its item

    __device__ __forceinline__ bool enter(Shared& sh) {
        first = true;
        if (!warp_wait(&sh.abort_flag, &sh.item_full[item % kItems], (item / kItems) & 1)) return false;
        const Item& i = sh.items[item % kItems];
        b = i.b;
        lo = i.lo;
        hi = i.hi;
        tile = i.tile;
        near = i.near;
        skip = i.skip;
        in_item = hi - lo;
        return true;
    }
    // false: a wait ran out
    __device__ __forceinline__ bool start(Shared& sh) {
        g = item = 0;
        left = static_cast<int>(sh.work.count);
        return left <= 0 || enter(sh);
    }
    __device__ __forceinline__ bool next(Shared& sh) {
        ++g;
        --left;
        first = --in_item == 0;
        if (!first) {
            if (++tile == hi) tile = lo;
            return true;
        }
        ++item;
        return left <= 0 || enter(sh);
    }
    // first row of the tile
    __device__ __forceinline__ int row() const { return (tile < near ? tile : tile + skip) * kTreeTileKeys; }
    // this warp needs nothing more of the item's description
    static __device__ __forceinline__ void release(Shared& sh, int item, int lane) {
        if (lane == 0) mbar_arrive(&sh.item_empty[item % kItems]);
    }
};

// ============================== operands ==================================
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t low_half_twice(uint32_t v) { return __byte_perm(v, v, 0x1010); }
__device__ __forceinline__ uint32_t high_half_twice(uint32_t v) { return __byte_perm(v, v, 0x3232); }

// Rows per box: a page's, 32 at most.
__device__ __forceinline__ int box_rows(const PagedCache& c) { return min(1 << c.row_shift, 32); }

// One slot: 64 rows (half a tile) x 128 features.  The rows' bytes land in the slot itself, where 32 rows' widened
// values go to: their codes, 64 bytes a row (64-byte swizzled), in the first of their two 4 KB pieces, 16 bytes of scales
// a row, of which eight are the slot's, in the second.  One warp takes these to registers, all of them, and writes
// the widened values over them.
constexpr uint32_t kHalfBytes = 4096;                      // 32 rows of a chunk
constexpr uint32_t kRawBytes = 64 * (64 + 16);

__device__ __forceinline__ void widen_half(uint32_t piece, int scale_byte, bool clean, int lane) {
    const int row = lane & 7, unit = lane >> 3;            // of eight rows; 32 features
    uint4 raw[4];
    uint32_t scales[4];
    // (64-byte swizzle: 16-byte unit u of row r lies at u ^ (r / 2 mod 4))
    const uint32_t from = piece + row * 64 + ((unit ^ ((row >> 1) & 3)) << 4);
    const uint32_t scale_from = piece + kChunkBytes + row * 16 + scale_byte + 2 * unit;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        raw[n] = ld_shared_v4(from + n * 512);
        scales[n] = ld_shared_u16(scale_from + n * 128);
    }
    __syncwarp();                                          // every lane has its bytes: they may be overwritten
    const uint32_t line = piece + (unit >> 1) * kChunkBytes + row * 128;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t s = widen_e4m3(static_cast<uint16_t>(scales[n]));
        if (clean) s &= __heq2_mask(*reinterpret_cast<__half2*>(&s), *reinterpret_cast<__half2*>(&s));
        const uint32_t lo = low_half_twice(s), hi = high_half_twice(s);
        const uint32_t w[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            widen_e2m1(w[i], h);
            const uint32_t f = i < 2 ? lo : hi;
            st_shared_v4(line + n * 1024 + (((4 * (unit & 1) + i) ^ row) << 4), mul_f16x2(h[0], f), mul_f16x2(h[1], f),
                         mul_f16x2(h[2], f), mul_f16x2(h[3], f));
        }
    }
}

// Writes that the tensor cores of this SM read: announced to the even CTA's barrier.
__device__ __forceinline__ void hand_over(uint32_t bar, int lane) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_peer(bar);
}

// This warp's eight query rows (of the CTA's 64): copied, then times a power of two in place,
// latents in f16.  `live` of them, from row0 of the tensor on.
__device__ __forceinline__ void fill_queries(const PagedParams& p, Shared& sh, long long row0, int live, int item, int fill,
                                             int lane) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + row0 * kDRow) + lane;
    const uint32_t q = smem_u32(sh.q);
    // unit 32 k + lane of a row: chunk 4 k + lane / 8
    const uint32_t dst = q + (lane >> 3) * kChunkBytes;
#pragma unroll 1
    for (int i = 0; i < live; ++i) {
        const uint32_t at = dst + sw128_offset(8 * fill + i, (lane & 7) * 16);
        cp_async_16(at, src + i * 72);
        cp_async_16(at + 4 * kChunkBytes, src + i * 72 + 32);
        if (lane < 8) cp_async_16(at + 8 * kChunkBytes, src + i * 72 + 64);
    }
    cp_async_commit();
    cp_async_wait_group<0>();
    const float inv_kv = 1.f / p.kv_scale;                 // a power of two
#pragma unroll 1
    for (int i = 0; i < live; ++i) {
        const uint32_t at = dst + sw128_offset(8 * fill + i, (lane & 7) * 16);   // (this lane's own copies)
        uint4 x[3];
        x[0] = ld_shared_v4(at);
        x[1] = ld_shared_v4(at + 4 * kChunkBytes);
        x[2] = lane < 8 ? ld_shared_v4(at + 8 * kChunkBytes) : make_uint4(0, 0, 0, 0);
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
            top = fmaxf(top, k < 2 ? m : m * inv_kv);
        }
        // (magnitudes as fp32 bits are in the order of integers)
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        const int e = query_exp(p, top);
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = __uint_as_float(w[j] << 16) * f, b = __uint_as_float(w[j] & 0xffff0000u) * f;
                o[j] = k < 2 ? pack_f16x2(a, b) : pack_bf16x2(a * inv_kv, b * inv_kv);
            }
            if (k < 2 || lane < 8) st_shared_v4(at + 4 * k * kChunkBytes, o[0], o[1], o[2], o[3]);
        }
        if (lane == 0) sh.factor_exp[item & 3][8 * fill + i] = static_cast<int8_t>(factor_exp(p, e));
    }
}

// The warps that write operands, all of them those of K, then those of V: 32 rows of a slot each.  K of a tile goes before
// V of the tile before it, as the products do.
__device__ void fill(const PagedParams& p, Shared& sh, uint32_t rank, int nth, int lane) {
    const int slot = nth >> 1;
    const uint32_t leader = map_to_rank(&sh, 0) - smem_u32(&sh);
    const uint32_t k_ready = smem_u32(&sh.k_ready[slot]) + leader, v_ready = smem_u32(&sh.v_ready[slot >> 1]) + leader;
    const uint32_t k_piece = smem_u32(sh.k[slot]) + (nth & 1) * kHalfBytes, v_piece = smem_u32(sh.v[slot]) + (nth & 1) * kHalfBytes;
    // (which eight of the sixteen scale bytes are the slot's)
    const int k_scale = 8 * (slot & 1), v_scale = 8 * (slot >> 1);
    const int total = static_cast<int>(sh.work.count);
    int item = 0, in_item = 0;                             // of the K at hand; its tiles still to come
    for (int g = 0; g <= total && total > 0; ++g) {
        if (g < total) {
            if (in_item == 0) {
                if (!warp_wait(&sh.abort_flag, &sh.item_full[item % kItems], (item / kItems) & 1)) break;
                const Item& i = sh.items[item % kItems];
                in_item = i.hi - i.lo;
                if (item > 0 && !warp_wait(&sh.abort_flag, &sh.q_empty, (item - 1) & 1)) break;
                const int r0 = i.rb * kTreeBlockRows + static_cast<int>(rank) * 64 + 8 * nth;
                fill_queries(p, sh, static_cast<long long>(i.b) * p.tokens * p.heads + r0,
                             min(i.n_tok * p.heads - r0, 8), item, nth, lane);
                hand_over(smem_u32(&sh.q_ready) + leader, lane);
                if (lane == 0) mbar_arrive(&sh.q_local[item & 1]);
                Walk::release(sh, item, lane);
                ++item;
            }
            --in_item;
            if (!warp_wait(&sh.abort_flag, &sh.k_raw[slot], g & 1)) break;
            widen_half(k_piece, k_scale, false, lane);
            hand_over(k_ready, lane);
        }
        if (g > 0) {
            if (!warp_wait(&sh.abort_flag, &sh.v_raw[slot], (g - 1) & 1)) break;
            widen_half(v_piece, v_scale, true, lane);
            hand_over(v_ready, lane);
        }
        if (g == total) return;
    }
    if (total > 0 && lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

// The warps that ask for the bytes: a slot's when the products with the tile before are done.
struct Producer {
    const PagedMaps& maps;
    const PagedParams& p;
    const int lane, box;                                   // rows per box; a lane has one of those of 64 rows
    const uint64_t policy;

    __device__ __forceinline__ int row() const { return box * (lane & (64 / box - 1)); }
    // page of this lane's box of the 64 rows from t0 on (one behind the last one: the box is zeros), and its row there
    __device__ __forceinline__ int page(int b, int t0) const {
        const int page = page_of(p.cache, b, t0 + row());
        return page < 0 ? p.cache.n_pages : page;
    }
    __device__ __forceinline__ int row_in_page(int t0) const { return (t0 + row()) & ((1 << p.cache.row_shift) - 1); }
    // 64 rows of a slot: 64 bytes of codes from byte `from` on
    __device__ __forceinline__ void slot(uint8_t* dst, uint64_t* bar, int from, int page, int in_page) const {
        if (lane == 0) mbar_arrive_expect_tx(bar, kRawBytes);
        __syncwarp();
        if (lane < 64 / box) {
            uint8_t* piece = dst + (row() >> 5) * kHalfBytes;
            tma_load_3d(piece + (row() & 31) * 64, &maps.codes, from, in_page, page, bar, policy);
            tma_load_3d(piece + kChunkBytes + (row() & 31) * 16, &maps.scales, kQ4Scales + 16 * (from >> 7), in_page, page,
                        bar, policy);
        }
    }
};

// K and the key values of this CTA's 64 rows.
__device__ void produce_keys(const PagedMaps& maps, const PagedParams& p, Shared& sh, uint32_t rank, int lane) {
    const Producer pr{maps, p, lane, box_rows(p.cache), l2_policy_evict_normal()};
    const uint32_t rope_bar = map_to_rank(&sh.rope_ready, 0);
    const int mine = 64 * static_cast<int>(rank);
    Walk c;
    bool ok = c.start(sh);
    if (c.left <= 0) return;
    int page = 0, at = 0;
    if (ok) {
        page = pr.page(c.b, c.row() + mine);
        at = pr.row_in_page(c.row() + mine);
    }
    while (ok) {
        const int g = c.g;
        if (c.first) Walk::release(sh, c.item, lane);
#pragma unroll 1
        for (int s = 0; s < kSlots && ok; ++s) {
            ok = g == 0 || warp_wait(&sh.abort_flag, &sh.k_empty[s], (g - 1) & 1);
            if (ok) pr.slot(sh.k[s], &sh.k_raw[s], 64 * s, page, at);
        }
        if (!ok) break;
        // (the even CTA announces both CTAs' bytes; the odd one's may land first: the phase is open until then)
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&sh.rope_ready, 2 * kChunkBytes);
        __syncwarp();
        if (lane < 64 / pr.box)
            tma_load_3d_pair(sh.rope + pr.row() * 128, &maps.rope, kQ4Rope, at, page, rope_bar, pr.policy);
        ok = c.next(sh);
        if (c.left <= 0) return;
        if (ok) {                                          // the next tile's place, looked up ahead
            page = pr.page(c.b, c.row() + mine);
            at = pr.row_in_page(c.row() + mine);
        }
    }
    if (lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

// V of the tile's rows, this CTA's 256 features; and this CTA's 64 rows of a later tile on their way to L2.
constexpr int kAhead = 3;                                  // tiles
__device__ void produce_values(const PagedMaps& maps, const PagedParams& p, Shared& sh, uint32_t rank, int lane) {
    const Producer pr{maps, p, lane, box_rows(p.cache), l2_policy_evict_normal()};
    Walk c;
    bool ok = c.start(sh);
    if (c.left <= 0) return;
    Walk ahead = c;
    int page[2] = {}, at[2] = {};
    auto find = [&] {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            page[kb] = pr.page(c.b, c.row() + 64 * kb);
            at[kb] = pr.row_in_page(c.row() + 64 * kb);
        }
    };
    if (ok) find();
    while (ok) {
        const int g = c.g;
        if (c.first) Walk::release(sh, c.item, lane);
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
            ok = g == 0 || warp_wait(&sh.abort_flag, &sh.v_empty[i], (g - 1) & 1);
            if (!ok) break;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                pr.slot(sh.v[2 * i + kb], &sh.v_raw[2 * i + kb], 128 * static_cast<int>(rank) + 64 * i, page[kb], at[kb]);
        }
        if (!ok) break;
        if (ahead.g < g) ahead = c;
        while (ahead.g < g + kAhead && ahead.left > 1) {
            // (an item that is not laid out yet is not waited for)
            if (ahead.in_item == 1 &&
                !__all_sync(0xffffffffu, mbar_test(&sh.item_full[(ahead.item + 1) % kItems], ((ahead.item + 1) / kItems) & 1)))
                break;
            if (!ahead.next(sh)) break;
            if (lane < 64 / pr.box) {
                const int t = ahead.row() + 64 * static_cast<int>(rank) + pr.row(), far = page_of(p.cache, ahead.b, t);
                if (far >= 0) bulk_prefetch_l2(row_in(p.cache, far, t), pr.box * MLA_Q4_ROW);
            }
        }
        ok = c.next(sh);
        if (c.left <= 0) return;
        if (ok) find();
    }
    if (lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

// ============================== MMA issue ==================================
// As in mla_tree_attend.cu: one warp issues everything, QK of a tile before PV of the tile
// before it (after it at an item's first tile), each barrier looked at ahead of its use.
struct Issue {
    Shared& sh;
    bool lead, ok;

    // after `seen` (an earlier look at the barrier): the phase is over
    __device__ __forceinline__ void need(bool seen, uint64_t* bar, uint32_t parity) {
        if (!seen) ok = wait_slowly(bar, parity, &sh.abort_flag) && ok;
    }
};

__device__ void issue(const PagedParams& p, Shared& sh, uint32_t tmem) {
    constexpr uint32_t idesc_qk = make_idesc_f16(128, 128, 0, 0), idesc_rope = make_idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idesc_pv = make_idesc_f16(128, 256, 0, 1);
    Issue is{sh, elect_one(), true};
    const uint64_t kd = make_sdesc(smem_u32(sh.k), 16, 1024, kLayoutSw128);
    const uint64_t vd = make_sdesc(smem_u32(sh.v), kChunkBytes, 1024, kLayoutSw128);
    const uint64_t rope = make_sdesc(smem_u32(sh.rope), 16, 1024, kLayoutSw128);
    const uint64_t q = make_sdesc(smem_u32(sh.q), 16, 1024, kLayoutSw128);
    const uint64_t pd = make_sdesc(smem_u32(sh.p), 16, 1024, kLayoutSw128);
    int item = 0, pv_item = -1;
    const int total = static_cast<int>(sh.work.count), lane = threadIdx.x & 31;
    int in_item = 0;                                       // tiles of the item still to come
    auto enter = [&] {
        is.need(false, &sh.item_full[item % kItems], (item / kItems) & 1);
        in_item = sh.items[item % kItems].hi - sh.items[item % kItems].lo;
        __syncwarp();
        Walk::release(sh, item, lane);
    };
    if (total > 0) enter();
    bool first = true;
    uint32_t pv_first = 0;                                 // the tile before this QK's was the first of its item
    bool see_k = false, see_p = false, see_v = false;
    for (int g = 0; g <= total && is.ok; ++g) {
        const uint32_t buf = g & 1, par = g & 1;           // of QK(g); PV(g - 1) has the other parity
        const uint32_t qk_first = first;
        const int pv_turn = first ? 0 : 1;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            if (turn == pv_turn) {
                if (g == 0) continue;
                is.need(see_p, &sh.p_ready, par ^ 1);
                if (pv_first && ++pv_item > 0) is.need(false, &sh.o_free, (pv_item - 1) & 1);
                tc_fence_after_sync();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    is.need(see_v, &sh.v_ready[i], par ^ 1);
                    if (i == 0)
                        see_v = mbar_test(&sh.v_ready[1], par ^ 1);
                    else
                        see_k = mbar_test(&sh.k_ready[0], par ^ pv_turn);   // of the QK that comes next
                    if (is.lead && is.ok) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            umma_pair_bf16(tmem + kTmemO + 128 * i, pd + (((k >> 2) * kChunkBytes + (k & 3) * 32u) >> 4),
                                           vd + (((2 * i + (k >> 2)) * kSlotBytes + (k & 3) * 2048u) >> 4), idesc_pv,
                                           k == 0 ? pv_first ^ 1u : 1u);
                        if (g < total) umma_commit_pair(&sh.v_empty[i]);
                    }
                }
                if (is.lead && is.ok) umma_commit_pair(&sh.o_done);
                see_p = see_v = false;
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
                    } else {
                        is.need(false, &sh.rope_ready, par);
                        if (pv_turn == 1 && g >= 1) {
                            see_p = mbar_test(&sh.p_ready, par ^ 1);
                            see_v = mbar_test(&sh.v_ready[0], par ^ 1);
                        }
                    }
                    if (s == 0) tc_fence_after_sync();
                    if (is.lead && is.ok) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = ((2 * s + (k >> 2)) * kChunkBytes + (k & 3) * 32u) >> 4;
                            umma_pair_bf16(d, q + off, kd + off, idesc_qk, (s | k) ? 1u : 0u);
                        }
                        if (s == kSlots - 1) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_pair_bf16(d, q + ((8 * kChunkBytes + k * 32u) >> 4), rope + (k * 32u >> 4),
                                               idesc_rope, 1u);
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
                    ++item;
                    enter();
                }
            }
        }
        pv_first = qk_first;
    }
    if (!is.ok && is.lead) raise_tree_error(&sh.abort_flag, p.status);
}

// ============================== softmax ====================================
// Place of a piece's feature quad, as the merge reads it: [slot][32-row group][quad][row].
__device__ __forceinline__ long long piece_quad(int slot, int row, int quad) {
    return ((static_cast<long long>(slot) * (kTreeBlockRows / 32) + (row >> 5)) * (kDLatent / 4) + quad) * 32 + (row & 31);
}

// 64 bytes of each of a warp's 32 rows, through its 2 KB of shared memory so that the stores of a
// row run along its features (16-byte units, swizzled by row pair).
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

__device__ __forceinline__ uint32_t low_bits32(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }
__device__ __forceinline__ int row_int(long long t) { return static_cast<int>(min(max(t, 0ll), 0x7fffffffll)); }

// Thread: 32 keys of one row.  Warps w and w + 4 share tensor-memory lanes 32 (w mod 4) ..
// and split their columns.
__device__ void softmax(const PagedParams& p, Shared& sh, uint32_t tmem, uint32_t rank, int cluster, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    const int sub = warp >> 2, half = (warp >> 1) & 1;     // keys 64 half + 32 sub ..; features 256 half + 128 sub ..
    const int quarter = 2 * half + sub;
    const int row = 32 * (warp & 1) + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t p_bar = map_to_rank(&sh.p_ready, 0), o_bar = map_to_rank(&sh.o_free, 0);
    const uint32_t p_line = smem_u32(sh.p[half]) + row * 128;
    bool ok = true, bad = false;
    const bool notes = rank == 0 && tid == 0;
    if (notes)
        for (int i = 0; i < kTreePieces; ++i) p.merge[i * p.clusters + cluster].pieces = 0;
    Walk c;
    ok = c.start(sh);
    // whether rows 8 (lane & 15) .. of the tile have a page, looked up a tile ahead
    int pages = 0;
    if (c.left > 0 && ok) pages = page_of(p.cache, c.b, c.row() + 8 * (lane & 15));
    while (c.left > 0 && ok) {
        // ---- one item: tiles of one row block
        const int item = c.item, g0 = c.g;
        const Item& it = sh.items[item % kItems];
        const int r = it.rb * kTreeBlockRows + static_cast<int>(rank) * 64 + row;
        const bool live = r < it.n_tok * p.heads;
        // this row's token attends rows [from, to) and those before sink
        const long long own = static_cast<long long>(it.d_pos) + r / p.heads;
        const int to = live ? row_int(own + 1) : 0;
        const int from = p.window > 0 ? row_int(own + 1 - p.window) : 0;
        // tiles whose rows every token attends: up to all_to, from all_from on or before sink
        const int all_to = row_int(static_cast<long long>(it.d_pos) + 1);
        const int all_from = p.window > 0 ? row_int(static_cast<long long>(it.d_pos) + it.n_tok - p.window) : 0;
        bad |= !warp_wait(&sh.abort_flag, &sh.q_local[item & 1], (item >> 1) & 1);
        const float c2 = p.unit * (live ? power_of_two(sh.factor_exp[item & 3][row]) : 1.f);
        float m_ref = -INFINITY, l = 0.f;
        bool last;
        do {
            const int g = c.g, buf = g & 1;
            last = c.in_item == 1;
            bool w = warp_wait(&sh.abort_flag, &sh.s_full[buf], (g >> 1) & 1);
            uint32_t s[32];
            if (w) {
                tmem_ld32_async(tmem + lanes + kTmemS + 64 * buf + 32 * sub, s);
                tmem_wait_ld32(s);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = 0;
            }
            const int t0 = c.row();
            const uint32_t here = __ballot_sync(0xffffffffu, pages >= 0);
            if (here != 0xffffffffu || t0 + kTreeTileKeys > all_to || (t0 < all_from && t0 + kTreeTileKeys > p.sink)) {
                const int t = t0 + 64 * half + 32 * sub;
                const uint32_t four = here >> (8 * half + 4 * sub) & 15;   // of eight rows each
                const uint32_t v = low_bits32(to - t) & (~low_bits32(from - t) | low_bits32(p.sink - t)) &
                                   ((four * 0x00204081u & 0x01010101u) * 0xffu);
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
            const float base = (m_ref > -INFINITY ? m_ref : 0.f) - kProbLog2;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = ex2_approx(fmaf(__uint_as_float(s[2 * i]), c2, -base));
                const float y = ex2_approx(fmaf(__uint_as_float(s[2 * i + 1]), c2, -base));
                sum[i & 1] += x;
                sum[2 + (i & 1)] += y;
                pk[i] = pack_f16x2(x, y);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            // P of the tile before has been read, and O holds all tiles before this one
            w = g == 0 || warp_wait(&sh.abort_flag, &sh.o_done, (g - 1) & 1);
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
            // ---- probabilities, f16, K-major lines of 64 keys
#pragma unroll
            for (int u = 0; u < 4; ++u)
                st_shared_v4(p_line + (((4 * sub + u) ^ (row & 7)) << 4), pk[4 * u], pk[4 * u + 1], pk[4 * u + 2],
                             pk[4 * u + 3]);
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            bad |= !w;                                     // the threads leave together at the next barrier
            if (lane == 0 && !bad) mbar_arrive_peer(p_bar);
            const bool entered = c.next(sh);
            bad |= !entered;
            if (c.left > 0 && entered) pages = page_of(p.cache, c.b, c.row() + 8 * (lane & 15));
        } while (!last);
        if (!ok) break;

        // ---- epilogue: l of the four quarters, O / l, log-sum-exp
        sh.red_sum[quarter][row] = l;
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, bad)) {
            ok = false;
            break;
        }
        const float lt = (sh.red_sum[0][row] + sh.red_sum[1][row]) + (sh.red_sum[2][row] + sh.red_sum[3][row]);
        const float inv = lt == 0.f ? 0.f : p.kv_scale / lt;
        const float lse2 = lt == 0.f ? -INFINITY : (m_ref - kProbLog2) + log2f(lt);
        const int b = it.b, rb = it.rb, live_rows = it.n_tok * p.heads;
        const bool whole = it.flags & kWhole;
        // place of the piece: the run's first item, one that ends with the run's length, another
        const int place = g0 == 0 ? 0 : c.g == sh.work.per ? 2 : 1, slot = kTreePieces * cluster + place;
        if (quarter == 0 && live) {
            if (whole)
                p.a.lse[static_cast<long long>(b) * p.tokens * p.heads + r] = lse2 * kLn2;
            else
                p.lse_part[slot * kTreeBlockRows + static_cast<int>(rank) * 64 + row] = lse2;
        }
        if (notes && it.flags & kOpens) {
            const bool cut = it.flags & kCut;
            const TreeCut of{it.n_rb, it.n_tiles, static_cast<int>(sh.work.per), it.begin};
            const int rows = min(kTreeBlockRows, live_rows - rb * kTreeBlockRows);
            // (an uncut job's pieces lie in the runs from this one to that of its last unit)
            const int pieces = cut ? -1 : (of.begin + (rb + 1) * of.n_tiles - 1) / of.per + 1;
            const int at = (cut ? place : 0) * p.clusters + cluster;
            p.merge[at] = TreeMerge{b, rb, rows | place << 16, pieces};
            if (cut) p.cut[at] = of;
        }
        const bool w = warp_wait(&sh.abort_flag, &sh.o_done, (c.g - 1) & 1);
        if (named_barrier_or(kBarSoftmax, kSoftmaxThreads, !w)) {
            ok = false;
            break;
        }
        // (P's buffer is free: the last product is done)
        const uint32_t stage = smem_u32(sh.p) + warp * 2048;
        const int row_w = 32 * (warp & 1);                 // this warp's first row of the 64
        const int n_rows = live_rows - (r - row) - row_w;
        const int f0 = 256 * half + 128 * sub;             // its first feature
        float4* piece = reinterpret_cast<float4*>(p.part) +
                        piece_quad(slot, static_cast<int>(rank) * 64 + row_w, f0 / 4) + lane;
        const int bytes = p.a.out_fp32 ? 4 : 2;
        char* out = static_cast<char*>(p.a.out) +
                    ((static_cast<long long>(b) * p.tokens * p.heads + r - row + row_w) * kDLatent + f0) * bytes;
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
            if (!p.a.out_fp32) {
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
        Walk::release(sh, item, lane);
        tc_fence_before_sync();
        __syncwarp();
        // O may be overwritten.  (Only if something will wait for it: the closing barrier orders no arrival.)
        if (lane == 0 && c.left > 0) mbar_arrive_peer(o_bar);
    }
    if (!ok && lane == 0) raise_tree_error(&sh.abort_flag, p.status);
}

// Requests without rows: their tokens' outputs, by the odd CTAs' otherwise idle warp.
__device__ void write_empty(const PagedParams& p, int cluster, int clusters, int lane) {
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

__device__ __noinline__ void find_work(const PagedParams& p, int cluster, int lane, TreeWork* work) {
    Cursor::find_work(p, cluster, lane, work);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_paged_attend_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    if (tid == 0) {
        prefetch_tensormap(&maps.codes);
        prefetch_tensormap(&maps.scales);
        prefetch_tensormap(&maps.rope);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.k_ready[i], 4);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.k_raw[i], 1);
            mbar_init(&sh.v_raw[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.v_ready[i], 8);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
        }
        mbar_init(&sh.rope_ready, 1);
        mbar_init(&sh.p_ready, 2 * kSoftmaxWarps);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.q_ready, 2 * kFillWarps);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.q_local[i], kFillWarps);
        mbar_init(&sh.o_free, 2 * kSoftmaxWarps);
        mbar_init(&sh.q_empty, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kItemReaders + (rank == 0 ? 1 : 0));
        }
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    __syncwarp();
    cluster_arrive();                                      // (after this thread's barrier initialisation)
    if (warp == kMmaWarp) tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == kScoutWarp) {
        find_work(p, cluster, lane, &sh.work);
    } else if (warp >= kFillWarp) {
        // query rows behind the last one: zeros, so that their scores are finite
        for (int i = tid - 32 * kFillWarp; i < static_cast<int>(kQBytes / 16); i += 32 * kFillWarps)
            reinterpret_cast<uint4*>(sh.q)[i] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_wait();                                        // both CTAs' barriers are initialised
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_base;
    if (p.stall_test && blockIdx.x == 0 && tid == 32 * kScoutWarp) {
        // test hook: a wait that runs out, so the abort path runs for real
        volatile int never = 0;
        if (!mbar_wait_bounded(&sh.stall_bar, 0, &never, kStallTestCycles)) raise_tree_error(&sh.abort_flag, p.status);
    }
    __syncwarp();
    // the dynamic window starts 1024-byte aligned (the 128-byte swizzle needs it)
    if ((smem_u32(smem_raw) & 1023u) != 0 && tid == 0) raise_tree_error(&sh.abort_flag, p.status);
    if (warp >= kFillWarp) {
        fill(p, sh, rank, warp - kFillWarp, lane);
    } else if (warp >= kSoftmaxWarp) {
        softmax(p, sh, tmem, rank, cluster, tid - 32 * kSoftmaxWarp);
    } else if (warp == kMmaWarp) {
        if (rank == 0)
            issue(p, sh, tmem);
        else
            write_empty(p, cluster, p.clusters, lane);
    } else if (warp == kKeyWarp) {
        produce_keys(maps, p, sh, rank, lane);
    } else if (warp == kValueWarp) {
        produce_values(maps, p, sh, rank, lane);
    } else {
        scout(p, sh, lane);
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

}  // namespace

cudaError_t paged_attend_prepare() {
    return cudaFuncSetAttribute(mla_paged_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(Shared)));
}

cudaError_t launch_paged_attend(const PagedMaps& maps, const PagedParams& p, bool pdl, cudaStream_t stream) {
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mla_paged_attend_kernel, maps, p);
    // (it waits for this kernel's end before it reads: it may always be launched ahead)
    return e != cudaSuccess ? e : launch_tree_merge(p, true, stream);
}

}  // namespace mla
