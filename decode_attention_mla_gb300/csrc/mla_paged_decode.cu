// mla_paged_decode.cu -- attention over the 4-bit paged cache for few query rows:
// warp-level MMAs on values widened in registers (include/mla_paged.h).
//
// Sixteen query rows (token * heads + head) are one MMA tile, and rows need be widened for nobody
// else, so nothing is gained by operands in shared memory: the tcgen05 kernel (mla_paged_attend.cu) writes
// and reads them there, 390 KB per 128 rows of a pair, whatever the number of query rows.  Here rows stay as they
// are in shared memory (416 bytes), and each warp takes its bytes from there twice, into the fragments
// of Q K^T and of P V.
//
// A group of eight warps shares the 64 rows of a slot.  Warp w has features 64 w .. + 63 (and 16 of the 64 key
// values of half of the rows): its scores are partial sums, which the warps exchange through shared memory; warp w then
// has the whole scores of rows 8 w .. + 7, and hands their probabilities to the others; and its part of O, 16 x 64
// fp32, stays in registers.  Two groups take alternate slots, each with a running maximum and sum of its own, and are
// joined at an item's end.  (Groups of four warps with 128 features: 204 us where eight take XX for 32 requests of 16
// heads: two warps per scheduler leave it idle two cycles of three.)
//
// Orders.  The contraction over features may go in any order: lane 4 g + j has, of row g of eight, features 16 j ..
// 16 j + 15 (a block: eight bytes of codes), four to a k-step.  Rows of a slot lie 416 bytes apart, eight banks on, so four
// rows' eight banks each are all 32.  For P V lane 4 g + j has features 8 g .. 8 g + 7 (four bytes) of rows j, 4 + j, 8 + j,
// 12 + j of sixteen: again all banks.  Two rows' codes are brought together in bytes (low and high half), so one
// conversion gives the pair of values that a fragment wants.
//
// A code times its scale is exact in f16 (six bits, 2^-10 .. 2688).  Queries are f16 times a power of two per row, probabilities
// f16 times 2^7, key values and their queries bf16, as in mla_paged_attend.cu; sums are fp32.  Codes are finite whatever
// the bytes, and a scale's NaN becomes 0 in P V (in Q K^T it stays: the row's scores are NaN); so rows that nobody
// attends need no clearing: their scores are masked, their probabilities 0.
//
// Work split: units of 128 rows (a slot per group) of all requests' blocks of sixteen query rows, one equal run per SM; pieces and
// their merge as in mla_tree_attend.cu.
//
// Bound: 16 MMAs and about 66 other instructions of a warp per row and SM, 17 cycles each way, beside 19 for its bytes from
// HBM.
//
// Warps: 0-7 and 8-15 the groups, 16 bulk copies and the run's items, 17 empty requests.
#include <cmath>

#include "mla_paged.cuh"

namespace mla {
namespace {

constexpr int kUnitRows = 128, kSlotRows = 64;
constexpr int kSlotBytes = kSlotRows * MLA_Q4_ROW;
constexpr int kRing = 6;
constexpr int kWarps = 8;                                  // of a group
constexpr int kGroupThreads = 32 * kWarps, kComputeThreads = 2 * kGroupThreads;
constexpr int kProducerWarp = 2 * kWarps, kEmptyWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kEmptyWarp + 1);
constexpr int kBarGroup = 1, kBarBoth = 3;                 // hardware barriers: of each group, of both
constexpr int kBlockRows = kDecodeBlockRows;
constexpr float kRescaleLog2 = 8.0f;                       // move the reference when a max grows past 2^8
constexpr float kProbLog2 = 7.0f;                          // P is held times 2^7
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kItems = 4;
constexpr int kSide = 2;                                   // chains of score products side by side

// What this run does of a row block: units lo .. hi - 1 of its n_units.
struct __align__(16) Item {
    int b, rb, lo, hi;
    int near, skip, d_pos, n_tok;                          // as r.lo, r.base of the request, and its own
    int n_units, runs, unused[2];                          // runs: that the block lies in, if this one opens it
};

struct __align__(128) Shared {
    uint8_t ring[kRing][kSlotBytes];
    // per group: partial scores by warp, eight rows, lane; at an item's end group 1's O by warp, tile, lane
    float4 part[2][kWarps][8][32];
    uint16_t p[2][16][80];                                 // per group: probabilities, row by row (padded), see place_of
    float red[2][kWarps][16];                              // per group: maxima or sums by warp, row
    float ml[2][16];                                       // group 1's maximum and sum
    Item items[kItems];
    uint64_t full[kRing], empty[kRing];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t stall_bar;
    uint32_t valid[kRing];                                 // which eight rows of a slot have a page
    int abort_flag;
};
static_assert(sizeof(Shared) <= 227 * 1024, "fits shared memory");

// ============================== the run ====================================
__device__ __forceinline__ int blocks_of(const PagedParams& p, const TreeRequest& r) {
    return (r.n_tok * p.heads + kBlockRows - 1) / kBlockRows;
}
__device__ __forceinline__ int units_of(const TreeRequest& r) { return r.hi / kUnitRows; }

// Whole warp: units of all requests, and the request that unit u0 lies in with the units before it (b = batch: none).
// (The host takes this kernel only where all units there could be fit 31 bits.)
struct Start {
    int total, b, before;
};
__device__ int count_units(const PagedParams& p, int lane) {
    int total = 0;
    for (int b = lane; b < p.batch; b += 32) {
        const TreeRequest r = load_paged_request<kUnitRows>(p, b);
        total += blocks_of(p, r) * units_of(r);
    }
    return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(total)));
}
__device__ Start find_start(const PagedParams& p, int u0, int lane) {
    Start s{0, p.batch, 0};
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        int u = 0;
        if (b0 + lane < p.batch) {
            const TreeRequest r = load_paged_request<kUnitRows>(p, b0 + lane);
            u = blocks_of(p, r) * units_of(r);
        }
        int incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const int first = s.before + incl - u;
        const uint32_t here = __ballot_sync(0xffffffffu, u > 0 && u0 >= first && u0 < first + u);
        if (here) {
            const int src = __ffs(here) - 1;
            s.b = b0 + src;
            s.before = __shfl_sync(0xffffffffu, first, src);
            return s;
        }
        s.before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return s;
}

__device__ __forceinline__ bool wait(Shared& sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, &sh.abort_flag));
}
__device__ __forceinline__ void raise(const PagedParams& p, Shared& sh) {
    *static_cast<volatile int*>(&sh.abort_flag) = 1;
    if (p.status) atomicCAS(p.status, 0, static_cast<int>(MLA_EDEVICE));
}

// ============================== producer ==================================
// One warp: the run's items, and the bytes of its slots.  A lane has a box (the rows of a page that lie in a
// slot) of one of a unit's two slots.
__device__ void produce(const PagedParams& p, Shared& sh, int lane) {
    const int total = count_units(p, lane);
    const int per = (total + p.clusters - 1) / p.clusters, cta = blockIdx.x;
    const int u0 = static_cast<int>(min(static_cast<long long>(per) * cta, static_cast<long long>(total)));
    const int u1 = min(u0 + per, total);
    const uint64_t policy = l2_policy_evict_normal();
    const int box = min(1 << p.cache.row_shift, kSlotRows), boxes = kSlotRows / box;   // of a slot
    const bool mine = lane < 2 * boxes;
    const int row = (lane & (boxes - 1)) * box + (lane >= boxes ? kSlotRows : 0);     // of the unit
    if (u0 < u1) {
        Start s = find_start(p, u0, lane);
        TreeRequest r = load_paged_request<kUnitRows>(p, s.b);
        int n = units_of(r), rb = (u0 - s.before) / n, at = (u0 - s.before) - rb * n;
        int b = s.b, u = u0, ring = 0, turn = 0, item = 0;
        while (u < u1) {
            // ---- an item
            const int hi = min(n, at + (u1 - u));
            if (item >= kItems && !wait(sh, &sh.item_empty[item % kItems], (item / kItems - 1) & 1)) break;
            if (lane == 0) {
                Item& i = sh.items[item % kItems];
                i.b = b;
                i.rb = rb;
                i.lo = at;
                i.hi = hi;
                i.near = r.lo;
                i.skip = static_cast<int>(r.base);
                i.d_pos = r.d_pos;
                i.n_tok = r.n_tok;
                i.n_units = n;
                // (runs end at multiples of per)
                i.runs = at == 0 ? (u + n - 1) / per - cta + 1 : 0;
                mbar_arrive(&sh.item_full[item % kItems]);
            }
            __syncwarp();
            // ---- its units' slots; pages are looked up a unit ahead
            auto place = [&](int unit, int& t) {
                t = (unit < r.lo ? unit : unit + static_cast<int>(r.base)) * kUnitRows + row;
                return mine ? page_of(p.cache, b, t) : -1;
            };
            int t, page = place(at, t);
            bool ok = true;
            for (; at < hi && ok; ++at, ++u) {
                const int now = page;
                const uint8_t* src = now >= 0 ? row_in(p.cache, now, t) : nullptr;
                if (at + 1 < hi) page = place(at + 1, t);
                const uint32_t have = __ballot_sync(0xffffffffu, now >= 0);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (turn > 0 && !wait(sh, &sh.empty[ring], (turn - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t here = have >> (q * boxes) & ((1u << boxes) - 1);
                    if (lane == 0) {
                        // eight rows a bit
                        uint32_t v = 0;
                        for (int k = 0; k < 8; ++k) v |= (here >> (8 * k / box) & 1) << k;
                        sh.valid[ring] = v;
                        mbar_arrive_expect_tx(&sh.full[ring], __popc(here) * box * MLA_Q4_ROW);
                    }
                    __syncwarp();
                    if (mine && (lane >= boxes) == (q == 1) && src)
                        bulk_copy_g2s(sh.ring[ring] + (row & (kSlotRows - 1)) * MLA_Q4_ROW, src, box * MLA_Q4_ROW,
                                      &sh.full[ring], policy);
                    if (++ring == kRing) {
                        ring = 0;
                        ++turn;
                    }
                }
            }
            if (!ok) {
                if (lane == 0) raise(p, sh);
                return;
            }
            ++item;
            if (u < u1 && at == n) {
                at = 0;
                if (++rb == blocks_of(p, r)) {
                    rb = 0;
                    do {
                        r = load_paged_request<kUnitRows>(p, ++b);
                        n = units_of(r);
                    } while (n == 0);
                }
            }
        }
        if (u < u1 && lane == 0) raise(p, sh);
        // no more items
        if (u == u1 && (item < kItems || wait(sh, &sh.item_empty[item % kItems], (item / kItems - 1) & 1)) && lane == 0) {
            sh.items[item % kItems].b = -1;
            mbar_arrive(&sh.item_full[item % kItems]);
        }
    } else if (lane == 0) {
        sh.items[0].b = -1;
        mbar_arrive(&sh.item_full[0]);
    }
}

// ============================== compute ====================================
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t clean_nan(uint32_t v) {
    return v & __heq2_mask(*reinterpret_cast<__half2*>(&v), *reinterpret_cast<__half2*>(&v));
}
// (Not volatile: with two warps per scheduler the order of loads, conversions and products counts.)
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int row_int(long long t) { return static_cast<int>(min(max(t, 0ll), 0x7fffffffll)); }

// Place in a row of P of slot row t: the four of 16 rows that a lane's fragment wants lie together.
__device__ __forceinline__ int place_of(int t) { return (t & 48) | (t & 3) << 2 | (t >> 2 & 3); }

struct Fragments {
    uint32_t q[4][4];                                      // f16, by k-step
    uint32_t rope[4];                                      // bf16
};

// This lane's query values: rows g and g + 8 of the block, features 64 w + 16 j .. + 15, key values 16 (w mod 4) + 4 j .. + 3,
// and what the rows were divided by.
__device__ __forceinline__ void load_queries(const PagedParams& p, Shared& sh, int group, int w, int lane, long long row0, int live,
                                             Fragments& f, float (&factor)[2]) {
    const int g = lane >> 2, j = lane & 3;
    uint4 x[2][2];
    uint2 y[2];
    const float inv_kv = 1.f / p.kv_scale;                 // a power of two
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint16_t* src = p.q + (row0 + g + 8 * h) * kDRow;
        const bool there = g + 8 * h < live;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            x[h][k] = there ? reinterpret_cast<const uint4*>(src + 64 * w + 16 * j)[k] : make_uint4(0, 0, 0, 0);
        y[h] = there ? *reinterpret_cast<const uint2*>(src + kDLatent + 16 * (w & 3) + 4 * j) : make_uint2(0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float top = 0.f, rope = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t v[4] = {x[h][k].x, x[h][k].y, x[h][k].z, x[h][k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u))));
        }
        const uint32_t v[2] = {y[h].x, y[h].y};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            rope = fmaxf(rope, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u))));
        top = fmaxf(top, rope * inv_kv);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (j == 0) sh.red[group][w][g + 8 * h] = top;
    }
    named_barrier_sync(kBarGroup + group, kGroupThreads);
    float scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sh.red[group][k][g + 8 * h]);
        const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -126), 126);
        scale[h] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        factor[h] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
    // k-step s: features 16 j + 4 s, + 1 (registers 0, 1) and + 2, + 3 (2, 3); rows g (0, 2) and g + 8 (1, 3)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t v[4] = {x[h][k].x, x[h][k].y, x[h][k].z, x[h][k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f.q[2 * k + (e >> 1)][2 * (e & 1) + h] =
                    pack_f16x2(__uint_as_float(v[e] << 16) * scale[h], __uint_as_float(v[e] & 0xffff0000u) * scale[h]);
        }
        const uint32_t v[2] = {y[h].x, y[h].y};
#pragma unroll
        for (int e = 0; e < 2; ++e)
            f.rope[2 * e + h] = pack_bf16x2(__uint_as_float(v[e] << 16) * scale[h] * inv_kv,
                                            __uint_as_float(v[e] & 0xffff0000u) * scale[h] * inv_kv);
    }
    // (`red` is written again after the next barrier of the group)
}

__device__ void compute(const PagedParams& p, Shared& sh, int group, int w, int lane) {
    const int g = lane >> 2, j = lane & 3;
    const int bar = kBarGroup + group;
    bool bad = false;
    // this lane's scores: rows g and g + 8, slot rows 8 w + 2 j, + 1
    const int key_place = place_of(8 * w + 2 * j);         // (of the next row four places on)
    int ring = group, turn = 0;
    // A hardware barrier has no time limit, so nobody leaves one alone: a group leaves together (its barriers tell
    // whether one of its waits ran out), and after the run or in the middle of it, it meets the other once more.
    for (int item = 0;; ++item) {
        bad = !wait(sh, &sh.item_full[item % kItems], (item / kItems) & 1);
        if (named_barrier_or(bar, kGroupThreads, bad)) {
            bad = true;
            break;
        }
        const Item& it = sh.items[item % kItems];
        if (it.b < 0) break;
        const int live = min(it.n_tok * p.heads - it.rb * kBlockRows, kBlockRows);
        const long long row0 = static_cast<long long>(it.b) * p.tokens * p.heads + it.rb * kBlockRows;
        Fragments f;
        float c2[2];
        load_queries(p, sh, group, w, lane, row0, live, f, c2);
        c2[0] *= p.scale_log2 * p.kv_scale;
        c2[1] *= p.scale_log2 * p.kv_scale;
        // slots whose rows every token attends: up to all_to, from all_from on or before sink
        const int all_to = row_int(static_cast<long long>(it.d_pos) + 1);
        const int all_from = p.window > 0 ? row_int(static_cast<long long>(it.d_pos) + it.n_tok - p.window) : 0;
        const int units = it.hi, near = it.near, skip = it.skip;
        float o[8][4];
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[m][k] = 0.f;
        float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int unit = it.lo; unit < units; ++unit) {
            const int t0 = (unit < near ? unit : unit + skip) * kUnitRows + kSlotRows * group;
            bad |= !wait(sh, &sh.full[ring], turn & 1);
            const uint8_t* slot = sh.ring[ring];
            const uint32_t valid = sh.valid[ring];
            // ---- partial scores of this warp's features: chains of products side by side
#pragma unroll
            for (int e0 = 0; e0 < 8; e0 += kSide) {
                float acc[kSide][4];
                uint2 raw[kSide];
                uint32_t by[kSide];
#pragma unroll
                for (int e = 0; e < kSide; ++e) {
                    const uint8_t* at = slot + (8 * (e0 + e) + g) * MLA_Q4_ROW;
                    raw[e] = *reinterpret_cast<const uint2*>(at + 32 * w + 8 * j);
                    const uint32_t s = at[kQ4Scales + 4 * w + j];
                    by[e] = widen_e4m3(static_cast<uint16_t>(s | s << 8));
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[e][k] = 0.f;
                    if (w >> 2 == e0 >> 2) {               // (the key values of 32 rows are four warps', of the others the others')
                        const uint2 rope = *reinterpret_cast<const uint2*>(at + kQ4Rope + 32 * (w & 3) + 8 * j);
                        mma_bf16(acc[e], f.rope, rope.x, rope.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t h[kSide][4];
#pragma unroll
                    for (int e = 0; e < kSide; ++e) {
                        widen_e2m1(i == 0 ? raw[e].x : raw[e].y, h[e]);
                        mma_f16(acc[e], f.q[2 * i], mul_f16x2(h[e][0], by[e]), mul_f16x2(h[e][1], by[e]));
                    }
#pragma unroll
                    for (int e = 0; e < kSide; ++e)
                        mma_f16(acc[e], f.q[2 * i + 1], mul_f16x2(h[e][2], by[e]), mul_f16x2(h[e][3], by[e]));
                }
#pragma unroll
                for (int e = 0; e < kSide; ++e)
                    sh.part[group][w][e0 + e][lane] = make_float4(acc[e][0], acc[e][1], acc[e][2], acc[e][3]);
            }
            if (named_barrier_or(bar, kGroupThreads, bad)) {
                bad = true;
                break;
            }
            // ---- whole scores of rows 8 w .. + 7
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 v = sh.part[group][k][w][lane];
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            }
            const bool here = valid >> w & 1;
            if (!here || t0 + kSlotRows > all_to || (t0 < all_from && t0 + kSlotRows > p.sink)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the row's token attends rows [from, to) and those before sink
                    const long long own = static_cast<long long>(it.d_pos) + (it.rb * kBlockRows + g + 8 * h) / p.heads;
                    const int to = g + 8 * h < live ? row_int(own + 1) : 0;
                    const int from = p.window > 0 ? row_int(own + 1 - p.window) : 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int t = t0 + 8 * w + 2 * j + k;
                        if (!(here && t < to && (t >= from || t < p.sink))) s[2 * h + k] = -INFINITY;
                    }
                }
            }
            float top[2], base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[2 * h] *= c2[h];
                s[2 * h + 1] *= c2[h];
                top[h] = fmaxf(s[2 * h], s[2 * h + 1]);
                base[h] = (m_ref[h] > -INFINITY ? m_ref[h] : 0.f) - kProbLog2;
            }
            float e[4];
            auto publish = [&] {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    e[k] = ex2_approx(s[k] - base[k >> 1]);
                    const __half v = __float2half_rn(e[k]);
                    sh.p[group][g + 8 * (k >> 1)][key_place + 4 * (k & 1)] = *reinterpret_cast<const uint16_t*>(&v);
                }
            };
            publish();
            if (named_barrier_or(bar, kGroupThreads, top[0] > m_ref[0] + kRescaleLog2 || top[1] > m_ref[1] + kRescaleLog2)) {
                // rare after the first slot: the rows' maxima move the references
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float t = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    if (j == 0) sh.red[group][w][g + 8 * h] = t;
                }
                named_barrier_sync(bar, kGroupThreads);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = g + 8 * h;
                    float t = sh.red[group][0][r];
#pragma unroll
                    for (int k = 1; k < kWarps; ++k) t = fmaxf(t, sh.red[group][k][r]);
                    if (t > m_ref[h] + kRescaleLog2) {
                        const float alpha = m_ref[h] > -INFINITY ? ex2_approx(m_ref[h] - t) : 1.f;
                        m_ref[h] = t;
                        base[h] = t - kProbLog2;
                        l[h] *= alpha;
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            o[m][2 * h] *= alpha;
                            o[m][2 * h + 1] *= alpha;
                        }
                    }
                }
                publish();
                named_barrier_sync(bar, kGroupThreads);
            }
            l[0] += e[0] + e[1];
            l[1] += e[2] + e[3];
            // ---- P V, this warp's features, 16 rows at a time
#pragma unroll
            for (int step = 0; step < 4; ++step) {
                const uint2 a0 = *reinterpret_cast<const uint2*>(&sh.p[group][g][16 * step + 4 * j]);
                const uint2 a1 = *reinterpret_cast<const uint2*>(&sh.p[group][g + 8][16 * step + 4 * j]);
                const uint32_t a[4] = {a0.x, a1.x, a0.y, a1.y};
                uint32_t x[4], by[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* at = slot + (16 * step + 4 * i + j) * MLA_Q4_ROW;
                    x[i] = *reinterpret_cast<const uint32_t*>(at + 32 * w + 4 * g);
                    by[i] = at[kQ4Scales + 4 * w + (g >> 1)];
                }
                const uint32_t s01 = clean_nan(widen_e4m3(static_cast<uint16_t>(by[0] | by[1] << 8)));
                const uint32_t s23 = clean_nan(widen_e4m3(static_cast<uint16_t>(by[2] | by[3] << 8)));
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                uint32_t even01[4], odd01[4], even23[4], odd23[4];
                widen_e2m1((x[0] & kLow) | (x[1] << 4 & ~kLow), even01);
                widen_e2m1((x[2] & kLow) | (x[3] << 4 & ~kLow), even23);
                widen_e2m1((x[0] >> 4 & kLow) | (x[1] & ~kLow), odd01);
                widen_e2m1((x[2] >> 4 & kLow) | (x[3] & ~kLow), odd23);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_f16(o[2 * i], a, mul_f16x2(even01[i], s01), mul_f16x2(even23[i], s23));
                    mma_f16(o[2 * i + 1], a, mul_f16x2(odd01[i], s01), mul_f16x2(odd23[i], s23));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[ring]);
            ring += 2;
            if (ring >= kRing) {
                ring -= kRing;
                ++turn;
            }
        }
        if (bad) break;
        // ---- the item's end: sums over the group's rows, then both groups
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (j == 0) sh.red[group][w][g + 8 * h] = l[h];
        }
        named_barrier_sync(bar, kGroupThreads);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            l[h] = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) l[h] += sh.red[group][k][r];
        }
        if (group == 1) {
#pragma unroll
            for (int m = 0; m < 8; ++m) sh.part[1][w][m][lane] = make_float4(o[m][0], o[m][1], o[m][2], o[m][3]);
            if (w == 0 && j == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sh.ml[0][g + 8 * h] = m_ref[h];
                    sh.ml[1][g + 8 * h] = l[h];
                }
            }
        }
        if (named_barrier_or(kBarBoth, kComputeThreads, false)) return;   // the other group has left
        if (group == 0) {
            float by0[2], by1[2], lse2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float m1 = sh.ml[0][g + 8 * h], l1 = sh.ml[1][g + 8 * h];
                const float m = fmaxf(m_ref[h], m1);
                // (a group without rows has the sum 0 and O = 0; a NaN stays one)
                by0[h] = m_ref[h] > -INFINITY ? ex2_approx(m_ref[h] - m) : 1.f;
                by1[h] = m1 > -INFINITY ? ex2_approx(m1 - m) : 1.f;
                const float sum = l[h] * by0[h] + l1 * by1[h];
                const float inv = sum == 0.f ? 0.f : p.kv_scale / sum;
                lse2[h] = sum == 0.f ? -INFINITY : (m - kProbLog2) + log2f(sum);
                by0[h] *= inv;
                by1[h] *= inv;
            }
            const bool whole = it.hi - it.lo == it.n_units;
            const int slot = kTreePieces * static_cast<int>(blockIdx.x) + (item == 0 ? 0 : 1);
            if (w == 0 && j == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (g + 8 * h >= live) continue;
                    if (whole)
                        p.a.lse[row0 + g + 8 * h] = lse2[h] * kLn2;
                    else
                        p.lse_part[slot * 32 + g + 8 * h] = lse2[h];
                }
            }
            if (w == 0 && lane == 0 && !whole && it.lo == 0)
                p.merge[blockIdx.x] = TreeMerge{it.b, it.rb, live | (item == 0 ? 0 : 1) << 16, it.runs};
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const float4 v = sh.part[1][w][m][lane];
                o[m][0] = o[m][0] * by0[0] + v.x * by1[0];
                o[m][1] = o[m][1] * by0[0] + v.y * by1[0];
                o[m][2] = o[m][2] * by0[1] + v.z * by1[1];
                o[m][3] = o[m][3] * by0[1] + v.w * by1[1];
            }
            // rows g, g + 8; features 64 w + 16 j + m (register 0) and + 8 (register 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                if (r >= live) continue;
                if (!whole || p.a.out_fp32) {
                    float4* dst = whole ? reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + (row0 + r) * kDLatent + 64 * w + 16 * j)
                                        : reinterpret_cast<float4*>(p.part) +
                                              (static_cast<long long>(slot) * (kDLatent / 4) + 16 * w + 4 * j) * 32 + r;
                    const int step = whole ? 1 : 32;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int m = 4 * (k & 1), c = 2 * h + (k >> 1);
                        dst[step * k] = make_float4(o[m][c], o[m + 1][c], o[m + 2][c], o[m + 3][c]);
                    }
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + (row0 + r) * kDLatent + 64 * w + 16 * j);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int c = 2 * h + k;
                        dst[k] = make_uint4(pack_bf16x2(o[0][c], o[1][c]), pack_bf16x2(o[2][c], o[3][c]),
                                            pack_bf16x2(o[4][c], o[5][c]), pack_bf16x2(o[6][c], o[7][c]));
                    }
                }
            }
        }
        named_barrier_sync(kBarBoth, kComputeThreads);     // group 1's O has been read
        if (lane == 0) mbar_arrive(&sh.item_empty[item % kItems]);
    }
    named_barrier_or(kBarBoth, kComputeThreads, true);
    if (bad && lane == 0) raise(p, sh);
}

__global__ void __launch_bounds__(kThreads, 1) mla_paged_decode_kernel(const __grid_constant__ PagedParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], 2 * kWarps);
        }
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == kProducerWarp) {
        if (lane == 0) {
            for (int i = 0; i < kTreePieces; ++i) p.merge[i * p.clusters + blockIdx.x].pieces = 0;
            __threadfence_block();
            if (p.stall_test && blockIdx.x == 0) {
                // test hook: a wait that runs out, so the abort path runs for real
                volatile int never = 0;
                if (!mbar_wait_bounded(&sh.stall_bar, 0, &never, kStallTestCycles)) raise(p, sh);
            }
        }
        __syncwarp();
        produce(p, sh, lane);
    } else if (warp == kEmptyWarp) {
        // requests without rows: their tokens' outputs
        for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
            const TreeRequest r = load_paged_request<kUnitRows>(p, b);
            if (r.hi > 0 || r.n_tok == 0) continue;
            const long long row0 = static_cast<long long>(b) * p.tokens * p.heads;
            const int rows = r.n_tok * p.heads, per = p.a.out_fp32 ? 128 : 64;   // 16-byte units per row
            for (int i = lane; i < rows; i += 32) p.a.lse[row0 + i] = -INFINITY;
            uint4* o = reinterpret_cast<uint4*>(p.a.out) + row0 * per;
            for (int i = lane; i < rows * per; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        compute(p, sh, warp / kWarps, warp % kWarps, lane);
    }
    __syncthreads();
    if (*static_cast<volatile int*>(&sh.abort_flag)) {
        // copies in flight get time to land before shared memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 2000ll * 1000ll) {
        }
    }
}

}  // namespace

cudaError_t paged_decode_prepare() {
    return cudaFuncSetAttribute(mla_paged_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(sizeof(Shared)));
}

cudaError_t launch_paged_decode(const PagedParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.clusters);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mla_paged_decode_kernel, p);
    return e != cudaSuccess ? e : launch_tree_merge(p, pdl, stream);
}

}  // namespace mla
