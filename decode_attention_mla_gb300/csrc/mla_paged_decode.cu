// mla_paged_decode.cu -- attention over the 4-bit paged cache for few query rows:
// warp-level MMAs on values widened in registers (include/mla_paged.h).
//
// Sixteen query rows (token * heads + head) are one MMA tile.  The tcgen05 kernel (mla_paged_attend.cu) passes 470 KB
// through each SM's shared memory per 128 cache rows of a pair, whatever the number of query rows.  Here rows stay as they
// are in shared memory (416 bytes) and are widened in registers: straight into the fragments of Q K^T, and by way of shared
// memory, which transposes them, into those of P V.
//
// A group of four warps shares the 32 rows of a slot.  Warp w has features 128 w .. + 127 (and 16 of the 64 key
// values): it widens them once, into the fragments of Q K^T and to shared memory of its own, from where ldmatrix
// brings them back transposed for P V.  Its scores are partial sums, which the warps exchange through shared memory;
// warp w then has the whole scores of rows 8 w .. + 7, and hands their probabilities to the others; and its part of O,
// 16 x 128 fp32, stays in registers.  Two groups take slots in turn, each with a running maximum and sum of its own,
// and are joined at an item's end.  (Measured on 32 requests of 16 heads, 157 us now: values widened a second time from the
// bytes for P V, 187; two chains of products beside each other in the place of four, 183; transposed by movmatrix instead of
// through shared memory, 180; three groups, which have 144 registers a thread, 187; queries read from shared memory, without a
// split of the registers, 168; an item's end left to one group, 162; the next slot's scores between a slot's softmax and its P V, 177.)
//
// Orders.  The contraction over features may go in any order: lane 4 g + j has, of row g of eight, features 16 j ..
// 16 j + 15 of 64 (a block: eight bytes of codes), four to a k-step.  Rows of a slot lie 416 bytes apart, eight banks on, so
// four rows' eight banks each are all 32.
//
// A code times its scale is exact in f16 (six bits, 2^-10 .. 2688).  Queries are f16 times a power of two per row, probabilities
// f16 times 2^7, key values and their queries bf16, as in mla_paged_attend.cu; sums are fp32.  Codes are finite whatever
// the bytes, and a scale's NaN becomes 0 in P V (in Q K^T it stays: the row's scores are NaN); so rows that nobody
// attends need no clearing: their scores are masked, their probabilities 0.
//
// Work split: units of 64 rows (a slot per group) of all requests' blocks of sixteen query rows, one equal run per SM; pieces and
// their merge as in mla_tree_attend.cu.
//
// Bound: 26 cycles of shared memory per row and SM (16 of them the widened values' way there and back, 4 the partial
// scores'), beside 17 of MMAs and 19 for its bytes from HBM; what is measured is 39, the rest being the chain from a
// slot's bytes to its P V, which two warps a scheduler hide in part.  Bytes alone, nothing computed: 87 us of those 157.
//
// Warps: 0-3 and 4-7 the groups, 8 bulk copies and the run's items, 9 empty requests, 10 and 11 none.
#include <cmath>

#include "mla_paged.cuh"

namespace mla {
namespace {

constexpr int kGroups = 2;                                 // (that halve an item's O between them at its end)
constexpr int kSlotRows = 32, kUnitRows = kGroups * kSlotRows;
constexpr int kSlotBytes = kSlotRows * MLA_Q4_ROW;
constexpr int kRing = 3 * kGroups;                         // (131072 rows, 16 heads: 34 us; with 4 * kGroups 38, 2 * kGroups 34, but
                                                           // 32 requests 165 for 162)
constexpr int kWarps = 4;                                  // of a group
constexpr int kGroupThreads = 32 * kWarps, kComputeThreads = kGroups * kGroupThreads;
constexpr int kProducerWarp = kGroups * kWarps, kEmptyWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kProducerWarp + 4);
// Three warpgroups of 168 registers a thread at launch: two that compute, and one for the rest.
constexpr int kLaunchRegs = 168, kComputeRegs = 208, kOtherRegs = 88;
static_assert(kThreads == 384 && kGroups * kComputeRegs + kOtherRegs <= 3 * kLaunchRegs, "an increase never waits for more than there is");
constexpr int kBarAll = 1, kBarGroup = 2;                  // hardware barriers: of all groups, of each
constexpr int kBlockRows = kDecodeBlockRows;
constexpr float kRescaleLog2 = 8.0f;                       // move the reference when a max grows past 2^8
constexpr float kProbLog2 = 7.0f;                          // P is held times 2^7
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kItems = 4;

// What this run does of a row block: units lo .. hi - 1 of its n_units.
struct __align__(16) Item {
    int b, rb, lo, hi;
    int near, skip, d_pos, n_tok;                          // as r.lo, r.base of the request, and its own
    int n_units, runs, unused[2];                          // runs: that the block lies in, if this one opens it
};

struct __align__(128) Shared {
    uint8_t ring[kRing][kSlotBytes];
    float4 part[kGroups][kWarps][4][32];                         // per group: partial scores by warp, eight rows, lane
    // per group and warp: a slot's values of the warp's features in f16, 256 bytes a row, 16-byte unit u of row r at u ^
    // (r mod 8); at an item's end half of its O, for the other group
    float4 v[kGroups][kWarps][kSlotRows * 16];
    uint4 q[9][kWarps][32];                                // query fragments by k-step (the last: key values), warp, lane
    uint16_t p[kGroups][16][40];                                 // per group: probabilities, row by row (padded)
    float red[kGroups][kWarps][16];                        // per group: maxima or sums by warp, row
    float top[kGroups][16], sum[kGroups][16];              // ... at an item's end
    float factor[16];                                      // of the query rows' scores
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
// slot) of one of a unit's slots.
__device__ void produce(const PagedParams& p, Shared& sh, int lane) {
    const int total = count_units(p, lane);
    const int per = (total + p.clusters - 1) / p.clusters, cta = blockIdx.x;
    const int u0 = static_cast<int>(min(static_cast<long long>(per) * cta, static_cast<long long>(total)));
    const int u1 = min(u0 + per, total);
    const uint64_t policy = l2_policy_evict_normal();
    const int box = min(1 << p.cache.row_shift, kSlotRows), boxes = kSlotRows / box;   // of a slot
    const bool mine = lane < kGroups * boxes;
    const int row = lane * box;                            // of the unit
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
                for (int q = 0; q < kGroups; ++q) {
                    if (turn > 0 && !wait(sh, &sh.empty[ring], (turn - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t here = have >> (q * boxes) & ((1u << boxes) - 1);
                    if (lane == 0) {
                        // eight rows a bit
                        uint32_t v = 0;
                        for (int k = 0; k < 4; ++k) v |= (here >> (8 * k / box) & 1) << k;
                        sh.valid[ring] = v;
                        mbar_arrive_expect_tx(&sh.full[ring], __popc(here) * box * MLA_Q4_ROW);
                    }
                    __syncwarp();
                    if (lane >= q * boxes && lane < (q + 1) * boxes && src)
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

// (Orders no other access: what it writes is read behind the group's next barrier.)
__device__ __forceinline__ void store_values(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

// The first group: the block's query rows as fragments.  A lane has rows g and g + 8, features 128 w + 64 k + 16 j .. + 15
// (k = 0, 1), key values 16 w + 4 j .. + 3.
__device__ __forceinline__ void load_queries(const PagedParams& p, Shared& sh, int w, int lane, long long row0, int live) {
    const int g = lane >> 2, j = lane & 3;
    uint4 x[2][4];
    uint2 y[2];
    const float inv_kv = 1.f / p.kv_scale;                 // a power of two
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint16_t* src = p.q + (row0 + g + 8 * h) * kDRow;
        const bool there = g + 8 * h < live;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[h][k] = there ? reinterpret_cast<const uint4*>(src + 128 * w + 64 * (k >> 1) + 16 * j)[k & 1] : make_uint4(0, 0, 0, 0);
        y[h] = there ? *reinterpret_cast<const uint2*>(src + kDLatent + 16 * w + 4 * j) : make_uint2(0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float top = 0.f, rope = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
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
        if (j == 0) sh.red[0][w][g + 8 * h] = top;
    }
    named_barrier_sync(kBarGroup, kGroupThreads);
    float scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sh.red[0][k][g + 8 * h]);
        const int e = query_exp(p, top);
        scale[h] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        if (w == 0 && j == 0) sh.factor[g + 8 * h] = p.unit * power_of_two(factor_exp(p, e));
    }
    // k-step 2 k + s: features 64 (k / 2) + 16 j + 8 (k mod 2) + 4 s, + 1 (registers 0, 1) and + 2, + 3 (2, 3); rows g (0, 2)
    // and g + 8 (1, 3)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a[4] = {x[0][k].x, x[0][k].y, x[0][k].z, x[0][k].w}, b[4] = {x[1][k].x, x[1][k].y, x[1][k].z, x[1][k].w};
        auto f16 = [](uint32_t v, float by) {
            return pack_f16x2(__uint_as_float(v << 16) * by, __uint_as_float(v & 0xffff0000u) * by);
        };
#pragma unroll
        for (int s = 0; s < 2; ++s)
            sh.q[2 * k + s][w][lane] = make_uint4(f16(a[2 * s], scale[0]), f16(b[2 * s], scale[1]), f16(a[2 * s + 1], scale[0]),
                                                  f16(b[2 * s + 1], scale[1]));
    }
    auto bf16 = [&](uint32_t v, float by) {
        return pack_bf16x2(__uint_as_float(v << 16) * by * inv_kv, __uint_as_float(v & 0xffff0000u) * by * inv_kv);
    };
    sh.q[8][w][lane] = make_uint4(bf16(y[0].x, scale[0]), bf16(y[1].x, scale[1]), bf16(y[0].y, scale[0]), bf16(y[1].y, scale[1]));
}

__device__ void compute(const PagedParams& p, Shared& sh, int group, int w, int lane) {
    const int g = lane >> 2, j = lane & 3;
    const int bar = kBarGroup + group;
    // addresses: values written (unit 2 j of row g), values read (transposed), P read
    const uint32_t values = smem_u32(sh.v[group][w]);
    const uint32_t v_write = values + g * 256, v_read = values + (8 * (lane >> 3 & 1) + (lane & 7)) * 256;
    const uint32_t p_read = smem_u32(&sh.p[group][(lane & 7) + 8 * (lane >> 3 & 1)][8 * (lane >> 4)]);
    int ring = group, turn = 0;
    // A hardware barrier has no time limit, so nobody leaves one alone: all leave together at an item's beginning; a group
    // whose wait runs out in the middle meets the others at the item's end, and all leave there.
    for (int item = 0;; ++item) {
        const bool there = wait(sh, &sh.item_full[item % kItems], (item / kItems) & 1);
        if (named_barrier_or(kBarAll, kComputeThreads, !there)) {
            if (lane == 0) raise(p, sh);
            return;
        }
        const Item& it = sh.items[item % kItems];
        if (it.b < 0) return;
        const int live = min(it.n_tok * p.heads - it.rb * kBlockRows, kBlockRows);
        const long long row0 = static_cast<long long>(it.b) * p.tokens * p.heads + it.rb * kBlockRows;
        if (group == 0) load_queries(p, sh, w, lane, row0, live);
        named_barrier_sync(kBarAll, kComputeThreads);
        uint4 held[9];                                     // this lane's query fragments
#pragma unroll
        for (int k = 0; k < 9; ++k) held[k] = sh.q[k][w][lane];
        const float c2[2] = {sh.factor[g], sh.factor[g + 8]};
        // slots whose rows every token attends: up to all_to, from all_from on or before sink
        const int all_to = row_int(static_cast<long long>(it.d_pos) + 1);
        const int all_from = p.window > 0 ? row_int(static_cast<long long>(it.d_pos) + it.n_tok - p.window) : 0;
        const int units = it.hi, near = it.near, skip = it.skip;
        float o[16][4];
#pragma unroll
        for (int m = 0; m < 16; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[m][k] = 0.f;
        float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int unit = it.lo; unit < units; ++unit) {
            const int t0 = (unit < near ? unit : unit + skip) * kUnitRows + kSlotRows * group;
            const bool bad = !wait(sh, &sh.full[ring], turn & 1);
            const uint8_t* slot = sh.ring[ring];
            const uint32_t valid = sh.valid[ring];
            // ---- the slot's values of this warp's features, widened once: into the fragments of its partial scores, and
            // to shared memory for P V.  Eight rows of each of four chains of products side by side
            float acc[4][4];
            const uint8_t* at = slot + g * MLA_Q4_ROW;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint2 rope = *reinterpret_cast<const uint2*>(at + 8 * e * MLA_Q4_ROW + kQ4Rope + 32 * w + 8 * j);
                const uint4 q = held[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[e][k] = 0.f;
                mma_bf16(acc[e], {q.x, q.y, q.z, q.w}, rope.x, rope.y);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint2 raw[4];
                uint32_t by[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    raw[e] = *reinterpret_cast<const uint2*>(at + 8 * e * MLA_Q4_ROW + 64 * w + 32 * k + 8 * j);
                    const uint32_t s = at[8 * e * MLA_Q4_ROW + kQ4Scales + 8 * w + 4 * k + j];
                    by[e] = widen_e4m3(static_cast<uint16_t>(s | s << 8));
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t h[4][4];
                    const uint4 q0 = held[4 * k + 2 * i], q1 = held[4 * k + 2 * i + 1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        widen_e2m1(i == 0 ? raw[e].x : raw[e].y, h[e]);
                        const uint32_t finite = clean_nan(by[e]);
                        // (a scale's NaN makes the row's scores NaN, through one of its products, but no value of V)
                        const uint32_t first = i == 0 ? mul_f16x2(h[e][0], by[e]) : 0u;
#pragma unroll
                        for (int n = 0; n < 4; ++n) h[e][n] = mul_f16x2(h[e][n], finite);
                        mma_f16(acc[e], {q0.x, q0.y, q0.z, q0.w}, i == 0 ? first : h[e][0], h[e][1]);
                        store_values(v_write + 2048 * e + (((8 * k + 2 * j + i) ^ g) << 4), h[e][0], h[e][1], h[e][2],
                                     h[e][3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma_f16(acc[e], {q1.x, q1.y, q1.z, q1.w}, h[e][2], h[e][3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sh.part[group][w][e][lane] = make_float4(acc[e][0], acc[e][1], acc[e][2], acc[e][3]);
            if (named_barrier_or(bar, kGroupThreads, bad)) {
                if (lane == 0) raise(p, sh);
                named_barrier_or(kBarAll, kComputeThreads, true);
                return;
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
                for (int k = 0; k < 4; ++k) e[k] = ex2_approx(s[k] - base[k >> 1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint32_t*>(&sh.p[group][g + 8 * h][8 * w + 2 * j]) = pack_f16x2(e[2 * h], e[2 * h + 1]);
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
                        for (int m = 0; m < 16; ++m) {
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
            for (int step = 0; step < 2; ++step) {
                uint32_t a[4];
                ldmatrix_x4(a, p_read + 32 * step);
#pragma unroll
                for (int m = 0; m < 16; m += 2) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(b, v_read + 4096 * step + (((m + (lane >> 4)) ^ (lane & 7)) << 4));
                    mma_f16(o[m], a, b[0], b[1]);
                    mma_f16(o[m + 1], a, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[ring]);
            ring += kGroups;
            if (ring >= kRing) {
                ring -= kRing;
                ++turn;
            }
        }
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
        if (w == 0 && j == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sh.top[group][g + 8 * h] = m_ref[h];
                sh.sum[group][g + 8 * h] = l[h];
            }
        }
        // each group hands half of its features' O to the other (its own values of the other's half of the slot's are used up)
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const float(&give)[4] = group == 0 ? o[8 + m] : o[m];
            sh.v[group][w][32 * m + lane] = make_float4(give[0], give[1], give[2], give[3]);
            if (group == 1) {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[m][k] = o[8 + m][k];
            }
        }
        if (named_barrier_or(kBarAll, kComputeThreads, false)) return;   // a group has left
        {
            const int other = 1 - group;
            float own[2], theirs[2], lse2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                const float t = sh.top[other][r], m = fmaxf(m_ref[h], t);
                // (a group without rows has the sum 0 and O = 0; a NaN stays one)
                own[h] = m_ref[h] > -INFINITY ? ex2_approx(m_ref[h] - m) : 1.f;
                theirs[h] = t > -INFINITY ? ex2_approx(t - m) : 1.f;
                const float sum = fmaf(sh.sum[other][r], theirs[h], l[h] * own[h]);
                const float inv = sum == 0.f ? 0.f : p.kv_scale / sum;
                lse2[h] = sum == 0.f ? -INFINITY : (m - kProbLog2) + log2f(sum);
                own[h] *= inv;
                theirs[h] *= inv;
            }
            const bool whole = it.hi - it.lo == it.n_units;
            const int slot = kTreePieces * static_cast<int>(blockIdx.x) + (item == 0 ? 0 : 1);
            if (group == 0 && w == 0 && j == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (g + 8 * h >= live) continue;
                    if (whole)
                        p.a.lse[row0 + g + 8 * h] = lse2[h] * kLn2;
                    else
                        p.lse_part[slot * 32 + g + 8 * h] = lse2[h];
                }
            }
            if (group == 0 && w == 0 && lane == 0 && !whole && it.lo == 0)
                p.merge[blockIdx.x] = TreeMerge{it.b, it.rb, live | (item == 0 ? 0 : 1) << 16, it.runs};
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const float4 v = sh.v[other][w][32 * m + lane];
                o[m][0] = fmaf(v.x, theirs[0], o[m][0] * own[0]);
                o[m][1] = fmaf(v.y, theirs[0], o[m][1] * own[0]);
                o[m][2] = fmaf(v.z, theirs[1], o[m][2] * own[1]);
                o[m][3] = fmaf(v.w, theirs[1], o[m][3] * own[1]);
            }
            // rows g, g + 8; features 128 w + 64 group + 8 m + 2 j, + 1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                if (r >= live) continue;
                const int from = 128 * w + 64 * group + 2 * j;
                if (!whole) {
                    float* piece = p.part + (static_cast<long long>(slot) * (kDLatent / 4) * 32 + r) * 4 + (j & 1) * 2;
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        *reinterpret_cast<float2*>(piece + (32 * w + 16 * group + 2 * m + (j >> 1)) * 128) = make_float2(o[m][2 * h], o[m][2 * h + 1]);
                } else if (p.a.out_fp32) {
                    float* dst = static_cast<float*>(p.a.out) + (row0 + r) * kDLatent + from;
#pragma unroll
                    for (int m = 0; m < 8; ++m) *reinterpret_cast<float2*>(dst + 8 * m) = make_float2(o[m][2 * h], o[m][2 * h + 1]);
                } else {
                    uint16_t* dst = static_cast<uint16_t*>(p.a.out) + (row0 + r) * kDLatent + from;
#pragma unroll
                    for (int m = 0; m < 8; ++m) *reinterpret_cast<uint32_t*>(dst + 8 * m) = pack_bf16x2(o[m][2 * h], o[m][2 * h + 1]);
                }
            }
        }
        // (the others' O has been read when all meet at the next item's beginning)
        if (lane == 0) mbar_arrive(&sh.item_empty[item % kItems]);
    }
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
            mbar_init(&sh.item_empty[i], kGroups * kWarps);
        }
        mbar_init(&sh.stall_bar, 1);
        sh.abort_flag = 0;
        mbar_init_fence();
    }
    __syncthreads();
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp < kProducerWarp) {
        warpgroup_regs_increase<kComputeRegs>();
        compute(p, sh, warp / kWarps, warp % kWarps, lane);
    } else {
        warpgroup_regs_decrease<kOtherRegs>();
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
        }
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
    // (the split of the registers counts on those of the launch)
    cudaFuncAttributes fa{};
    const cudaError_t e = cudaFuncGetAttributes(&fa, mla_paged_decode_kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kLaunchRegs || fa.maxThreadsPerBlock < kThreads) return cudaErrorInvalidConfiguration;
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
    // (it waits for this kernel's end before it reads: it may always be launched ahead)
    return e != cudaSuccess ? e : launch_tree_merge(p, true, stream);
}

}  // namespace mla
