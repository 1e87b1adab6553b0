// mla_paged_append.cu -- new rows of the 4-bit cache and the queries beside them:
// norms, rotation, quantisation and the write, in one pass; and rows read back
// (include/mla_paged.h).
//
//   x' = x * rstd * w,   rstd = (mean(x^2) + eps)^(-1/2)
//   block of 16: s = E4M3(max|x'| / (6 kv_scale)),  code = E2M1(x' / (s kv_scale))
//
// A value next to a border between two codes falls to the side that the last bit of
// rstd says, and one code more or less is a third of the value.  So rstd is the fp32
// number next to the exact one: the sum of squares is kept as a pair of fp32
// numbers (squares of bf16 values are exact in fp32; the pair's sums, Knuth's two-sum,
// lose 2^-48), and the reciprocal root is corrected once with the residual 1 - m r^2,
// taken exactly with fma.  The products x * rstd * w are rounded one after the other.
//
// Bound: bytes (128 in and 128 out per query head; 1152 in and 416 out per row).  Warps work
// alone, as in mla_rope.cu: a warp takes up to 32 heads of one token, eight lanes a head, or
// the token's row, of which a lane has 16 consecutive latent values: a block with its scale.
// 4696 ragged tokens of 128 heads (161 MB): 32 us, 5.0 TB/s; the same loads and stores with nothing computed take 28.5.
// Heads' arithmetic is on pairs of fp32 numbers, and the norm's sums and roots of a warp's 32 heads are one lane's each
// (one number at a time, every lane a root per head: 38 us, issue slots half taken).
#include <cmath>
#include <cstdint>

#include <cuda_fp8.h>

#include "device_utils.cuh"
#include "mla_q4.cuh"
#include "mla_rope.cuh"

namespace mla {
namespace {

// Registers held to 72, seven blocks per SM: 4696 tokens of 128 heads 32 us; with 80 and six blocks 35, blocks of 256 threads
// 36 (a warp's 32 heads are 4 KB on their way: with 28 warps, seven eighths of what hides the memory's latency).
constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 7;
constexpr int kHeadPasses = 8;                             // of four heads each, per warp

// (hi, lo) += x, hi + lo exact but for what leaves lo.
__device__ __forceinline__ void two_add(float& hi, float& lo, float x) {
    const float s = __fadd_rn(hi, x);
    const float t = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(x, t));
    hi = s;
}
// The fp32 number next to (hi + lo)^(-1/2).
__device__ __forceinline__ float rsqrt_pair(float hi, float lo) {
    const float r = rsqrtf(hi);
    if (!(hi > 0x1p-120f && hi < 0x1p120f)) return r;      // (0, infinity, NaN: as rsqrt; no bits to win at the ends)
    const float p = __fmul_rn(r, r), pe = fmaf(r, r, -p);
    const float h = __fmul_rn(hi, p), he = fmaf(hi, p, -h);
    const float e = __fsub_rn(1.f, h) - he - fmaf(hi, pe, __fmul_rn(lo, p));
    return fmaf(0.5f * r, e, r);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Eight values as E2M1, the first in the low bits.
__device__ __forceinline__ uint32_t narrow_e2m1(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Norm of 64 elements in eight lanes (each lane its unit's eight; the sum is that of all lanes
// with the same lane / 8).
__device__ __forceinline__ void norm_unit(float (&f)[8], const float (&w)[8], float eps) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = rsqrtf(fmaf(sum, 1.f / kDRope, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
}

// Two fp32 numbers in a 64-bit register, and products of both.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// A unit's four pairs (x, y): x of pairs 0, 1 and of 2, 3, then y.
template <bool kInterleaved>
__device__ __forceinline__ void widen_pairs(const uint4 v, uint64_t (&x)[2], uint64_t (&y)[2]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    auto lo = [&](int i) { return __uint_as_float(w[i] << 16); };
    auto hi = [&](int i) { return __uint_as_float(w[i] & 0xffff0000u); };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[i] = kInterleaved ? pack2(lo(2 * i), lo(2 * i + 1)) : pack2(lo(i), hi(i));
        y[i] = kInterleaved ? pack2(hi(2 * i), hi(2 * i + 1)) : pack2(lo(2 + i), hi(2 + i));
    }
}
template <bool kInterleaved>
__device__ __forceinline__ uint4 narrow_pairs(const uint64_t (&x)[2], const uint64_t (&y)[2]) {
    const float2 a = unpack2(x[0]), b = unpack2(x[1]), c = unpack2(y[0]), d = unpack2(y[1]);
    if (kInterleaved) return make_uint4(pack_bf16x2(a.x, c.x), pack_bf16x2(a.y, c.y), pack_bf16x2(b.x, d.x), pack_bf16x2(b.y, d.y));
    return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y));
}

struct AppendParams4 {
    mla_paged_append_args a;
    PagedCache cache;
    float kv_scale, sixth;                                 // 1 / (6 kv_scale)
};

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) mla_paged_append_kernel(const __grid_constant__ AppendParams4 p,
                                                                    int units_per_token) {
    grid_dependency_wait();
    allow_dependent_launch();
    const mla_paged_append_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(blockIdx.x) * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int n = w / units_per_token, part = w - n * units_per_token;
    const int b = blockIdx.y;
    if (n >= a.tokens) return;
    const bool is_row = p.cache.pages && part == units_per_token - 1;
    // (loads that wait for nothing, side by side)
    const int n_tok = a.n_tokens ? a.n_tokens[b] : a.tokens;
    const int pos = a.positions[static_cast<long long>(b) * a.tokens + n];
    const int d = is_row ? a.d_pos[b] : 0;
    if (n >= n_tok) return;
    const int half = a.rot_dim >> 1;
    const int u = lane & 7;
    const bool rotated = 4 * u < half;                     // half is a multiple of 4: a unit whole or not at all
    int lo, hi;
    unit_offsets(u, half, kInterleaved, lo, hi);
    if (is_row) {
        // ---- the row
        const long long t = static_cast<long long>(d) + n;
        if (d < 0 || t >= paged_rows(p.cache)) return;     // uniform over the warp, as below
        const int page = page_of(p.cache, b, static_cast<int>(t));
        const uint4* c = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c) + b * a.c_batch +
                                                        n * a.c_token) + 2 * lane;
        const uint4 v0 = c[0], v1 = c[1];
        uint4 k = make_uint4(0, 0, 0, 0);
        if (lane < 8)
            k = load_unit(static_cast<const uint16_t*>(a.k_rope) + b * a.k_rope_batch + n * a.k_rope_token, lo, hi);
        uint4 g0 = make_uint4(0, 0, 0, 0), g1 = g0, gk = g0;
        if (a.c_norm) {
            g0 = static_cast<const uint4*>(a.c_norm)[2 * lane];
            g1 = static_cast<const uint4*>(a.c_norm)[2 * lane + 1];
        }
        if (a.k_norm) gk = load_unit(static_cast<const uint16_t*>(a.k_norm), lo, hi);
        if (page < 0) return;
        uint8_t* row = row_in(p.cache, page, static_cast<int>(t));
        float sn0, cs0, cs[4], sn[4];
        pair_angle(pos, a.turns, half, a.amplitude, lane, sn0, cs0);
        unit_angles(u, sn0, cs0, cs, sn);
        float f[16];
        {
            float x[8];
            widen8(v0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = x[i];
            widen8(v1, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[8 + i] = x[i];
        }
        if (a.c_norm) {
            float sum = 0.f, low = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) two_add(sum, low, __fmul_rn(f[i], f[i]));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                // (each pair of lanes adds the larger lane's numbers to the smaller's: the same in both)
                const float s = __shfl_xor_sync(0xffffffffu, sum, o), l = __shfl_xor_sync(0xffffffffu, low, o);
                const bool up = lane & o;
                float x = up ? s : sum, xl = up ? l : low;
                two_add(x, xl, up ? sum : s);
                sum = x;
                low = xl + (up ? low : l);
            }
            sum *= 1.f / kDLatent;
            low *= 1.f / kDLatent;
            two_add(sum, low, a.eps);
            const float r = rsqrt_pair(sum, low);
            float x[8];
            widen8(g0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], r), x[i]);
            widen8(g1, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[8 + i] = __fmul_rn(__fmul_rn(f[8 + i], r), x[i]);
        }
        float top = fabsf(f[0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) top = max_nan(top, fabsf(f[i]));
        const uint8_t scale =
            __nv_cvt_float_to_fp8(__fmul_rn(top, p.sixth), __NV_SATFINITE, __NV_E4M3);   // NaN stays NaN
        const float step = __fmul_rn(__low2float(__half2(__nv_cvt_fp8_to_halfraw(scale, __NV_E4M3), __half())), p.kv_scale);
        const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __fmul_rn(f[i], inv);
        reinterpret_cast<uint2*>(row)[lane] = make_uint2(narrow_e2m1(f), narrow_e2m1(f + 8));
        row[kQ4Scales + lane] = scale;
        float x[8];
        widen8(k, x);
        if (a.k_norm) {
            float g[8];
            widen8(gk, g);
            norm_unit(x, g, a.eps);
        }
        if (rotated) rotate_unit(x, kInterleaved, cs, sn);
        if (lane < 8) {
            const uint4 o = narrow8(x);
            uint16_t* dst = reinterpret_cast<uint16_t*>(row + kQ4Rope);
            *reinterpret_cast<uint2*>(dst + lo) = make_uint2(o.x, o.y);
            *reinterpret_cast<uint2*>(dst + hi) = make_uint2(o.z, o.w);
        }
        return;
    }
    // ---- up to 32 heads of the token: all loads before the angles
    uint4 v[kHeadPasses];
    const int h0 = kHeadPasses * 4 * part + (lane >> 3);
    const uint16_t* src = static_cast<const uint16_t*>(a.q_rope) + b * a.q_rope_batch + n * a.q_rope_token;
#pragma unroll
    for (int j = 0; j < kHeadPasses; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (h0 + 4 * j < a.heads) {
            const uint16_t* q = src + (h0 + 4 * j) * a.q_rope_head;
            v[j] = kInterleaved ? *reinterpret_cast<const uint4*>(q + lo) : load_unit(q, lo, hi);
        }
    }
    float sn0, cs0, cs[4], sn[4];
    pair_angle(pos, a.turns, half, a.amplitude, lane, sn0, cs0);
    unit_angles(u, sn0, cs0, cs, sn);
    // x' = x r wx cos - y r wy sin,  y' = y r wy cos + x r wx sin (a pair that is not rotated: x r wx, y r wy): the weights
    // go into the angles
    uint64_t wx[2] = {pack2(1.f, 1.f), pack2(1.f, 1.f)}, wy[2] = {wx[0], wx[0]};
    if (a.q_norm) widen_pairs<kInterleaved>(load_unit(static_cast<const uint16_t*>(a.q_norm), lo, hi), wx, wy);
    uint64_t xx[2], yx[2], yy[2], xy[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t c = rotated ? pack2(cs[2 * i], cs[2 * i + 1]) : pack2(1.f, 1.f);
        xx[i] = mul2(wx[i], c);
        yy[i] = mul2(wy[i], c);
        xy[i] = mul2(wx[i], pack2(sn[2 * i], sn[2 * i + 1]));
        yx[i] = mul2(wy[i], pack2(-sn[2 * i], -sn[2 * i + 1]));
    }
    float r = 1.f;
    if (a.q_norm) {
        // sums of squares of all eight passes' heads; lane u of eight ends with those of pass u
        float sum[kHeadPasses];
#pragma unroll
        for (int j = 0; j < kHeadPasses; ++j) {
            uint64_t x[2], y[2];
            widen_pairs<kInterleaved>(v[j], x, y);
            const float2 t = unpack2(fma2(y[1], y[1], fma2(y[0], y[0], fma2(x[1], x[1], mul2(x[0], x[0])))));
            sum[j] = t.x + t.y;
        }
        static_assert(kHeadPasses == 8, "as many passes as a head has lanes");
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int j = 0; j < o; ++j) {
                const float mine = up ? sum[j + o] : sum[j], other = up ? sum[j] : sum[j + o];
                sum[j] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
        r = rsqrtf(fmaf(sum[0], 1.f / kDRope, a.eps));
    }
    uint16_t* dst = static_cast<uint16_t*>(a.q_out) + b * a.q_out_batch + n * a.q_out_token;
#pragma unroll
    for (int j = 0; j < kHeadPasses; ++j) {
        if (kHeadPasses * 4 * part + 4 * j >= a.heads) break;   // uniform over the warp
        uint64_t x[2], y[2];
        widen_pairs<kInterleaved>(v[j], x, y);
        if (a.q_norm) {
            const float f = __shfl_sync(0xffffffffu, r, (lane & 24) | j);
            const uint64_t by = pack2(f, f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[i] = mul2(x[i], by);
                y[i] = mul2(y[i], by);
            }
        }
        uint64_t rx[2], ry[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rx[i] = mul2(x[i], xx[i]);
            ry[i] = mul2(y[i], yy[i]);
            if (rotated) {
                rx[i] = fma2(y[i], yx[i], rx[i]);
                ry[i] = fma2(x[i], xy[i], ry[i]);
            }
        }
        if (h0 + 4 * j < a.heads) {
            const uint4 o = narrow_pairs<kInterleaved>(rx, ry);
            uint16_t* q = dst + (h0 + 4 * j) * a.q_out_head;
            if (kInterleaved) {
                *reinterpret_cast<uint4*>(q + lo) = o;
            } else {
                *reinterpret_cast<uint2*>(q + lo) = make_uint2(o.x, o.y);
                *reinterpret_cast<uint2*>(q + hi) = make_uint2(o.z, o.w);
            }
        }
    }
}

struct ReadParams {
    mla_paged_read_args a;
    PagedCache cache;
    float kv_scale;
};

// A warp per row: a lane has a block of 16 values, and two of the 64 key values.
__global__ void __launch_bounds__(kThreads) mla_paged_read_kernel(const __grid_constant__ ReadParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int n = static_cast<int>(blockIdx.x) * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int b = blockIdx.y;
    if (n >= p.a.rows) return;
    const int n_rows = p.a.n_rows ? p.a.n_rows[b] : p.a.rows;
    const long long t = static_cast<long long>(p.a.first ? p.a.first[b] : 0) + n;
    if (n >= n_rows) return;
    const int page = t >= 0 && t < paged_rows(p.cache) ? page_of(p.cache, b, static_cast<int>(t)) : -1;
    uint16_t* out = static_cast<uint16_t*>(p.a.out) + b * p.a.out_batch + n * p.a.out_row;
    uint32_t o[8], key = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0;
    if (page >= 0) {
        const uint8_t* row = row_in(p.cache, page, static_cast<int>(t));
        const uint2 w = reinterpret_cast<const uint2*>(row)[lane];
        const uint8_t scale = row[kQ4Scales + lane];
        key = reinterpret_cast<const uint32_t*>(row + kQ4Rope)[lane];
        const uint32_t s = widen_e4m3(static_cast<uint16_t>(scale | scale << 8));
        uint32_t h[8];
        widen_e2m1(w.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
        widen_e2m1(w.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = f16x2_to_float2(mul_f16x2(h[i], s));   // exact
            o[i] = pack_bf16x2(v.x * p.kv_scale, v.y * p.kv_scale);
        }
    }
    uint4* dst = reinterpret_cast<uint4*>(out) + 2 * lane;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    reinterpret_cast<uint32_t*>(out + kDLatent)[lane] = key;
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool off8(long long stride) { return stride % 8 != 0; }
// Several entries of `width` elements lie in one place, or across one another.
bool piled(int count, long long stride, int width) { return count > 1 && stride > -width && stride < width; }

int check(const mla_paged_append_args* a) {
    if (!a || a->batch < 1 || a->batch > 65535 || a->tokens < 1 || a->tokens > (1 << 28)) return MLA_EINVAL;
    if (a->heads < 0 || a->heads > 128) return MLA_EUNSUPPORTED;
    if (a->rot_dim < 8 || a->rot_dim > 64 || a->rot_dim % 8 != 0) return MLA_EUNSUPPORTED;
    if (a->interleaved != 0 && a->interleaved != 1) return MLA_EINVAL;
    if (!(a->amplitude > 0.f) || !std::isfinite(a->amplitude)) return MLA_EINVAL;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return MLA_EINVAL;
    if (!a->turns || !a->positions) return MLA_EINVAL;
    const bool rows = a->cache.pages != nullptr;
    if (rows ? (!a->c || !a->k_rope || !a->d_pos) : (a->c || a->k_rope || a->d_pos || a->c_norm || a->k_norm))
        return MLA_EINVAL;
    if (!rows && a->heads == 0) return MLA_EINVAL;
    if (a->heads > 0 ? (!a->q_rope || !a->q_out) : (a->q_rope || a->q_out || a->q_norm)) return MLA_EINVAL;
    if (rows) {
        const int rc = check_cache(&a->cache);
        if (rc != MLA_OK) return rc;
        if (off(a->c, 16) || off(a->k_rope, 16) || off8(a->c_batch) || off8(a->c_token) || off8(a->k_rope_batch) ||
            off8(a->k_rope_token) || off(a->d_pos, 4) || off(a->c_norm, 16) || off(a->k_norm, 16))
            return MLA_EALIGN;
    }
    if (a->heads > 0 &&
        (off(a->q_rope, 16) || off(a->q_out, 16) || off8(a->q_rope_batch) || off8(a->q_rope_token) ||
         off8(a->q_rope_head) || off8(a->q_out_batch) || off8(a->q_out_token) || off8(a->q_out_head) ||
         off(a->q_norm, 16)))
        return MLA_EALIGN;
    if (off(a->turns, 8) || off(a->positions, 4) || off(a->n_tokens, 4)) return MLA_EALIGN;
    if (a->heads > 0 && (piled(a->batch, a->q_out_batch, kDRope) || piled(a->tokens, a->q_out_token, kDRope) ||
                         piled(a->heads, a->q_out_head, kDRope)))
        return MLA_EINVAL;
    return MLA_OK;
}

int launch_blocks(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, long long warps, int batch, void* stream) {
    const long long per = kThreads / 32, blocks = (warps + per - 1) / per;
    if (blocks > 0x7fffffffLL) return MLA_EINVAL;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg->gridDim = dim3(static_cast<unsigned>(blocks), batch);
    cfg->blockDim = dim3(kThreads);
    cfg->stream = static_cast<cudaStream_t>(stream);
    cfg->attrs = attr;
    cfg->numAttrs = 1;
    return MLA_OK;
}

}  // namespace

int check_cache(const mla_paged_cache* c) {
    if (!c->pages || !c->page_table || c->n_pages < 1 || c->columns < 1) return MLA_EINVAL;
    if (c->page_rows < 8 || c->page_rows > 1024 || (c->page_rows & (c->page_rows - 1)) != 0) return MLA_EINVAL;
    if (static_cast<long long>(c->columns) * c->page_rows > 0x7fffff00LL) return MLA_EINVAL;
    if (c->page_stride < static_cast<long long>(c->page_rows) * MLA_Q4_ROW) return MLA_EINVAL;
    int e = 0;
    if (!(c->kv_scale >= 0x1p-64f) || !(c->kv_scale <= 0x1p64f) || std::frexp(c->kv_scale, &e) != 0.5f) return MLA_EINVAL;
    if (c->page_stride % 16 != 0 || off(c->pages, 16) || off(c->page_table, 4)) return MLA_EALIGN;
    return MLA_OK;
}

PagedCache paged_cache(const mla_paged_cache* c) {
    PagedCache p{static_cast<uint8_t*>(c->pages), c->page_stride, c->page_table, c->n_pages, c->columns, 0};
    while ((1 << p.row_shift) < c->page_rows) ++p.row_shift;
    return p;
}

}  // namespace mla

extern "C" int mla_paged_append(const mla_paged_append_args* args, void* stream) {
    int rc = mla::check(args);
    if (rc != MLA_OK) return rc;
    mla::AppendParams4 p{*args, {}, 1.f, 1.f};
    if (args->cache.pages) {
        p.cache = mla::paged_cache(&args->cache);
        p.kv_scale = args->cache.kv_scale;
        p.sixth = static_cast<float>(1.0 / 6.0 / args->cache.kv_scale);
    }
    const int units = (args->heads + 4 * mla::kHeadPasses - 1) / (4 * mla::kHeadPasses) + (args->cache.pages ? 1 : 0);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    rc = mla::launch_blocks(&cfg, &attr, static_cast<long long>(args->tokens) * units, args->batch, stream);
    if (rc != MLA_OK) return rc;
    return mla::launch_status(cudaLaunchKernelEx(
        &cfg, args->interleaved ? mla::mla_paged_append_kernel<true> : mla::mla_paged_append_kernel<false>, p, units));
}

extern "C" int mla_paged_read(const mla_paged_read_args* args, void* stream) {
    if (!args || args->batch < 1 || args->batch > 65535 || args->rows < 1 || args->rows > (1 << 28) || !args->out)
        return MLA_EINVAL;
    int rc = mla::check_cache(&args->cache);
    if (rc != MLA_OK) return rc;
    if (args->out_row < MLA_D_ROW) return MLA_EINVAL;
    if (mla::off(args->out, 16) || mla::off8(args->out_batch) || mla::off8(args->out_row) || mla::off(args->first, 4) ||
        mla::off(args->n_rows, 4))
        return MLA_EALIGN;
    if (mla::piled(args->batch, args->out_batch, MLA_D_ROW)) return MLA_EINVAL;
    const mla::ReadParams p{*args, mla::paged_cache(&args->cache), args->cache.kv_scale};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    rc = mla::launch_blocks(&cfg, &attr, args->rows, args->batch, stream);
    if (rc != MLA_OK) return rc;
    return mla::launch_status(cudaLaunchKernelEx(&cfg, mla::mla_paged_read_kernel, p));
}
