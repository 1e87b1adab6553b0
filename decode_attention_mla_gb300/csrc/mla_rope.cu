// mla_rope.cu -- rotary positions of the new tokens' queries and keys, and the
// append of their rows to the latent cache (include/mla_rope.h).
//
//   (x, y) -> (A (x cos t - y sin t), A (y cos t + x sin t)),   t = p f_j
//
// The angle.  f_j / (2 pi) is held as a 64-bit fraction of a turn F_j; the
// product p F_j taken modulo 2^64 is the exact fraction of a turn at position
// p (F_j's own rounding, 2^-53 relative, moves the angle by less than 1e-9 at
// position 2^20), where fp32 products of far positions would be off by
// hundredths of a radian.  Its top 32 bits, as a signed fraction, go to
// sincospif.
//
// Bound: bytes (128 in and 128 out per query head, 1152 in and 1152 or 576 out
// per row).  One CTA per token: 32 threads take the token's 32 sines and
// cosines once for all heads, eight threads rotate a head (four pairs each, one
// 16-byte or two 8-byte loads), so a thread has the loads of its up to four
// heads in flight before the angles are needed; the last 72 threads move the
// cache row meanwhile.
#include <cmath>
#include <cstdint>

#include <cuda_fp8.h>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_rope.h"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadsPerPass = kRopeThreads / 8;
constexpr int kHeadPasses = 128 / kHeadsPerPass;
constexpr int kRowUnits = kDRow / 8;                       // 72 units of 8 elements
constexpr int kRowThread0 = kRopeThreads - kRowUnits;      // the threads that move the cache row

struct Unit {                                              // four pairs: x[i], y[i]
    float x[4], y[4];
};

__device__ __forceinline__ void widen8(const uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint2 narrow8_e4m3(const float (&f)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(f[i] / scale, __NV_SATFINITE, __NV_E4M3))
                     << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

// Unit u (of 8) of a head's 64 elements: pairs 4u .. 4u + 3.  Interleaved
// pairs are elements 8u .. 8u + 7 (the ones behind rot_dim pass through in
// place).  Half layout: elements 4u .. and half + 4u ..; the pairs behind the
// rotated ones hold the eight copied elements rot_dim + 2 (4u - half) ...
// Element offsets of a unit's two groups of four.
__device__ __forceinline__ void unit_offsets(int u, int half, int interleaved, int& lo, int& hi) {
    if (interleaved) {
        lo = 8 * u;
        hi = 8 * u + 4;
    } else if (4 * u < half) {
        lo = 4 * u;
        hi = half + 4 * u;
    } else {
        lo = 2 * half + 2 * (4 * u - half);
        hi = lo + 4;
    }
}

// The unit's eight elements in the order of its two groups.
__device__ __forceinline__ void rotate_unit(float (&f)[8], int u, int half, int interleaved, const float* cs,
                                            const float* sn) {
    if (4 * u >= half) return;                             // copied elements
    // half is a multiple of 4, so a unit is rotated whole or not at all
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = cs[4 * u + i], s = sn[4 * u + i];
        const int a = interleaved ? 2 * i : i, b = interleaved ? 2 * i + 1 : i + 4;
        const float x = f[a], y = f[b];
        f[a] = x * c - y * s;
        f[b] = y * c + x * s;
    }
}

__device__ __forceinline__ uint4 load_unit(const uint16_t* p, int lo, int hi) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + lo), b = *reinterpret_cast<const uint2*>(p + hi);
    return make_uint4(a.x, a.y, b.x, b.y);
}

__global__ void __launch_bounds__(kRopeThreads) mla_rope_kernel(const mla_rope_args a) {
    __shared__ float cs[MLA_ROPE_MAX_PAIRS], sn[MLA_ROPE_MAX_PAIRS];
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependent_launch();
    for (long long work = blockIdx.x; work < static_cast<long long>(a.batch) * a.tokens; work += gridDim.x) {
        const int b = static_cast<int>(work / a.tokens);
        const int n = static_cast<int>(work - static_cast<long long>(b) * a.tokens);
        if (a.n_tokens && n >= a.n_tokens[b]) continue;    // uniform over the CTA
        const int half = a.rot_dim >> 1;
        // ---- loads of this thread's heads
        const int u = tid & 7;
        int lo, hi;
        unit_offsets(u, half, a.interleaved, lo, hi);
        const uint16_t* qsrc =
            static_cast<const uint16_t*>(a.q_rope) + b * a.q_rope_batch + n * a.q_rope_token;
        uint4 v[kHeadPasses];
#pragma unroll
        for (int i = 0; i < kHeadPasses; ++i) {
            const int h = (tid >> 3) + kHeadsPerPass * i;
            if (h < a.heads) {
                const uint16_t* p = qsrc + h * a.q_rope_head;
                v[i] = a.interleaved ? *reinterpret_cast<const uint4*>(p + lo) : load_unit(p, lo, hi);
            }
        }
        // ---- the cache row's unit
        const int unit = tid - kRowThread0;
        long long row = -1;
        int row_lo = 0, row_hi = 4;
        uint4 rv = make_uint4(0, 0, 0, 0);
        if (a.kv && unit >= 0) {
            const int d = a.d_pos[b];
            const long long r = (a.row_offset ? a.row_offset[b] : 0) + d + n;
            if (d >= 0 && r >= 0 && r < a.kv_rows) row = r;
            if (unit < 64) {
                row_lo = 8 * unit;
                row_hi = row_lo + 4;
                rv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c) + b * a.c_batch +
                                                     n * a.c_token + 8 * unit);
            } else {
                unit_offsets(unit - 64, half, a.interleaved, row_lo, row_hi);
                rv = load_unit(static_cast<const uint16_t*>(a.k_rope) + b * a.k_rope_batch + n * a.k_rope_token,
                               row_lo, row_hi);
                row_lo += kDLatent;
                row_hi += kDLatent;
            }
        }
        // ---- angles, once per token
        const int pos = a.positions[static_cast<long long>(b) * a.tokens + n];
        if (tid < half) {
            const unsigned long long turn =
                static_cast<unsigned long long>(static_cast<long long>(pos)) * a.turns[tid];
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;   // units of pi
            float s, c;
            sincospif(x, &s, &c);
            cs[tid] = a.amplitude * c;
            sn[tid] = a.amplitude * s;
        }
        __syncthreads();
        uint16_t* qdst = static_cast<uint16_t*>(a.q_out) + b * a.q_out_batch + n * a.q_out_token;
#pragma unroll
        for (int i = 0; i < kHeadPasses; ++i) {
            const int h = (tid >> 3) + kHeadsPerPass * i;
            if (h < a.heads) {
                float f[8];
                widen8(v[i], f);
                rotate_unit(f, u, half, a.interleaved, cs, sn);
                const uint4 o = narrow8(f);
                uint16_t* p = qdst + h * a.q_out_head;
                if (a.interleaved) {
                    *reinterpret_cast<uint4*>(p + lo) = o;
                } else {
                    *reinterpret_cast<uint2*>(p + lo) = make_uint2(o.x, o.y);
                    *reinterpret_cast<uint2*>(p + hi) = make_uint2(o.z, o.w);
                }
            }
        }
        if (row >= 0) {
            float f[8];
            widen8(rv, f);
            if (unit >= 64) rotate_unit(f, unit - 64, half, a.interleaved, cs, sn);
            if (a.kv_fp8) {
                const uint2 o = narrow8_e4m3(f, a.kv_scale);
                uint8_t* p = static_cast<uint8_t*>(a.kv) + row * a.row_stride;
                *reinterpret_cast<uint32_t*>(p + row_lo) = o.x;
                *reinterpret_cast<uint32_t*>(p + row_hi) = o.y;
            } else {
                const uint4 o = narrow8(f);
                uint16_t* p = static_cast<uint16_t*>(a.kv) + row * a.row_stride;
                *reinterpret_cast<uint2*>(p + row_lo) = make_uint2(o.x, o.y);
                *reinterpret_cast<uint2*>(p + row_hi) = make_uint2(o.z, o.w);
            }
            if (unit == 0) {
                if (a.row_positions) a.row_positions[row] = pos;
                if (a.row_weights) a.row_weights[row] = 0.f;
            }
        }
        __syncthreads();                                   // cs and sn are rewritten for the next token
    }
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool off8(long long stride) { return stride % 8 != 0; }

int check(const mla_rope_args* a) {
    if (!a || a->batch < 1 || a->batch > 65535 || a->tokens < 1) return MLA_EINVAL;
    if (a->heads < 0 || a->heads > 128) return MLA_EUNSUPPORTED;
    if (a->rot_dim < 8 || a->rot_dim > 64 || a->rot_dim % 8 != 0) return MLA_EUNSUPPORTED;
    if ((a->interleaved != 0 && a->interleaved != 1) || (a->kv_fp8 != 0 && a->kv_fp8 != 1)) return MLA_EINVAL;
    if (!(a->amplitude > 0.f) || !std::isfinite(a->amplitude)) return MLA_EINVAL;
    if (!a->turns || !a->positions) return MLA_EINVAL;
    const bool rows = a->kv != nullptr;
    if (rows ? (!a->c || !a->k_rope || !a->d_pos) : (a->c || a->k_rope || a->row_positions || a->row_weights))
        return MLA_EINVAL;
    if (!rows && a->heads == 0) return MLA_EINVAL;
    if (a->heads > 0 && (!a->q_rope || !a->q_out)) return MLA_EINVAL;
    if (rows) {
        if (a->kv_rows < 1 || a->row_stride < MLA_D_ROW || (a->batch > 1 && !a->row_offset)) return MLA_EINVAL;
        if (a->kv_fp8 && (!(a->kv_scale > 0.f) || !std::isfinite(a->kv_scale))) return MLA_EINVAL;
        if (a->row_stride % (a->kv_fp8 ? 16 : 8) != 0 || off(a->kv, 16) || off(a->c, 16) || off(a->k_rope, 16) ||
            off8(a->c_batch) || off8(a->c_token) || off8(a->k_rope_batch) || off8(a->k_rope_token))
            return MLA_EALIGN;
        if (off(a->d_pos, 4) || off(a->row_offset, 8) || off(a->row_positions, 4) || off(a->row_weights, 4))
            return MLA_EALIGN;
    }
    if (a->heads > 0 &&
        (off(a->q_rope, 16) || off(a->q_out, 16) || off8(a->q_rope_batch) || off8(a->q_rope_token) ||
         off8(a->q_rope_head) || off8(a->q_out_batch) || off8(a->q_out_token) || off8(a->q_out_head)))
        return MLA_EALIGN;
    if (off(a->turns, 8) || off(a->positions, 4) || off(a->n_tokens, 4)) return MLA_EALIGN;
    return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" int mla_rope_table(const mla_rope_spec* spec, unsigned long long* turns) {
    if (!spec || !turns) return MLA_EINVAL;
    const mla_rope_spec s = *spec;
    if (s.rot_dim < 8 || s.rot_dim > 64 || s.rot_dim % 8 != 0) return MLA_EINVAL;
    if (!std::isfinite(s.base) || !(s.base >= 1.0)) return MLA_EINVAL;
    if (s.scaling != MLA_ROPE_PLAIN && s.scaling != MLA_ROPE_LINEAR && s.scaling != MLA_ROPE_YARN) return MLA_EINVAL;
    if (s.scaling != MLA_ROPE_PLAIN && (!std::isfinite(s.factor) || !(s.factor >= 1.0))) return MLA_EINVAL;
    const double pi2 = 6.283185307179586476925;
    double low = 0, high = 0;
    if (s.scaling == MLA_ROPE_YARN) {
        if (!std::isfinite(s.original_ctx) || !(s.original_ctx >= 1.0) || !std::isfinite(s.beta_fast) ||
            !(s.beta_slow > 0.0) || !(s.beta_fast > s.beta_slow) || !(s.base > 1.0))
            return MLA_EINVAL;
        // pair that turns beta times over original_ctx positions
        auto pair_of = [&](double beta) {
            return s.rot_dim * std::log(s.original_ctx / (beta * pi2)) / (2 * std::log(s.base));
        };
        low = std::fmax(std::floor(pair_of(s.beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(s.beta_slow)), s.rot_dim - 1.0);
    }
    for (int j = 0; j < s.rot_dim / 2; ++j) {
        double f = std::pow(s.base, -2.0 * j / s.rot_dim);
        if (s.scaling == MLA_ROPE_LINEAR) f /= s.factor;
        if (s.scaling == MLA_ROPE_YARN) {
            const double r = std::fmin(std::fmax((j - low) / std::fmax(high - low, 1e-3), 0.0), 1.0);
            f = f * (1 - r) + f / s.factor * r;
        }
        turns[j] = static_cast<unsigned long long>(std::ldexp(f / pi2, 64));   // f <= 1: below 2^62
    }
    return MLA_OK;
}

extern "C" int mla_rope_append(const mla_rope_args* args, void* stream) {
    const int rc = mla::check(args);
    if (rc != MLA_OK) return rc;
    const long long work = static_cast<long long>(args->batch) * args->tokens;
    const unsigned grid = static_cast<unsigned>(work < (1LL << 30) ? work : (1LL << 30));
    mla::mla_rope_kernel<<<grid, mla::kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(*args);
    return mla::launch_status(cudaGetLastError());
}
