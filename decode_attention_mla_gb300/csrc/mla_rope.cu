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
// per row).  Warps work alone: a warp rotates up to 32 heads of one token, eight
// lanes a head, all its loads (16 bytes a lane and four heads) in flight before
// the angles are needed; lane j takes the sine and cosine of pair j, and lanes
// get their pairs' by shuffles.  (A CTA per token with the angles in shared
// memory: 63 us where this form takes 31 us for 8192 ragged tokens of 128 heads.)
#include <cmath>
#include <cstdint>

#include <cuda_fp8.h>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_rope.cuh"
#include "mla_rope.h"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadPasses = 8;                             // of four heads each, per warp

__device__ __forceinline__ uint2 narrow8_e4m3(const float (&f)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(f[i] / scale, __NV_SATFINITE, __NV_E4M3))
                     << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

// A warp's unit: up to 32 heads of one token, or (the token's last unit) its
// cache row.
__global__ void __launch_bounds__(kRopeThreads) mla_rope_kernel(const __grid_constant__ mla_rope_args a,
                                                                int units_per_token) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int w = static_cast<int>(blockIdx.x) * (kRopeThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int n = w / units_per_token, part = w - n * units_per_token;
    const int b = blockIdx.y;
    if (n >= a.tokens || (a.n_tokens && n >= a.n_tokens[b])) return;
    const int half = a.rot_dim >> 1;
    const int u = lane & 7;
    const int pos = a.positions[static_cast<long long>(b) * a.tokens + n];
    const bool is_row = a.kv && part == units_per_token - 1;
    int lo, hi;
    unit_offsets(u, half, a.interleaved, lo, hi);
    // ---- loads: this lane's units of up to eight heads, or of the row
    uint4 v[kHeadPasses];
    long long row = -1;
    const int h0 = kHeadPasses * 4 * part + (lane >> 3);
    if (is_row) {
        const int d = a.d_pos[b];
        const long long r = (a.row_offset ? a.row_offset[b] : 0) + d + n;
        if (d >= 0 && r >= 0 && r < a.kv_rows) row = r;
        if (row < 0) return;                               // uniform over the warp
        const uint4* c = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.c) + b * a.c_batch +
                                                        n * a.c_token);
        v[0] = c[lane];
        v[1] = c[lane + 32];
        if (lane < 8)
            v[2] = load_unit(static_cast<const uint16_t*>(a.k_rope) + b * a.k_rope_batch + n * a.k_rope_token, lo, hi);
    } else {
        const uint16_t* src = static_cast<const uint16_t*>(a.q_rope) + b * a.q_rope_batch + n * a.q_rope_token;
#pragma unroll
        for (int j = 0; j < kHeadPasses; ++j)
            if (h0 + 4 * j < a.heads) {
                const uint16_t* p = src + (h0 + 4 * j) * a.q_rope_head;
                v[j] = a.interleaved ? *reinterpret_cast<const uint4*>(p + lo) : load_unit(p, lo, hi);
            }
    }
    // ---- angles: lane j takes pair j of the token; a unit's four pairs by shuffles
    float s, c, cs[4], sn[4];
    pair_angle(pos, a.turns, half, a.amplitude, lane, s, c);
    unit_angles(u, s, c, cs, sn);
    const bool rotated = 4 * u < half;                     // half is a multiple of 4: a unit whole or not at all
    if (is_row) {
        float f[8];
        if (a.kv_fp8) {
            uint8_t* p = static_cast<uint8_t*>(a.kv) + row * a.row_stride;
            widen8(v[0], f);
            reinterpret_cast<uint2*>(p)[lane] = narrow8_e4m3(f, a.kv_scale);
            widen8(v[1], f);
            reinterpret_cast<uint2*>(p)[lane + 32] = narrow8_e4m3(f, a.kv_scale);
            if (lane < 8) {
                widen8(v[2], f);
                if (rotated) rotate_unit(f, a.interleaved, cs, sn);
                const uint2 o = narrow8_e4m3(f, a.kv_scale);
                *reinterpret_cast<uint32_t*>(p + kDLatent + lo) = o.x;
                *reinterpret_cast<uint32_t*>(p + kDLatent + hi) = o.y;
            }
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.kv) + row * a.row_stride;
            reinterpret_cast<uint4*>(p)[lane] = v[0];
            reinterpret_cast<uint4*>(p)[lane + 32] = v[1];
            if (lane < 8) {
                widen8(v[2], f);
                if (rotated) rotate_unit(f, a.interleaved, cs, sn);
                const uint4 o = narrow8(f);
                *reinterpret_cast<uint2*>(p + kDLatent + lo) = make_uint2(o.x, o.y);
                *reinterpret_cast<uint2*>(p + kDLatent + hi) = make_uint2(o.z, o.w);
            }
        }
        if (lane == 0) {
            if (a.row_positions) a.row_positions[row] = pos;
            if (a.row_weights) a.row_weights[row] = 0.f;
        }
        return;
    }
    uint16_t* dst = static_cast<uint16_t*>(a.q_out) + b * a.q_out_batch + n * a.q_out_token;
#pragma unroll
    for (int j = 0; j < kHeadPasses; ++j)
        if (h0 + 4 * j < a.heads) {
            float f[8];
            widen8(v[j], f);
            if (rotated) rotate_unit(f, a.interleaved, cs, sn);
            const uint4 o = narrow8(f);
            uint16_t* p = dst + (h0 + 4 * j) * a.q_out_head;
            if (a.interleaved) {
                *reinterpret_cast<uint4*>(p + lo) = o;
            } else {
                *reinterpret_cast<uint2*>(p + lo) = make_uint2(o.x, o.y);
                *reinterpret_cast<uint2*>(p + hi) = make_uint2(o.z, o.w);
            }
        }
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool off8(long long stride) { return stride % 8 != 0; }

int check(const mla_rope_args* a) {
    if (!a || a->batch < 1 || a->batch > 65535 || a->tokens < 1 || a->tokens > (1 << 28)) return MLA_EINVAL;
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
    const int units = (args->heads + 4 * mla::kHeadPasses - 1) / (4 * mla::kHeadPasses) + (args->kv ? 1 : 0);
    const long long warps = static_cast<long long>(args->tokens) * units;
    const long long per = mla::kRopeThreads / 32;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + per - 1) / per), args->batch);
    cfg.blockDim = dim3(mla::kRopeThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return mla::launch_status(cudaLaunchKernelEx(&cfg, mla::mla_rope_kernel, *args, units));
}
