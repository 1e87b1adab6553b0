// mla_paged_attend.cu -- attention over the 4-bit paged cache (include/mla_paged.h).
//
// A warp per query row: a lane has sixteen features (one block of a row) and two of the
// 64 rotated ones; rows one after the other, a running maximum and sum.
#include "mla_paged.cuh"

namespace mla {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) mla_paged_attend_kernel(const __grid_constant__ PagedParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int per = p.t.tokens * p.t.heads;
    const int b = static_cast<int>(row / per), i = static_cast<int>(row - static_cast<long long>(b) * per) / p.t.heads;
    if (b >= p.t.batch) return;
    if (p.t.a.n_tokens && i >= p.t.a.n_tokens[b]) return;
    float q[16], o[16];
    const uint16_t* src = p.q + row * kDRow;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        q[k] = __uint_as_float(static_cast<uint32_t>(src[16 * lane + k]) << 16);
        o[k] = 0.f;
    }
    const float q0 = __uint_as_float(static_cast<uint32_t>(src[kDLatent + 2 * lane]) << 16);
    const float q1 = __uint_as_float(static_cast<uint32_t>(src[kDLatent + 2 * lane + 1]) << 16);
    float m = -INFINITY, l = 0.f;
    const int d = p.t.a.d_pos[b];
    const long long last = d < 0 ? -1 : static_cast<long long>(d) + i;
    const long long recent = p.window > 0 ? last - p.window + 1 : 0;
    const long long end = min(last + 1, static_cast<long long>(paged_rows(p.cache)));
    for (long long t = 0; t < end; ++t) {
        if (t >= p.sink && t < recent) {
            t = recent - 1;
            continue;
        }
        const int page = page_of(p.cache, b, static_cast<int>(t));
        if (page < 0) continue;
        const uint8_t* kv = row_in(p.cache, page, static_cast<int>(t));
        const uint2 w = reinterpret_cast<const uint2*>(kv)[lane];
        const uint8_t scale = kv[kQ4Scales + lane];
        const uint32_t key = reinterpret_cast<const uint32_t*>(kv + kQ4Rope)[lane];
        const uint32_t s2 = widen_e4m3(static_cast<uint16_t>(scale | scale << 8));
        uint32_t h[8];
        widen_e2m1(w.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
        widen_e2m1(w.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
        float c[16], s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 v = f16x2_to_float2(mul_f16x2(h[k], s2));
            c[2 * k] = v.x * p.kv_scale;
            c[2 * k + 1] = v.y * p.kv_scale;
            s = fmaf(q[2 * k], c[2 * k], fmaf(q[2 * k + 1], c[2 * k + 1], s));
        }
        s = fmaf(q0, __uint_as_float(key << 16), fmaf(q1, __uint_as_float(key & 0xffff0000u), s));
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.t.scale_log2;
        const float top = fmaxf(m, s);
        if (s == -INFINITY) continue;
        const float a = exp2f(m - top), e = exp2f(s - top);
        m = top;
        l = l * a + e;
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = fmaf(e, c[k], o[k] * a);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane == 0) p.t.a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] *= inv;
    if (p.t.a.out_fp32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.t.a.out) + row * kDLatent) + 4 * lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.t.a.out) + row * kDLatent) + 2 * lane;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            dst[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
    }
}

}  // namespace

cudaError_t paged_attend_prepare() { return cudaSuccess; }

cudaError_t launch_paged_attend(const PagedParams& p, bool pdl, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const long long rows = static_cast<long long>(p.t.batch) * p.t.tokens * p.t.heads;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mla_paged_attend_kernel, p);
}

}  // namespace mla
