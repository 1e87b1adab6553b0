// mla_tree.cu -- attention of a tree of drafted tokens over the latent cache,
// and the weight that each cache row gets from it (include/mla_tree.h).
#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "mla_internal.h"
#include "mla_tree.h"

namespace mla {
namespace {

constexpr int kTreeMagic = 0x4d4c5431;                     // "MLT1"
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

struct TreeParams {
    mla_tree_args a;
    int batch, tokens, heads;
    float scale_log2;
    float* weights;
    float decay;
};

struct Request {
    long long base;
    int d_pos, n_tok;
    int lo, hi;                                            // rows [lo, hi) of the request lie inside the cache
};

__device__ __forceinline__ Request load_request(const TreeParams& p, int b) {
    Request r;
    r.base = p.a.row_offset ? p.a.row_offset[b] : 0;
    r.d_pos = p.a.d_pos[b];
    r.n_tok = p.a.n_tokens ? min(max(p.a.n_tokens[b], 0), p.tokens) : p.tokens;
    const long long rows = r.d_pos < 0 ? 0 : static_cast<long long>(r.d_pos) + r.n_tok;
    const long long lo = r.base < 0 ? -r.base : 0, hi = p.a.kv_rows - r.base;
    r.hi = static_cast<int>(hi < rows ? (hi < 0 ? 0 : hi) : rows);
    r.lo = static_cast<int>(lo < r.hi ? lo : r.hi);
    return r;
}
__device__ __forceinline__ unsigned long long token_mask(const TreeParams& p, int b, int i, int n_tok) {
    const unsigned long long m =
        p.a.mask ? p.a.mask[static_cast<long long>(b) * p.tokens + i] : (~0ull >> (63 - i));
    return n_tok < 64 ? m & ((1ull << n_tok) - 1) : m;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// 18 elements of a 576-element row: 2 * lane + 64 i, + 1
__device__ __forceinline__ void load_row(const uint16_t* row, int lane, float (&v)[18]) {
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 2 * lane + 64 * i);
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
}

// One warp per (request, token, head).
__global__ void __launch_bounds__(kThreads) mla_tree_kernel(const TreeParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(p.batch) * p.tokens * p.heads) return;
    const int b = static_cast<int>(w / (p.tokens * p.heads));
    const int i = static_cast<int>(w / p.heads - static_cast<long long>(b) * p.tokens);
    const Request r = load_request(p, b);
    if (i >= r.n_tok) return;
    const unsigned long long mask = token_mask(p, b, i, r.n_tok);
    float q[18], k[18], o[16];
    load_row(static_cast<const uint16_t*>(p.a.q) + w * kDRow, lane, q);
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int t = r.lo; t < r.hi; ++t) {
        if (t >= r.d_pos && !(mask >> (t - r.d_pos) & 1)) continue;
        load_row(static_cast<const uint16_t*>(p.a.kv) + (r.base + t) * p.a.row_stride, lane, k);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 18; ++j) s += q[j] * k[j];
        s = warp_sum(s) * p.scale_log2;
        const float mn = fmaxf(m, s);
        const float al = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);
        l = l * al + pr;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = o[j] * al + pr * k[j];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long at = w * kDLatent + 2 * lane + 64 * j;
        if (p.a.out_fp32)
            *reinterpret_cast<float2*>(static_cast<float*>(p.a.out) + at) = make_float2(o[2 * j] * inv, o[2 * j + 1] * inv);
        else
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.a.out) + at) =
                pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
    }
    if (lane == 0) p.a.lse[w] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// One warp per cache row of a request.
__global__ void __launch_bounds__(kThreads) mla_tree_weights_kernel(const TreeParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const Request r = load_request(p, b);
    const int warps = gridDim.x * (kThreads / 32);
    for (int t = r.lo + blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < r.hi; t += warps) {
        float q[18], k[18];
        load_row(static_cast<const uint16_t*>(p.a.kv) + (r.base + t) * p.a.row_stride, lane, k);
        float sum = 0.f;
        for (int i = 0; i < r.n_tok; ++i) {
            if (t >= r.d_pos && !(token_mask(p, b, i, r.n_tok) >> (t - r.d_pos) & 1)) continue;
            for (int h = 0; h < p.heads; ++h) {
                const long long w = (static_cast<long long>(b) * p.tokens + i) * p.heads + h;
                const float lse = p.a.lse[w];
                if (lse == -INFINITY) continue;
                load_row(static_cast<const uint16_t*>(p.a.q) + w * kDRow, lane, q);
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 18; ++j) s += q[j] * k[j];
                sum += exp2f(warp_sum(s) * p.scale_log2 - lse * kLog2e);
            }
        }
        if (lane == 0) {
            float* dst = p.weights + r.base + t;
            *dst = p.decay == 0.f ? sum : p.decay * *dst + sum;
        }
    }
}

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

int check_shape(const mla_tree_shape* s) {
    if (!s) return MLA_EINVAL;
    if (s->batch < 1 || s->batch > 4096 || s->tokens < 1 || s->tokens > MLA_TREE_MAX_TOKENS) return MLA_EINVAL;
    if (!(s->scale > 0.f) || !std::isfinite(s->scale)) return MLA_EINVAL;
    if (s->num_sms < 0 || (s->pdl != 0 && s->pdl != 1) || (s->stall_test != 0 && s->stall_test != 1))
        return MLA_EINVAL;
    if (s->heads < 1 || s->heads > 128) return MLA_EUNSUPPORTED;
    return MLA_OK;
}

void layout(mla_tree_plan_t* pl) {
    pl->grid = pl->num_sms;
    pl->status_offset = 0;
    pl->part_offset = 256;
    pl->lse_part_offset = 256;
    pl->scratch_bytes = 256;
}

int check_plan(const mla_tree_plan_t* pl) {
    if (!pl || pl->magic != kTreeMagic || check_shape(&pl->shape) != MLA_OK || pl->num_sms < 1) return MLA_EINVAL;
    mla_tree_plan_t want = *pl;
    layout(&want);
    if (pl->grid != want.grid || pl->status_offset != want.status_offset || pl->part_offset != want.part_offset ||
        pl->lse_part_offset != want.lse_part_offset || pl->scratch_bytes != want.scratch_bytes)
        return MLA_EINVAL;
    return MLA_OK;
}

int check_args(const mla_tree_plan_t* pl, const mla_tree_args* a, bool weights) {
    if (!a || !a->q || !a->kv || !a->d_pos || !a->lse || (!weights && !a->out)) return MLA_EINVAL;
    if (a->kv_rows < 1 || a->row_stride < MLA_D_ROW) return MLA_EINVAL;
    if (a->kv_rows > 0x7fffff00LL) return MLA_EUNSUPPORTED;
    if (pl->shape.batch > 1 && !a->row_offset) return MLA_EINVAL;
    if (a->out_fp32 != 0 && a->out_fp32 != 1) return MLA_EINVAL;
    if (a->row_stride % 8 != 0 || off(a->q, 16) || off(a->kv, 16) || (!weights && off(a->out, 16)) ||
        off(a->lse, 4) || off(a->d_pos, 4) || off(a->row_offset, 8) || off(a->mask, 8) || off(a->n_tokens, 4))
        return MLA_EALIGN;
    return MLA_OK;
}

int check_scratch(const mla_tree_plan_t* pl, const void* scratch, size_t bytes) {
    return !scratch || off(scratch, 256) || bytes < pl->scratch_bytes ? MLA_ESCRATCH : MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_tree_plan(const mla_tree_shape* shape, mla_tree_plan_t* plan) {
    if (!plan) return MLA_EINVAL;
    int rc = mla::check_shape(shape);
    if (rc != MLA_OK) return rc;
    mla_tree_plan_t pl{};
    pl.shape = *shape;
    pl.magic = mla::kTreeMagic;
    pl.num_sms = shape->num_sms;
    if (pl.num_sms == 0) {
        int dev = 0;
        rc = mla::current_device(&dev);
        if (rc == MLA_OK) rc = mla::device_sm_count(dev, &pl.num_sms);
        if (rc != MLA_OK) return rc;
    }
    mla::layout(&pl);
    *plan = pl;
    return MLA_OK;
}

int mla_tree_forward(const mla_tree_plan_t* plan, const mla_tree_args* args, void* scratch, size_t scratch_bytes,
                     void* stream) {
    int rc = mla::check_plan(plan);
    if (rc == MLA_OK) rc = mla::check_args(plan, args, false);
    if (rc == MLA_OK) rc = mla::check_scratch(plan, scratch, scratch_bytes);
    if (rc != MLA_OK) return rc;
    mla::TreeParams p{*args, plan->shape.batch, plan->shape.tokens, plan->shape.heads,
                      plan->shape.scale * mla::kLog2e, nullptr, 0.f};
    const long long rows = static_cast<long long>(p.batch) * p.tokens * p.heads;
    const unsigned grid = static_cast<unsigned>((rows + mla::kThreads / 32 - 1) / (mla::kThreads / 32));
    mla::mla_tree_kernel<<<grid, mla::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return mla::launch_status(cudaGetLastError());
}

int mla_tree_weights(const mla_tree_plan_t* plan, const mla_tree_args* args, float* weights, float decay,
                     void* scratch, size_t scratch_bytes, void* stream) {
    int rc = mla::check_plan(plan);
    if (rc == MLA_OK) rc = mla::check_args(plan, args, true);
    if (rc == MLA_OK && (!weights || !(decay >= 0.f) || !(decay <= 1.f))) rc = MLA_EINVAL;
    if (rc == MLA_OK && mla::off(weights, 4)) rc = MLA_EALIGN;
    if (rc == MLA_OK) rc = mla::check_scratch(plan, scratch, scratch_bytes);
    if (rc != MLA_OK) return rc;
    mla::TreeParams p{*args, plan->shape.batch, plan->shape.tokens, plan->shape.heads,
                      plan->shape.scale * mla::kLog2e, weights, decay};
    mla::mla_tree_weights_kernel<<<dim3(plan->num_sms * 4, p.batch), mla::kThreads, 0,
                                   static_cast<cudaStream_t>(stream)>>>(p);
    return mla::launch_status(cudaGetLastError());
}

}  // extern "C"
