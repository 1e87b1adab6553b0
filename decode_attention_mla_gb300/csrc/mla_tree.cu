// mla_tree.cu -- attention of a tree of drafted tokens over the latent cache,
// and the weight that each cache row gets from it (include/mla_tree.h).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "mla_tree.cuh"

namespace mla {
namespace {

constexpr int kTreeMagic = 0x4d4c5431;                     // "MLT1"

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The caller's scale in base-2 units, as the kernels take it.
float scale_log2(float scale) { return static_cast<float>(scale * 1.4426950408889634); }

int check_shape(const mla_tree_shape* s) {
    if (!s) return MLA_EINVAL;
    if (s->batch < 1 || s->batch > 4096 || s->tokens < 1 || s->tokens > MLA_TREE_MAX_TOKENS) return MLA_EINVAL;
    if (!(s->scale > 0.f) || !std::isfinite(scale_log2(s->scale))) return MLA_EINVAL;
    if (s->num_sms < 0 || (s->pdl != 0 && s->pdl != 1) || (s->stall_test != 0 && s->stall_test != 1))
        return MLA_EINVAL;
    if (s->heads < 1 || s->heads > 128) return MLA_EUNSUPPORTED;
    return MLA_OK;
}

// Scratch: status word, the pairs' merge notes, their pieces and the pieces'
// log-sum-exps, each region 256-byte aligned.
constexpr size_t kMergeOffset = 256;
// Pairs of SMs to use.
int tree_pairs(int num_sms) { return num_sms < 2 ? 1 : num_sms / 2; }
void layout(mla_tree_plan_t* pl) {
    const size_t pairs = static_cast<size_t>(tree_pairs(pl->num_sms));
    pl->grid = static_cast<int>(2 * pairs);
    pl->status_offset = 0;
    pl->part_offset = up256(kMergeOffset + pairs * kTreePieces * (sizeof(TreeMerge) + sizeof(TreeCut)));
    pl->lse_part_offset = pl->part_offset + pairs * kTreePieces * kTreeBlockRows * kDLatent * sizeof(float);
    pl->scratch_bytes = up256(pl->lse_part_offset + pairs * kTreePieces * kTreeBlockRows * sizeof(float));
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

std::atomic<int> g_tree_prepared[kMaxDevices];
std::mutex g_tree_mutex;

// Kernel attributes, once per device, outside any capture.
int prepare(cudaStream_t st, bool may_capture) {
    int dev = 0;
    const int rc = current_device(&dev);
    if (rc != MLA_OK) return rc;
    if (g_tree_prepared[dev].load(std::memory_order_acquire)) return MLA_OK;
    if (may_capture) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
            cudaGetLastError();
            return MLA_ECUDA;
        }
        if (cs != cudaStreamCaptureStatusNone) return MLA_ENOTREADY;
    }
    std::lock_guard<std::mutex> lock(g_tree_mutex);
    if (launch_status(tree_attend_prepare()) != MLA_OK || launch_status(tree_weights_prepare()) != MLA_OK)
        return MLA_ECUDA;
    g_tree_prepared[dev].store(1, std::memory_order_release);
    return MLA_OK;
}

// Height of the boxes that a row block's last query rows come in (64: none needed).
int q_tail(const mla_tree_plan_t* pl) {
    const int rest = (pl->shape.tokens * pl->shape.heads + 7) / 8 * 8 % 64;
    return rest ? rest : 64;
}

TreeParams params(const mla_tree_plan_t* pl, const mla_tree_args* a, void* scratch) {
    char* base = static_cast<char*>(scratch);
    TreeParams p{};
    p.a = *a;
    p.batch = pl->shape.batch;
    p.tokens = pl->shape.tokens;
    p.heads = pl->shape.heads;
    p.q_tail = q_tail(pl);
    p.clusters = pl->grid / 2;
    p.block_rows = kTreeBlockRows;
    p.scale_log2 = scale_log2(pl->shape.scale);
    p.merge = reinterpret_cast<TreeMerge*>(base + kMergeOffset);
    p.cut = reinterpret_cast<TreeCut*>(p.merge + kTreePieces * p.clusters);
    p.part = reinterpret_cast<float*>(base + pl->part_offset);
    p.lse_part = reinterpret_cast<float*>(base + pl->lse_part_offset);
    p.status = reinterpret_cast<int*>(base + pl->status_offset);
    p.stall_test = pl->shape.stall_test;
    return p;
}

int encode_q(const mla_tree_plan_t* pl, const mla_tree_args* a, TreeMaps* maps, uint32_t chunks) {
    const long long rows = static_cast<long long>(pl->shape.batch) * pl->shape.tokens * pl->shape.heads;
    const int rc = encode_bf16_row_chunks(&maps->q, a->q, rows, MLA_D_ROW, 64, chunks);
    if (rc != MLA_OK || q_tail(pl) == 64) return rc;
    return encode_bf16_row_chunks(&maps->q_tail, a->q, rows, MLA_D_ROW, q_tail(pl), 1);
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
        if (rc == MLA_OK) rc = mla::prepare(nullptr, false);
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = mla::prepare(st, true);
    if (rc != MLA_OK) return rc;
    mla::TreeMaps maps{};
    rc = mla::encode_bf16_row_chunks(&maps.kv, args->kv, args->kv_rows, args->row_stride, 64, 2);
    if (rc == MLA_OK) rc = mla::encode_bf16_row_chunks(&maps.rope, args->kv, args->kv_rows, args->row_stride, 64, 1);
    if (rc == MLA_OK) rc = mla::encode_q(plan, args, &maps, MLA_D_ROW / 64);
    if (rc != MLA_OK) return rc;
    return mla::launch_status(
        mla::launch_tree_attend(maps, mla::params(plan, args, scratch), plan->shape.pdl != 0, st));
}

int mla_tree_weights(const mla_tree_plan_t* plan, const mla_tree_args* args, float* weights, float decay,
                     void* scratch, size_t scratch_bytes, void* stream) {
    int rc = mla::check_plan(plan);
    if (rc == MLA_OK) rc = mla::check_args(plan, args, true);
    if (rc == MLA_OK && (!weights || !(decay >= 0.f) || !(decay <= 1.f))) rc = MLA_EINVAL;
    if (rc == MLA_OK && mla::off(weights, 4)) rc = MLA_EALIGN;
    if (rc == MLA_OK) rc = mla::check_scratch(plan, scratch, scratch_bytes);
    if (rc != MLA_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = mla::prepare(st, true);
    if (rc != MLA_OK) return rc;
    mla::TreeMaps maps{};
    rc = mla::encode_bf16_row_chunks(&maps.k, args->kv, args->kv_rows, args->row_stride, 128, 1);
    if (rc == MLA_OK) rc = mla::encode_q(plan, args, &maps, 1);
    if (rc != MLA_OK) return rc;
    mla::TreeParams p = mla::params(plan, args, scratch);
    p.weights = weights;
    p.decay = decay;
    return mla::launch_status(mla::launch_tree_weights(maps, p, plan->shape.pdl != 0, st));
}

}  // extern "C"
