// mla_paged.cu -- attention over the 4-bit paged cache: plan, checks and launch
// (include/mla_paged.h).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "mla_paged.cuh"

namespace mla {
namespace {

constexpr int kPagedMagic = 0x4d4c5034;                    // "MLP4"

bool off(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

int check_shape(const mla_paged_shape* s) {
    if (!s) return MLA_EINVAL;
    if (s->batch < 1 || s->batch > 4096 || s->tokens < 1 || s->tokens > MLA_PAGED_MAX_TOKENS) return MLA_EINVAL;
    if (!(s->scale > 0.f) || !(s->scale < 0x1p60f)) return MLA_EINVAL;
    if (s->num_sms < 0 || (s->pdl != 0 && s->pdl != 1) || (s->stall_test != 0 && s->stall_test != 1))
        return MLA_EINVAL;
    if (s->heads < 1 || s->heads > 128) return MLA_EUNSUPPORTED;
    return MLA_OK;
}

// Scratch as of a tree plan: status word, the runs' merge notes, their pieces and the pieces'
// log-sum-exps, each region 256-byte aligned.  A run is a pair's (pieces of 128 query rows) or, with few
// query rows, an SM's (pieces of 16, in the place of 32): twice as many notes, fewer bytes.
constexpr size_t kMergeOffset = 256;
int pairs_of(int num_sms) { return num_sms < 2 ? 1 : num_sms / 2; }
void layout(mla_paged_plan_t* pl) {
    const size_t pairs = static_cast<size_t>(pairs_of(pl->num_sms));
    pl->grid = static_cast<int>(2 * pairs);
    pl->status_offset = 0;
    pl->part_offset = up256(kMergeOffset + 2 * pairs * kTreePieces * (sizeof(TreeMerge) + sizeof(TreeCut)));
    pl->lse_part_offset = pl->part_offset + pairs * kTreePieces * kTreeBlockRows * kDLatent * sizeof(float);
    pl->scratch_bytes = up256(pl->lse_part_offset + pairs * kTreePieces * kTreeBlockRows * sizeof(float));
}

int check_plan(const mla_paged_plan_t* pl) {
    if (!pl || pl->magic != kPagedMagic || check_shape(&pl->shape) != MLA_OK || pl->num_sms < 1) return MLA_EINVAL;
    mla_paged_plan_t want = *pl;
    layout(&want);
    if (pl->grid != want.grid || pl->status_offset != want.status_offset || pl->part_offset != want.part_offset ||
        pl->lse_part_offset != want.lse_part_offset || pl->scratch_bytes != want.scratch_bytes)
        return MLA_EINVAL;
    return MLA_OK;
}

int check_args(const mla_paged_args* a) {
    if (!a || !a->q || !a->d_pos || !a->lse || !a->out) return MLA_EINVAL;
    if (a->window < 0 || a->sink < 0 || (a->out_fp32 != 0 && a->out_fp32 != 1)) return MLA_EINVAL;
    const int rc = check_cache(&a->cache);
    if (rc != MLA_OK) return rc;
    return off(a->q, 16) || off(a->out, 16) || off(a->lse, 4) || off(a->d_pos, 4) || off(a->n_tokens, 4) ? MLA_EALIGN
                                                                                                         : MLA_OK;
}

std::atomic<int> g_paged_prepared[kMaxDevices];
std::mutex g_paged_mutex;

// Kernel attributes, once per device, outside any capture.
int prepare(cudaStream_t st, bool may_capture) {
    int dev = 0;
    const int rc = current_device(&dev);
    if (rc != MLA_OK) return rc;
    if (g_paged_prepared[dev].load(std::memory_order_acquire)) return MLA_OK;
    if (may_capture) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(st, &cs) != cudaSuccess) {
            cudaGetLastError();
            return MLA_ECUDA;
        }
        if (cs != cudaStreamCaptureStatusNone) return MLA_ENOTREADY;
    }
    std::lock_guard<std::mutex> lock(g_paged_mutex);
    if (launch_status(paged_attend_prepare()) != MLA_OK || launch_status(paged_decode_prepare()) != MLA_OK)
        return MLA_ECUDA;
    g_paged_prepared[dev].store(1, std::memory_order_release);
    return MLA_OK;
}

// Few query rows, or little work: on warp-level MMAs, sixteen query rows at a time and an SM's run each; the tcgen05 kernel does
// 128 in the time of 16, but takes about 5 us longer to begin and end.
// Rows.  Measured, us (requests x cache rows): with 16 query rows per request 10.1 and 13.4 (1 x 255), 19.3 and 29.4 (8 x 4096), 144
// and 250 (32 x 32768); with 32 10.2 and 13.5, 23.1 and 30.0, 271 and 251; with 48 27.4 and 33.3 (8 x 4096), 400 and 253.
// Work, in units of 64 cache rows per SM, a block of sixteen query rows counting as two more (requests x query rows x cache
// rows): 1 x 128 x 255 0.3 units, 10.2 and 15.4 us; 1 x 128 x 2000 1.8, 14.3 and 16.7; 8 x 128 x 255 2.5, 12.6 and 17.5; 2 x 64 x
// 3000 2.6, 18.0 and 18.5; 7 x 64 x 1000 3.3, 17.3 and 19.8; but 1 x 128 x 4000 3.4, 19.2 and 17.4; 1 x 128 x 10000 8.4, 25.5 and 22.0.
// (How long the requests are, the host does not know: it takes the table's length, or what a window leaves of it.  So the rule
// by work is one for tables about as long as their requests, and with 17 .. 32 query rows and long caches the choice is the
// slower one by the 8 % above: a table for 32768 rows says nothing of whether 4096 or 32768 are in it.  The kernel counts
// units in an int.)
constexpr int kFewRows = 32, kFewUnits = 3;
bool few_rows(const mla_paged_plan_t* pl, const mla_paged_args* a) {
    const long long rows = static_cast<long long>(pl->shape.tokens) * pl->shape.heads;
    const long long blocks = pl->shape.batch * ((rows + kDecodeBlockRows - 1) / kDecodeBlockRows);
    const long long table = static_cast<long long>(a->cache.columns) * a->cache.page_rows;
    if (blocks * (table / 64 + 2) >= (1ll << 30)) return false;
    const long long seen = a->window > 0 ? static_cast<long long>(a->window) + a->sink + pl->shape.tokens : table;
    return rows <= kFewRows || blocks * (std::min(table, seen) / 64 + 3) <= static_cast<long long>(kFewUnits) * pl->num_sms;
}

PagedParams params(const mla_paged_plan_t* pl, const mla_paged_args* a, void* scratch, bool few) {
    char* base = static_cast<char*>(scratch);
    PagedParams p{};
    p.a.d_pos = a->d_pos;
    p.a.n_tokens = a->n_tokens;
    p.a.out = a->out;
    p.a.out_fp32 = a->out_fp32;
    p.a.lse = a->lse;
    p.batch = pl->shape.batch;
    p.tokens = pl->shape.tokens;
    p.heads = pl->shape.heads;
    p.clusters = few ? pl->grid : pl->grid / 2;
    p.block_rows = few ? kDecodeBlockRows : kTreeBlockRows;
    p.merge = reinterpret_cast<TreeMerge*>(base + kMergeOffset);
    p.cut = reinterpret_cast<TreeCut*>(p.merge + kTreePieces * p.clusters);
    p.part = reinterpret_cast<float*>(base + pl->part_offset);
    p.lse_part = reinterpret_cast<float*>(base + pl->lse_part_offset);
    p.status = reinterpret_cast<int*>(base + pl->status_offset);
    p.stall_test = pl->shape.stall_test;
    p.cache = paged_cache(&a->cache);
    p.q = static_cast<const uint16_t*>(a->q);
    p.kv_scale = a->cache.kv_scale;
    int carry = 0;                                         // (a mantissa next to 1 is rounded up to it)
    p.unit = 2 * std::frexp(static_cast<float>(std::frexp(pl->shape.scale * 1.4426950408889634 * p.kv_scale, &p.unit_exp)), &carry);
    p.unit_exp += carry - 1;
    p.least_exp = std::max(-126, -126 - p.unit_exp);
    p.window = a->window;
    p.sink = a->sink;
    return p;
}

}  // namespace
}  // namespace mla

extern "C" {

int mla_paged_plan(const mla_paged_shape* shape, mla_paged_plan_t* plan) {
    if (!plan) return MLA_EINVAL;
    int rc = mla::check_shape(shape);
    if (rc != MLA_OK) return rc;
    mla_paged_plan_t pl{};
    pl.shape = *shape;
    pl.magic = mla::kPagedMagic;
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

int mla_paged_forward(const mla_paged_plan_t* plan, const mla_paged_args* args, void* scratch, size_t scratch_bytes,
                      void* stream) {
    int rc = mla::check_plan(plan);
    if (rc == MLA_OK) rc = mla::check_args(args);
    if (rc == MLA_OK && (!scratch || mla::off(scratch, 256) || scratch_bytes < plan->scratch_bytes)) rc = MLA_ESCRATCH;
    if (rc != MLA_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = mla::prepare(st, true);
    if (rc != MLA_OK) return rc;
    const bool few = mla::few_rows(plan, args);
    const mla::PagedParams p = mla::params(plan, args, scratch, few);
    if (few) return mla::launch_status(mla::launch_paged_decode(p, plan->shape.pdl != 0, st));
    mla::PagedMaps maps;
    rc = mla::encode_q4_boxes(&maps.codes, &args->cache, 64, CU_TENSOR_MAP_SWIZZLE_64B);
    if (rc == MLA_OK) rc = mla::encode_q4_boxes(&maps.scales, &args->cache, 16, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc == MLA_OK) rc = mla::encode_q4_boxes(&maps.rope, &args->cache, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != MLA_OK) return rc;
    return mla::launch_status(
        mla::launch_paged_attend(maps, p, plan->shape.pdl != 0, st));
}

}  // extern "C"
