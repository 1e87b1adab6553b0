// mla_paged.cuh -- what the host side and the kernel of the attention over the
// 4-bit paged cache share.
#pragma once

#include "mla_q4.cuh"
#include "mla_tree.cuh"

namespace mla {

struct PagedParams {
    TreeParams t;                                          // outputs, sizes, pieces and their notes
    PagedCache cache;
    const uint16_t* q;
    float kv_scale;
    int window, sink;
};

cudaError_t paged_attend_prepare();
cudaError_t launch_paged_attend(const PagedParams& p, bool pdl, cudaStream_t stream);

}  // namespace mla
