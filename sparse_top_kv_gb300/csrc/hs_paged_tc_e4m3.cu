// hs_paged_tc_e4m3.cu -- hs_paged_decode's tensor-core kernel for e4m3 caches.
#include "hs_paged_tc.cuh"

namespace hs_paged {
int launch_tc_e4m3(PagedArgs& a, int d, int group, hs_stream_t stream) {
    // Parts that hold the bits of a query's elements, 8 of bf16, 11 of fp16 (all of
    // them down to about 2^-14 of the row's largest).
    return a.q_is_half ? tc::launch_kind<tc::kE4m3, 3>(a, d, group, stream)
                       : tc::launch_kind<tc::kE4m3, 2>(a, d, group, stream);
}
}  // namespace hs_paged
