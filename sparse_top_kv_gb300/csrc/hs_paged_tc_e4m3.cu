// hs_paged_tc_e4m3.cu -- hs_paged_decode's tensor-core kernel for e4m3 caches.
#include "hs_paged_tc.cuh"

namespace hs_paged {
int launch_tc_e4m3(PagedArgs& a, int d, int group, hs_stream_t stream) {
    return tc::launch_kind<tc::kE4m3>(a, d, group, stream);
}
}  // namespace hs_paged
