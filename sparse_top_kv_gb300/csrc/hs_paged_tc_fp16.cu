// hs_paged_tc_fp16.cu -- hs_paged_decode's tensor-core kernel for fp16 caches.
#include "hs_paged_tc.cuh"

namespace hs_paged {
int launch_tc_fp16(PagedArgs& a, int d, int group, hs_stream_t stream) {
    return tc::launch_kind<tc::kFp16, 1>(a, d, group, stream);
}
}  // namespace hs_paged
