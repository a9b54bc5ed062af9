// hs_paged_e4m3.cu -- hs_paged_decode's attention kernel for e4m3 caches.
#include "hs_paged_core.cuh"

namespace hs_paged {
int launch_e4m3(PagedArgs& a, int d, int group, hs_stream_t stream) {
    return core::launch_kind<core::kE4m3>(a, d, group, stream);
}
}  // namespace hs_paged
