// hs_paged_bf16.cu -- hs_paged_decode's attention kernel for bf16 caches.
#include "hs_paged_core.cuh"

namespace hs_paged {
int launch_bf16(PagedArgs& a, int d, int group, hs_stream_t stream) {
    return core::launch_kind<core::kBf16>(a, d, group, stream);
}
}  // namespace hs_paged
