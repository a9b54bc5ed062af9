// hs_prefill_bf16.cu -- hs_paged_prefill's attention kernel for bf16 caches.
#include "hs_prefill_tc.cuh"

namespace hs_prefill {
int launch_bf16(const PrefillArgs& a, int d, int bt, hs_stream_t stream) {
    return tc::launch_kind<tc::kBf16>(a, d, bt, stream);
}
}  // namespace hs_prefill
