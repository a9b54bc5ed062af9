// hs_prefill_e4m3.cu -- hs_paged_prefill's attention kernel for E4M3 caches.
#include "hs_prefill_tc.cuh"

namespace hs_prefill {
int launch_e4m3(const PrefillArgs& a, int d, int bt, hs_stream_t stream) {
    return tc::launch_kind<tc::kE4m3>(a, d, bt, stream);
}
}  // namespace hs_prefill
