// hs_prefill_fp16.cu -- hs_paged_prefill's attention kernel for fp16 caches.
#include "hs_prefill_tc.cuh"

namespace hs_prefill {
int launch_fp16(const PrefillArgs& a, int d, int bt, hs_stream_t stream) {
    return tc::launch_kind<tc::kFp16>(a, d, bt, stream);
}
}  // namespace hs_prefill
