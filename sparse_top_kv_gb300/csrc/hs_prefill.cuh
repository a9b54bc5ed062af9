// hs_prefill.cuh -- hs_paged_prefill: arguments shared by the dispatcher
// (hs_prefill.cu) and the attention kernel.
#pragma once

#include "hs_paged.cuh"

namespace hs_prefill {

using hs_paged::kLn2;
using hs_paged::kLog2e;
using hs_paged::kMaxHeads;
using hs_paged::kMaxRows;

struct PrefillArgs {
    const void* q;  // [tokens, heads, D], tokens q_stride elements apart
    const void* k;
    const void* v;
    int64_t q_stride, page_stride, row_stride, head_stride;  // elements
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* cu_new;
    const int32_t* seq_lens;
    const float* k_scale;  // [kv_heads] or nullptr (E4M3)
    const float* v_scale;
    int32_t tokens, rows, heads, kv_heads, group, num_pages, page_size, max_len, window, sinks;
    int32_t page_shift;  // log2 of page_size, or -1
    float scale_log2;    // scale * log2(e)
    void* out;           // [tokens, heads, D]
    float* lse;          // [tokens, heads] or nullptr
    int32_t* status;
};

// Where request r's new tokens stand, and its cached tokens.
struct Request {
    int first, n, T;
};
__device__ __forceinline__ Request request_of(const PrefillArgs& a, int r) {
    Request x;
    x.first = min(max(a.cu_new[r], 0), a.tokens);
    x.n = max(0, min(a.cu_new[r + 1], a.tokens) - x.first);
    x.T = min(max(a.seq_lens[r], 0), a.max_len);
    return x;
}
__device__ __forceinline__ int block_of(const PrefillArgs& a, int t) {
    return a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size;
}

}  // namespace hs_prefill
