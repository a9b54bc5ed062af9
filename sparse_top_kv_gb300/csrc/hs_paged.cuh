// hs_paged.cuh -- attention of one new token per request over every cached
// token of a paged KV cache: arguments, work plan and helpers shared by the
// attention kernels (hs_paged_core.cuh, one translation unit per cache type)
// and the dispatcher with its finishing kernels (hs_paged.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "hs_common.cuh"

namespace hs_paged {

constexpr int kKey = 16;           // cached tokens per warp step
constexpr int kMaxRows = 4096;     // requests of one call (their plan sits in shared memory)
constexpr int kMaxCtas = 1024;     // most CTAs of the attention kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PagedArgs {
    const void* q;  // [rows, heads, D], rows q_stride elements apart
    const void* k;
    const void* v;
    int64_t q_stride, page_stride, row_stride, head_stride;  // elements
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* seq_lens;
    const float* k_scale;  // [kv_heads] or nullptr (E4M3)
    const float* v_scale;
    int32_t rows, heads, kv_heads, num_pages, page_size, max_len, window, sinks;
    int32_t q_is_half;  // E4M3 caches: the query is fp16 (else bf16)
    float scale_log2;   // scale * log2(e)
    void* out;          // [rows, heads, D]
    float* lse;         // [rows, heads] or nullptr
    float* score;       // [rows, score_stride] or nullptr
    int64_t score_stride;
    float decay;
    // Workspace.
    int32_t* plan;      // [8] header, then prefix [rows + 1]
    float* lse2;        // [rows, heads] log2 units (scored calls)
    float* part_ml;     // [2 * ctas][unit heads][2]
    float* part_o;      // [2 * ctas][unit heads][D]
    float* logits;      // [rows, heads, logit_stride] log2 units (scored calls)
    int64_t logit_stride;
    int32_t unit_heads_max;
    int32_t ctas;
    int32_t* status;
};

// Tokens a request attends to: its last `window` (all without a window) and
// the first `sinks` before them.  Index i of them is token
// i < sc ? i : i - sc + w0.
struct Visible {
    int n, sc, w0;
};
__device__ __forceinline__ Visible visible_of(int len, int max_len, int window, int sinks) {
    const int T = min(max(len, 0), max_len);
    Visible v;
    const int wc = window > 0 ? min(T, window) : T;
    v.w0 = T - wc;
    v.sc = window > 0 ? min(sinks, v.w0) : 0;
    v.n = wc + v.sc;
    return v;
}

// The plan, the same in every CTA.  A unit is one request x one chunk of its
// heads (hs KV heads x up to GM query heads of each); its tokens are cut into
// tiles of ts = warps / hs steps of 16.  The units' tiles, one after another,
// are dealt to n CTAs in equal contiguous runs, so ragged batches load every
// SM alike and one long context uses all of them.
struct Plan {
    int hs, n, chunks;
    int64_t tiles;
};
__device__ __forceinline__ int64_t run_begin(const Plan& p, int c) {
    return p.tiles * c / p.n;
}
__device__ __forceinline__ int run_of(const Plan& p, int64_t tile) {
    int c = int(tile * p.n / p.tiles);
    while (c > 0 && run_begin(p, c) > tile) --c;
    while (c + 1 < p.n && run_begin(p, c + 1) <= tile) ++c;
    return c;
}

int launch_bf16(const PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_fp16(const PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_e4m3(const PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_bf16(const PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_fp16(const PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_e4m3(const PagedArgs& a, int d, int group, hs_stream_t stream);

}  // namespace hs_paged
