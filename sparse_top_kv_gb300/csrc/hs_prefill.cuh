// hs_prefill.cuh -- hs_paged_prefill: arguments and work plan shared by the
// dispatcher with its merge kernel (hs_prefill.cu) and the attention kernel
// (hs_prefill_tc.cuh, one translation unit per cache type).
#pragma once

#include "hs_paged.cuh"
#include "hs_plan.h"

namespace hs_prefill {

using hs_paged::kLn2;
using hs_paged::kLog2e;
using hs_paged::kMaxHeads;
using hs_paged::kMaxRows;

constexpr int kTile = 128;      // query rows and cached tokens of a tile
constexpr int kMaxCtas = 1024;  // most CTAs of the attention kernel

// A unit whose tokens several CTAs share, written by the CTA of its first part.
struct SharedUnit {
    int32_t cont;   // tiles of this run's first unit where that began in an earlier one
    // The unit whose first part this run has, if it is shared:
    int32_t valid;
    int32_t slot;   // of that part
    int32_t last;   // the last run with a part of it
    int32_t first, tokens, kvh;
    int32_t blind;  // whether the call has queries that attend to nothing (alike in all)
};

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
    int32_t q_is_half;   // E4M3 caches: the query is fp16 (else bf16)
    float scale_log2;    // scale * log2(e)
    void* out;           // [tokens, heads, D]
    int32_t out_wide;    // out is 32-byte aligned
    float* lse;          // [tokens, heads] or nullptr
    int32_t tq;          // new tokens of a query tile: 128 / group
    int32_t tb;          // and of a unit: one or two query tiles
    int32_t ctas;
    // Workspace: two partial states per CTA (of the units that its run begins
    // and ends in) and the shared units.
    float* part_ml;      // [2 * ctas][unit rows][2]
    float* part_o;       // [2 * ctas][D / 8][unit rows][8]
    SharedUnit* shared;  // [ctas]
    int32_t unit_rows;   // 128 or 256
    // Places (tokens' time) that a unit takes besides its tokens: its queries'
    // loads, the first product and the output.
    int32_t extra;
    int32_t* status;
};

// How a call is cut into work.  A unit is one KV head x one block of a
// request's new tokens: one or two query tiles, each 128 rows of (token, query
// head of the KV head).  Units stand one after another (requests, their KV
// heads, their blocks), each over as many places as cached tokens it sees and
// a.extra more, and the places are dealt to the CTAs in equal contiguous runs;
// a unit whose places several CTAs got is cut at tiles of 128 cached tokens
// and merged.  So ragged batches, causal blocks of growing length and one
// long context load every SM alike.  Queries that attend to nothing are in no unit:
// the kernel that merges writes their zeros.

using hs_plan::Request;
__device__ __forceinline__ Request request_of(const PrefillArgs& a, int r) {
    return hs_plan::request(a.cu_new[r], a.cu_new[r + 1], a.seq_lens[r], a.tokens, a.max_len);
}
__device__ __forceinline__ int block_of(const PrefillArgs& a, int t) {
    return a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size;
}
__device__ __forceinline__ int blocks_of(const PrefillArgs& a, int n) {
    return (n + a.tb - 1) / a.tb;
}
// Places of the first b blocks of a request.
__device__ __forceinline__ int64_t places(const PrefillArgs& a, const Request& x, int b) {
    return hs_plan::places_of_blocks(x, a.tb, a.window, a.extra, b);
}
__device__ __forceinline__ int64_t places_of(const PrefillArgs& a, const Request& x) {
    return x.n > 0 ? places(a, x, blocks_of(a, x.n)) * a.kv_heads : 0;
}
// Places of one block.
__device__ __forceinline__ int cost_of(const PrefillArgs& a, const Request& x, int b) {
    return hs_plan::places_of_block(x, a.tb, a.window, a.extra, b);
}
// First place of CTA c's run: per = total / ctas each, and one more for the first
// `rest` of them.
__device__ __forceinline__ int64_t run_begin(int64_t per, int rest, int c) {
    return per * c + min(c, rest);
}
// a / b, both positive.  (64-bit divisions were half the plan's time.)
__device__ __forceinline__ int64_t quotient(int64_t a, int32_t b) {
    return a >> 32 == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
// The tile that place `at` of a unit stands for.
__device__ __forceinline__ int tile_at(int64_t at, int cost, int tiles) {
    return at <= 0 ? 0 : at >= cost ? tiles : int(quotient(at * tiles, cost));
}

// The attention kernel over a cache type; bt: tokens of a TMA box, or 0 where threads
// load.
int launch_bf16(const PrefillArgs& a, int d, int bt, hs_stream_t stream);
int launch_fp16(const PrefillArgs& a, int d, int bt, hs_stream_t stream);
int launch_e4m3(const PrefillArgs& a, int d, int bt, hs_stream_t stream);

}  // namespace hs_prefill
