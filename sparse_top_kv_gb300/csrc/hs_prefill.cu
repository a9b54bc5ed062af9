// hs_prefill.cu -- hs_paged_prefill: argument checks, workspace layout and the
// merge of units that several CTAs shared.  The attention kernel itself is in
// hs_prefill_tc.cuh.
#include <cuda.h>

#include <type_traits>

#include "hs_prefill.cuh"

namespace hs_paged {
namespace tc {
using Encode = decltype(&cuTensorMapEncodeTiled);
Encode encoder();
}  // namespace tc
}  // namespace hs_paged

namespace hs_prefill {

namespace tc {
int encode(CUtensorMap* m, int dtype, int dims, const void* base, const cuuint64_t* size,
           const cuuint64_t* stride, const cuuint32_t* box) {
    const hs_paged::tc::Encode f = hs_paged::tc::encoder();
    if (f == nullptr) return HS_ERR_CUDA;
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    const CUtensorMapDataType type = dtype == HS_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : dtype == HS_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUresult r =
        f(m, type, cuuint32_t(dims), const_cast<void*>(base), size, stride, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE,
          // E4M3 rows are converted by threads, in their own order.
          dtype == HS_E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? HS_OK : HS_ERR_CUDA;
}
int encode_map(CUtensorMap* m, const void* base, const PrefillArgs& a, int kv_dtype, int d,
               int bt) {
    const cuuint64_t elt = kv_dtype == HS_E4M3 ? 1 : 2;
    // A dimension of one entry may have any stride; the encoder wants a valid one.
    const auto bytes = [&](int64_t stride, int64_t n) {
        return n > 1 ? cuuint64_t(stride) * elt : cuuint64_t(d) * elt;
    };
    const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(a.page_size), cuuint64_t(a.kv_heads),
                                cuuint64_t(a.num_pages)};
    const cuuint64_t strides[3] = {bytes(a.row_stride, a.page_size),
                                   bytes(a.head_stride, a.kv_heads),
                                   bytes(a.page_stride, a.num_pages)};
    // E4M3: the dims of a ring unit; else one swizzled block's.
    const int wide = kv_dtype != HS_E4M3 || d == 64 ? 64 : 128;
    const cuuint32_t box[4] = {cuuint32_t(wide), cuuint32_t(bt), 1u, 1u};
    return encode(m, kv_dtype, 4, base, dims, strides, box);
}
int encode_q_map(CUtensorMap* m, const PrefillArgs& a, int dtype, int d) {
    const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(a.heads), cuuint64_t(a.tokens)};
    const cuuint64_t strides[2] = {
        cuuint64_t(d) * 2,
        a.tokens > 1 ? cuuint64_t(a.q_stride) * 2 : cuuint64_t(a.heads) * d * 2};
    const cuuint32_t box[3] = {64u, cuuint32_t(a.group), cuuint32_t(a.tq)};
    return encode(m, dtype, 3, a.q, dims, strides, box);
}
}  // namespace tc

namespace {

// Tokens of a TMA box, or 0 where threads have to load: pages without runs of
// 8 tokens (a swizzle's rows), broadcast strides.
int box_tokens(const PrefillArgs& a, int kv_dtype) {
    const int64_t most = int64_t(1) << 38;  // elements; the encoder takes strides below 2^40 bytes
    if (a.page_size % 8 != 0 || a.num_pages <= 0 ||
        (a.kv_heads > 1 && (a.head_stride <= 0 || a.head_stride >= most)) ||
        (a.num_pages > 1 && (a.page_stride <= 0 || a.page_stride >= most)) || a.row_stride <= 0 ||
        a.row_stride >= most || (a.tokens > 1 && (a.q_stride <= 0 || a.q_stride >= most)))
        return 0;
    int bt = kTile;
    while (a.page_size % bt) bt /= 2;
    return bt;
}

// Whether units are of one query tile, whose softmax two warpgroups share, rather
// than of two with one each (a head size of 256 has no other): E4M3 caches, whose
// conversion leaves little time for anything else, where two tiles would mostly be
// one.  Groups of 4, 64 requests over up to 4096 tokens: 4 new tokens each 180 ->
// 154 us, up to 32 191 -> 168; 64, two tiles, 306 -> 425.  (16-bit caches: 3 % either
// way.)  By half, so that a long prompt among single tokens has two.
bool one_tile(const PrefillArgs& a, int kv_dtype, int bt) {
    return kv_dtype == HS_E4M3 && bt > 0 && int64_t(a.tokens) * 2 <= int64_t(a.rows) * a.tq;
}

constexpr int kMergeThreads = 128;
constexpr int kMergeDims = 16;  // dims of a block

// Queries that attend to nothing: 0 and -inf, by the whole grid.  (As units of the
// attention kernel, planned as if they saw each other: 64 single tokens over 4 K beside
// a prompt of 8192 tokens that was refused 566 us, now 218, without the prompt
// 198; the same inputs again and again.)
template <int D>
__device__ __noinline__ void write_zeros(const PrefillArgs& a) {
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * gridDim.y * kMergeThreads;
    const int64_t me = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kMergeThreads + threadIdx.x;
    for (int r0 = 0; r0 < a.rows; r0 += 32) {
        Request x{};
        if (r0 + lane < a.rows) x = request_of(a, r0 + lane);
        for (uint32_t some = __ballot_sync(0xffffffffu, x.blind > 0); some != 0; some &= some - 1) {
            const int from = __ffs(some) - 1;
            // A token's heads are packed: one run of rows.
            const int64_t row = int64_t(__shfl_sync(0xffffffffu, x.first - x.blind, from)) * a.heads;
            const int64_t n = int64_t(__shfl_sync(0xffffffffu, x.blind, from)) * a.heads;
            uint4* out = static_cast<uint4*>(a.out) + row * (D / 8);
            for (int64_t i = me; i < n * (D / 8); i += step) out[i] = make_uint4(0u, 0u, 0u, 0u);
            if (a.lse != nullptr)
                for (int64_t i = me; i < n; i += step) a.lse[row + i] = -CUDART_INF_F;
        }
    }
}

// Joins the parts of a shared unit: out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p -
// M) l_p.  Block (c, y): 16 dims of 128 rows of the unit whose first part CTA c
// had; a thread per row, as the partial states lie.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ PrefillArgs a,
                                                              int out_bf16) {
    constexpr int kParts = D / kMergeDims;
    __shared__ int slots[kMaxCtas];
    __shared__ int count;
    hs::pdl_wait();
    hs::pdl_trigger();
    const int c = blockIdx.x;
    const SharedUnit u = a.shared[c];
    if (u.blind) write_zeros<D>(a);
    if (!u.valid) return;
    // The slots of the unit's parts, in order; CTAs without a tile have none.
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int n = 1;
        for (int c0 = c + 1; c0 <= u.last; c0 += 32) {
            const int p = c0 + lane;
            const bool has = p <= u.last && a.shared[p].cont > 0;
            const uint32_t all = __ballot_sync(0xffffffffu, has);
            if (has) slots[n + __popc(all & ((1u << lane) - 1u))] = 2 * p;
            n += __popc(all);
        }
        if (lane == 0) {
            slots[0] = u.slot;
            count = n;
        }
    }
    __syncthreads();
    const int n = count, w = blockIdx.y / kParts, part = blockIdx.y % kParts, r = threadIdx.x;
    const int tok = r / a.group, hd = r - tok * a.group;
    if (tok >= a.tq || w * a.tq + tok >= u.tokens) return;
    const int j = w * kTile + r;
    float M = -CUDART_INF_F, L = 0.f;
    float o[kMergeDims];
#pragma unroll
    for (int i = 0; i < kMergeDims; ++i) o[i] = 0.f;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + j;
    const float4* po = reinterpret_cast<const float4*>(a.part_o) +
                       (int64_t(part * (kMergeDims / 8)) * a.unit_rows + j) * 2;
    constexpr int kAhead = 4;  // parts in flight
    for (int p0 = 0; p0 < n; p0 += kAhead) {
        float2 s[kAhead];
        float4 x[kAhead][kMergeDims / 4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            s[k] = make_float2(-CUDART_INF_F, 0.f);
            if (p0 + k >= n) continue;
            const int64_t slot = slots[p0 + k];
            s[k] = __ldcg(ml + slot * a.unit_rows);
#pragma unroll
            for (int i = 0; i < kMergeDims / 4; ++i)
                x[k][i] = __ldcg(po + (slot * (D / 8) + i / 2) * a.unit_rows * 2 + i % 2);
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) m = fmaxf(m, s[k].x);
        const float ref = m == -CUDART_INF_F ? 0.f : m, keep = exp2f(M - ref);
        M = m;
        L *= keep;
#pragma unroll
        for (int i = 0; i < kMergeDims; ++i) o[i] *= keep;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (p0 + k >= n) break;
            const float f = exp2f(s[k].x - ref);
            L = fmaf(f, s[k].y, L);
#pragma unroll
            for (int i = 0; i < kMergeDims / 4; ++i) {
                o[4 * i] = fmaf(f, x[k][i].x, o[4 * i]);
                o[4 * i + 1] = fmaf(f, x[k][i].y, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(f, x[k][i].z, o[4 * i + 2]);
                o[4 * i + 3] = fmaf(f, x[k][i].w, o[4 * i + 3]);
            }
        }
    }
    float f = L == 0.f ? 0.f : 1.f / L;
    if (a.v_scale != nullptr && L != 0.f) f *= a.v_scale[u.kvh];
    const int64_t qh = int64_t(u.first + w * a.tq + tok) * a.heads + u.kvh * a.group + hd;
    uint32_t y[kMergeDims / 2];
#pragma unroll
    for (int i = 0; i < kMergeDims / 2; ++i) {
        const float p = L == 0.f ? 0.f : o[2 * i] * f, q = L == 0.f ? 0.f : o[2 * i + 1] * f;
        const __nv_bfloat162 yb = __floats2bfloat162_rn(p, q);
        const __half2 yh = __floats2half2_rn(p, q);
        y[i] = out_bf16 ? *reinterpret_cast<const uint32_t*>(&yb)
                        : *reinterpret_cast<const uint32_t*>(&yh);
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + qh * D + part * kMergeDims);
    out[0] = make_uint4(y[0], y[1], y[2], y[3]);
    out[1] = make_uint4(y[4], y[5], y[6], y[7]);
    if (part == 0 && a.lse != nullptr)
        a.lse[qh] = L == 0.f ? -CUDART_INF_F : (M + log2f(L)) * kLn2;
}

struct Layout {
    int64_t ml, o, shared, total;
    int32_t unit_rows, ctas;
};

// Workspace: the partial states (two slots per CTA) and the shared units.
// Nothing in it survives a call.
Layout layout(int32_t d) {
    Layout w;
    w.unit_rows = d == 256 ? kTile : 2 * kTile;
    w.ctas = int32_t(hs::min64(kMaxCtas, hs_host::num_sms()));
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    w.ml = take(int64_t(2) * w.ctas * w.unit_rows * 2 * 4);
    w.o = take(int64_t(2) * w.ctas * w.unit_rows * d * 4);
    w.shared = take(int64_t(w.ctas) * sizeof(SharedUnit));
    w.total = at;
    return w;
}

bool too_large(int32_t tokens, int32_t rows, int32_t heads, int32_t max_len) {
    // The places of a call are counted in 63 bits, those of a block in 31.
    return rows > kMaxRows || heads > kMaxHeads || max_len > (1 << 30) || tokens > (1 << 24) ||
           (int64_t(tokens) + rows) * heads >= int64_t(1) << 31;
}

bool bad_shape(int32_t tokens, int32_t rows, int32_t heads, int32_t kv_heads, int32_t d,
               int32_t max_len, int32_t window, int32_t sinks) {
    return tokens < 0 || rows < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 ||
           d <= 0 || max_len < 0 || window < 0 || sinks < 0;
}

}  // namespace
}  // namespace hs_prefill

using namespace hs_prefill;

extern "C" int64_t hs_paged_prefill_workspace_bytes(int32_t tokens, int32_t rows, int32_t heads,
                                                    int32_t kv_heads, int32_t d, int32_t max_len,
                                                    int32_t window, int32_t num_sinks) {
    if (bad_shape(tokens, rows, heads, kv_heads, d, max_len, window, num_sinks) ||
        too_large(tokens, rows, heads, max_len))
        return -1;
    return rows == 0 || tokens == 0 ? 0 : layout(d).total;
}

extern "C" int hs_paged_prefill(const void* q, int64_t q_stride, int32_t q_dtype, int32_t tokens,
                                const void* k, const void* v, int32_t kv_dtype,
                                int64_t page_stride, int64_t row_stride, int64_t head_stride,
                                int32_t num_pages, int32_t page_size, const int32_t* block_table,
                                int64_t bt_stride, int32_t max_blocks, int32_t max_len,
                                const int32_t* cu_new, const int32_t* seq_lens,
                                const float* k_scale, const float* v_scale, int32_t rows,
                                int32_t heads, int32_t kv_heads, int32_t d, int32_t window,
                                int32_t num_sinks, float scale, void* out, float* lse,
                                void* workspace, int64_t workspace_bytes, int32_t* status,
                                hs_stream_t stream) {
    if (bad_shape(tokens, rows, heads, kv_heads, d, max_len, window, num_sinks) ||
        page_size <= 0 || num_pages < 0 || max_blocks < 0 || q_stride < 0 || page_stride < 0 ||
        row_stride < 0 || head_stride < 0 || bt_stride < 0 || q_dtype < HS_BF16 ||
        q_dtype > HS_FP16 || kv_dtype < HS_BF16 || kv_dtype > HS_E4M3 ||
        int64_t(max_blocks) * page_size < max_len)
        return HS_ERR_INVALID_ARG;
    if ((d != 64 && d != 128 && d != 256) || heads / kv_heads > 128 ||
        (kv_dtype != HS_E4M3 && kv_dtype != q_dtype) ||
        (kv_dtype != HS_E4M3 && (k_scale != nullptr || v_scale != nullptr)))
        return HS_ERR_UNSUPPORTED;
    if (too_large(tokens, rows, heads, max_len)) return HS_ERR_CAPACITY;
    if (rows == 0 || tokens == 0) return HS_OK;
    if (q == nullptr || k == nullptr || v == nullptr || cu_new == nullptr || seq_lens == nullptr ||
        out == nullptr || (block_table == nullptr && max_len > 0))
        return HS_ERR_INVALID_ARG;
    const auto al = [](const void* p, uintptr_t n) {
        return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
    };
    const int64_t per16 = kv_dtype == HS_E4M3 ? 16 : 8;  // elements of 16 bytes
    if (!al(q, 16) || q_stride % 8 || !al(k, 16) || !al(v, 16) || page_stride % per16 ||
        row_stride % per16 || head_stride % per16 || !al(out, 16) || !al(lse, 4) ||
        !al(workspace, 256) || !al(seq_lens, 4) || !al(cu_new, 4) || !al(block_table, 4) ||
        !al(k_scale, 4) || !al(v_scale, 4) || !al(status, 4))
        return HS_ERR_MISALIGNED;
    PrefillArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.page_stride = page_stride;
    a.row_stride = row_stride;
    a.head_stride = head_stride;
    a.block_table = block_table;
    a.bt_stride = bt_stride;
    a.cu_new = cu_new;
    a.seq_lens = seq_lens;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.tokens = tokens;
    a.rows = rows;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.group = heads / kv_heads;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (page_size == (1 << i)) a.page_shift = i;
    a.max_len = max_len;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.out_wide = al(out, 32);
    a.lse = lse;
    a.status = status;
    a.q_is_half = q_dtype == HS_FP16;
    // Longer ones than any context see as much.
    a.window = int32_t(hs::min64(window, 1 << 30));
    a.sinks = int32_t(hs::min64(num_sinks, 1 << 30));
    Layout w = layout(d);
    if (workspace == nullptr || workspace_bytes < w.total) return HS_ERR_CAPACITY;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.tq = kTile / a.group;
    const int bt = box_tokens(a, kv_dtype);
    if (one_tile(a, kv_dtype, bt)) w.unit_rows = kTile;
    a.tb = a.tq * (w.unit_rows / kTile);
    a.ctas = w.ctas;
    a.part_ml = reinterpret_cast<float*>(ws + w.ml);
    a.part_o = reinterpret_cast<float*>(ws + w.o);
    a.shared = reinterpret_cast<SharedUnit*>(ws + w.shared);
    a.unit_rows = w.unit_rows;
    // (E4M3: 64 requests of up to 48 tokens over up to 4 K 234 us with 256, 195 with
    // 512; bf16: 8192 fresh tokens 382 us with 256, 392 with 512, 398 with 128.)
    a.extra = kv_dtype == HS_E4M3 ? 512 : 256;
    const int rc = kv_dtype == HS_BF16   ? launch_bf16(a, d, bt, stream)
                   : kv_dtype == HS_FP16 ? launch_fp16(a, d, bt, stream)
                                         : launch_e4m3(a, d, bt, stream);
    if (rc != HS_OK) return rc;
    const dim3 grid{unsigned(a.ctas), unsigned(w.unit_rows / kTile * (d / kMergeDims))}, block{kMergeThreads};
    const int bf = q_dtype == HS_BF16;
    if (d == 64) return hs_host::launch_pdl(merge_kernel<64>, grid, block, 0, stream, a, bf);
    if (d == 128) return hs_host::launch_pdl(merge_kernel<128>, grid, block, 0, stream, a, bf);
    return hs_host::launch_pdl(merge_kernel<256>, grid, block, 0, stream, a, bf);
}
