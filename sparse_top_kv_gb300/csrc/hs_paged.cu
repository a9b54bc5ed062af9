// hs_paged.cu -- hs_paged_decode: argument checks, workspace layout, the
// merge of split contexts and the running attention scores.  The attention
// kernel itself is in hs_paged_core.cuh.
#include <cuda.h>

#include <atomic>

#include "hs_paged.cuh"

namespace hs_paged {

namespace tc {

// The driver's tensor map encoder (a host-side function; no link to libcuda).
using Encode = decltype(&cuTensorMapEncodeTiled);
Encode encoder() {
    static std::atomic<Encode> fn{nullptr};
    Encode f = fn.load(std::memory_order_acquire);
    if (f != nullptr) return f;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult res = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess || p == nullptr) {
        cudaGetLastError();
        return nullptr;
    }
    f = reinterpret_cast<Encode>(p);
    fn.store(f, std::memory_order_release);
    return f;
}

int encode_map(CUtensorMap* m, int kv, const void* base, const PagedArgs& a, int d, int bt,
               int hs_box) {
    const Encode f = encoder();
    if (f == nullptr) return HS_ERR_CUDA;
    const cuuint64_t elt = kv == HS_E4M3 ? 1 : 2;
    // A dimension of one entry may have any stride; the encoder wants a valid one.
    const auto bytes = [&](int64_t stride, int64_t n) {
        return n > 1 ? cuuint64_t(stride) * elt : cuuint64_t(d) * elt;
    };
    const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(a.page_size), cuuint64_t(a.kv_heads),
                                cuuint64_t(a.num_pages)};
    const cuuint64_t strides[3] = {bytes(a.row_stride, a.page_size),
                                   bytes(a.head_stride, a.kv_heads),
                                   bytes(a.page_stride, a.num_pages)};
    const cuuint32_t box[4] = {cuuint32_t(128 / elt), cuuint32_t(bt), cuuint32_t(hs_box), 1u};
    const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    const CUtensorMapDataType type = kv == HS_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                     : kv == HS_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUresult r =
        f(m, type, 4, const_cast<void*>(base), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? HS_OK : HS_ERR_CUDA;
}

}  // namespace tc

namespace {

// The tensor-core kernel takes caches whose boxes of 16 tokens and more lie
// inside a page and whose rows fill 128-byte blocks; others (small or odd
// pages, E4M3 heads of 64 bytes, broadcast strides) run on warp-level MMAs.
bool tensor_map_ok(const PagedArgs& a, int kv_dtype, int d) {
    const int64_t most = int64_t(1) << 38;  // elements; the encoder takes strides below 2^40 bytes
    return a.page_size % 16 == 0 && !(kv_dtype == HS_E4M3 && d == 64) && a.num_pages > 0 &&
           (a.kv_heads == 1 || (a.head_stride > 0 && a.head_stride < most)) &&
           (a.num_pages == 1 || (a.page_stride > 0 && a.page_stride < most)) &&
           a.row_stride > 0 && a.row_stride < most;
}

constexpr int kMergeThreads = 256;
constexpr int kScoreThreads = 128;
constexpr int kScoreTokens = 4 * kScoreThreads;  // tokens of one scoring step

// Merge of the units whose tiles were dealt to several CTAs (the others were
// written by their CTA): out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// A block takes every gridDim.y-th head of a request; a warp reads every
// eighth partial row, so all loads of a merge are in flight at once.  The
// plan depends on seq_lens alone, which no longer changes once the attention
// kernel lets this one start, so it is found while that kernel still runs.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_units(const __grid_constant__ PagedArgs a,
                                                             int out_bf16) {
    constexpr int NW = kMergeThreads / 32;
    constexpr int V4 = D / 4;                    // float4s of a row
    constexpr int PL = V4 > 32 ? V4 / 32 : 1;    // float4s of a lane
    __shared__ float wt[kMaxCtas];
    __shared__ float red[NW];
    __shared__ int sums[NW][4];
    __shared__ float4 acc[NW][V4];
    hs::pdl_trigger();
    const int group = a.heads / a.kv_heads, gch = (group + a.gm - 1) / a.gm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x;
    int n[4] = {0, 0, 0, 0};  // tiles of all rows, and of those before this one, both ways
    for (int r = tid; r < a.rows; r += kMergeThreads) {
        const int len = a.seq_lens[r];
        const int n0 = tiling_of(a, len, a.lth[0]).n, n1 = tiling_of(a, len, a.lth[1]).n;
        n[0] += n0;
        n[1] += n1;
        if (r < row) {
            n[2] += n0;
            n[3] += n1;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = __reduce_add_sync(0xffffffffu, n[i]);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][i] = n[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        n[i] = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) n[i] += sums[w][i];
    }
    const int way = way_of(a, n[0]);
    const Plan pl = plan_of(a, way, way == 0 ? n[0] : n[1]);
    const int row_tiles = tiling_of(a, a.seq_lens[row], a.lth[way]).n;
    const int first_tile = (way == 0 ? n[2] : n[3]) * a.chunks[way];
    const int hs = a.hs[way];
    hs::pdl_wait();
    for (int h = blockIdx.y; h < a.heads; h += gridDim.y) {
        const int kvh = h / group, gi = h % group;
        const int64_t qh = int64_t(row) * a.heads + h;
        const int chunk = kvh / hs * gch + gi / a.gm;
        const int hu = (kvh % hs) * a.gm + gi % a.gm;
        const int start = first_tile + chunk * row_tiles;
        const int c0 = run_of(pl, start), c1 = run_of(pl, start + row_tiles - 1);
        if (c0 == c1) continue;
        const int parts = c1 - c0 + 1;
        // Only the first CTA's part can sit in its second slot.
        const int64_t first =
            int64_t(2 * c0 + (start > run_begin(pl, c0) ? 1 : 0)) * a.unit_heads_max + hu;
        auto part = [&](int p) {
            return p == 0 ? first : int64_t(2 * (c0 + p)) * a.unit_heads_max + hu;
        };
        float m[(kMaxCtas + kMergeThreads - 1) / kMergeThreads];
        float M = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < kMaxCtas / kMergeThreads; ++i) {
            const int p = tid + i * kMergeThreads;
            m[i] = p < parts ? __ldcg(a.part_ml + 2 * part(p)) : -CUDART_INF_F;
            M = fmaxf(M, m[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) red[warp] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) M = fmaxf(M, red[i]);
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxCtas / kMergeThreads; ++i) {
            const int p = tid + i * kMergeThreads;
            if (p < parts) {
                const float w = exp2f(m[i] - ref);
                wt[p] = w;
                L = fmaf(w, __ldcg(a.part_ml + 2 * part(p) + 1), L);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        __syncthreads();
        if (lane == 0) red[warp] = L;
        float4 s[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int p = warp; p < parts; p += NW) {
            const float w = wt[p];
            const float4* po = reinterpret_cast<const float4*>(a.part_o + part(p) * D);
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int c = lane + 32 * i;
                if (c < V4) {
                    const float4 x = __ldcg(po + c);
                    s[i].x = fmaf(w, x.x, s[i].x);
                    s[i].y = fmaf(w, x.y, s[i].y);
                    s[i].z = fmaf(w, x.z, s[i].z);
                    s[i].w = fmaf(w, x.w, s[i].w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane + 32 * i < V4) acc[warp][lane + 32 * i] = s[i];
        __syncthreads();
        L = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) L += red[i];
        for (int d = tid; d < D; d += kMergeThreads) {
            float O = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) O += reinterpret_cast<const float*>(acc[i])[d];
            float r = L == 0.f ? 0.f : O / L;
            if (a.v_scale != nullptr) r *= __ldg(a.v_scale + kvh);
            if (out_bf16) static_cast<__nv_bfloat16*>(a.out)[qh * D + d] = __float2bfloat16_rn(r);
            else static_cast<__half*>(a.out)[qh * D + d] = __float2half_rn(r);
        }
        if (tid == 0) {
            const float lg = L == 0.f ? -CUDART_INF_F : M + log2f(L);
            if (a.lse != nullptr) a.lse[qh] = lg * kLn2;
            if (a.lse2 != nullptr) a.lse2[qh] = lg;
        }
        __syncthreads();
    }
}

// score[r][t] := decay * score[r][t] + sum_h 2^(x[r][h][t] - lse2[r][h]), the
// heads in order; tokens outside the window only decay.  Four tokens a
// thread, so that a warp reads 512 contiguous bytes of a head's logits.
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const __grid_constant__ PagedArgs a,
                                                              int blocks_per_row) {
    hs::pdl_trigger();
    hs::pdl_wait();
    const int row = blockIdx.x / blocks_per_row, part = blockIdx.x % blocks_per_row;
    const Tiling vis = tiling_of(a, a.seq_lens[row], 0);
    const int nvis = vis.T - vis.w0 + vis.sc;
    float* score = a.score + int64_t(row) * a.score_stride;
    const float* lse2 = a.lse2 + int64_t(row) * a.heads;
    // The visible tokens.
    for (int64_t i0 = int64_t(part) * kScoreTokens; i0 < nvis;
         i0 += int64_t(blocks_per_row) * kScoreTokens) {
        const int i = int(i0) + 4 * threadIdx.x;
        if (i >= nvis) break;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        const float* x = a.logits + int64_t(row) * a.heads * a.logit_stride + i;
#pragma unroll 8
        for (int h = 0; h < a.heads; ++h) {
            const float ls = __ldg(lse2 + h);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(x + h * a.logit_stride));
            // A head without any weight (LSE = -inf) adds nothing.
            const float ref = ls == -CUDART_INF_F ? 0.f : ls;
            w[0] += exp2f(v.x - ref);
            w[1] += exp2f(v.y - ref);
            w[2] += exp2f(v.z - ref);
            w[3] += exp2f(v.w - ref);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + j >= nvis) break;
            const int t = i + j < vis.sc ? i + j : i + j - vis.sc + vis.w0;
            score[t] = a.decay == 0.f ? w[j] : fmaf(a.decay, score[t], w[j]);
        }
    }
    // Tokens between the sinks and the window.
    if (a.decay != 1.f)
        for (int64_t t = vis.sc + int64_t(part) * kScoreThreads + threadIdx.x; t < vis.w0;
             t += int64_t(blocks_per_row) * kScoreThreads)
            score[t] = a.decay == 0.f ? 0.f : a.decay * score[t];
}

struct Layout {
    int64_t lse2, ml, o, logits, total, logit_stride;
    int32_t unit_heads, ctas;
};

int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// Workspace: the partial states (two slots per CTA: the unit that its run
// begins in and the one that it ends in) and, for scored calls, the log2 LSE
// and the logits.  Nothing in it survives a call.
Layout layout(int32_t rows, int32_t heads, int32_t kv_heads, int32_t d, int32_t max_len,
              int32_t window, int32_t sinks, bool scored) {
    Layout w;
    const int group = heads / kv_heads;
    const int gm = group <= 8 ? 8 : 16;
    int hs_max = 1;
    while (hs_max < 8 && kv_heads % (2 * hs_max) == 0) hs_max *= 2;
    w.unit_heads = hs_max * gm;
    w.ctas = int32_t(hs::min64(kMaxCtas, hs_host::num_sms()));
    const int64_t vis = window > 0 ? hs::min64(max_len, int64_t(window) + sinks) : max_len;
    w.logit_stride = up(vis, kKey);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    w.lse2 = take(scored ? int64_t(rows) * heads * 4 : 0);
    w.ml = take(int64_t(2) * w.ctas * w.unit_heads * 2 * 4);
    w.o = take(int64_t(2) * w.ctas * w.unit_heads * d * 4);
    w.logits = take(scored ? int64_t(rows) * heads * w.logit_stride * 4 : 0);
    w.total = at;
    return w;
}

bool bad_shape(int32_t rows, int32_t heads, int32_t kv_heads, int32_t d, int32_t max_len,
               int32_t window, int32_t sinks) {
    return rows < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || d <= 0 ||
           max_len < 0 || window < 0 || sinks < 0;
}

}  // namespace
}  // namespace hs_paged

using namespace hs_paged;

extern "C" int64_t hs_paged_decode_workspace_bytes(int32_t rows, int32_t heads, int32_t kv_heads,
                                                   int32_t d, int32_t max_len, int32_t window,
                                                   int32_t num_sinks, int32_t with_score) {
    if (bad_shape(rows, heads, kv_heads, d, max_len, window, num_sinks)) return -1;
    if (rows == 0) return 0;
    return layout(rows, heads, kv_heads, d, max_len, window, num_sinks, with_score != 0).total;
}

extern "C" int hs_paged_decode(const void* q, int64_t q_stride, int32_t q_dtype, const void* k,
                               const void* v, int32_t kv_dtype, int64_t page_stride,
                               int64_t row_stride, int64_t head_stride, int32_t num_pages,
                               int32_t page_size, const int32_t* block_table, int64_t bt_stride,
                               int32_t max_blocks, int32_t max_len, const int32_t* seq_lens,
                               const float* k_scale, const float* v_scale, int32_t rows,
                               int32_t heads, int32_t kv_heads, int32_t d, int32_t window,
                               int32_t num_sinks, float scale, float* score, int64_t score_stride,
                               float score_decay, void* out, float* lse, void* workspace,
                               int64_t workspace_bytes, int32_t* status, hs_stream_t stream) {
    if (bad_shape(rows, heads, kv_heads, d, max_len, window, num_sinks) || page_size <= 0 ||
        num_pages < 0 || max_blocks < 0 || q_stride < 0 || page_stride < 0 || row_stride < 0 ||
        head_stride < 0 || bt_stride < 0 || q_dtype < HS_BF16 || q_dtype > HS_FP16 ||
        kv_dtype < HS_BF16 || kv_dtype > HS_E4M3 || int64_t(max_blocks) * page_size < max_len ||
        (score != nullptr && score_stride < max_len))
        return HS_ERR_INVALID_ARG;
    const int group = heads / kv_heads;
    if ((d != 64 && d != 128 && d != 256) ||
        (kv_dtype != HS_E4M3 && kv_dtype != q_dtype) ||
        (kv_dtype != HS_E4M3 && (k_scale != nullptr || v_scale != nullptr)))
        return HS_ERR_UNSUPPORTED;
    // Tiles (of 16 tokens of a KV head at least) are counted in 31 bits.
    if (rows > kMaxRows ||
        int64_t(rows) * heads * (int64_t(max_len) / 16 + 2) >= (int64_t(1) << 31))
        return HS_ERR_CAPACITY;
    if (rows == 0) return HS_OK;
    if (q == nullptr || k == nullptr || v == nullptr || seq_lens == nullptr || out == nullptr ||
        (block_table == nullptr && max_len > 0))
        return HS_ERR_INVALID_ARG;
    const auto al = [](const void* p, uintptr_t n) {
        return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
    };
    const int64_t per16 = kv_dtype == HS_E4M3 ? 16 : 8;  // elements of 16 bytes
    if (!al(q, 16) || q_stride % 8 || !al(k, 16) || !al(v, 16) || page_stride % per16 ||
        row_stride % per16 || head_stride % per16 || !al(out, 16) || !al(score, 4) ||
        !al(lse, 4) || !al(workspace, 256) || !al(seq_lens, 4) || !al(block_table, 4) ||
        !al(k_scale, 4) || !al(v_scale, 4))
        return HS_ERR_MISALIGNED;
    const Layout w =
        layout(rows, heads, kv_heads, d, max_len, window, num_sinks, score != nullptr);
    if (workspace == nullptr || workspace_bytes < w.total) return HS_ERR_CAPACITY;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    PagedArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.page_stride = page_stride;
    a.row_stride = row_stride;
    a.head_stride = head_stride;
    a.block_table = block_table;
    a.bt_stride = bt_stride;
    a.seq_lens = seq_lens;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.rows = rows;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_len = max_len;
    a.window = window;
    a.sinks = num_sinks;
    a.q_is_half = q_dtype == HS_FP16;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.score = score;
    a.score_stride = score_stride;
    a.decay = score_decay;
    a.lse2 = score != nullptr ? reinterpret_cast<float*>(ws + w.lse2) : nullptr;
    a.part_ml = reinterpret_cast<float*>(ws + w.ml);
    a.part_o = reinterpret_cast<float*>(ws + w.o);
    a.logits = score != nullptr ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
    a.logit_stride = w.logit_stride;
    a.unit_heads_max = w.unit_heads;
    a.ctas = w.ctas;
    a.status = status;
    int rc;
    if (tensor_map_ok(a, kv_dtype, d)) {
        if (kv_dtype == HS_BF16) rc = launch_tc_bf16(a, d, group, stream);
        else if (kv_dtype == HS_FP16) rc = launch_tc_fp16(a, d, group, stream);
        else rc = launch_tc_e4m3(a, d, group, stream);
    } else if (kv_dtype == HS_BF16) rc = launch_bf16(a, d, group, stream);
    else if (kv_dtype == HS_FP16) rc = launch_fp16(a, d, group, stream);
    else rc = launch_e4m3(a, d, group, stream);
    if (rc != HS_OK) return rc;
    // A block per head where the blocks of a wave suffice, else several heads.
    const int by = int(hs::max64(1, hs::min64(heads, 4 * int64_t(w.ctas) / rows)));
    const int bf = q_dtype == HS_BF16;
    const dim3 mg{unsigned(rows), unsigned(by)}, mt{kMergeThreads};
    if (d == 64) rc = hs_host::launch_pdl(merge_units<64>, mg, mt, 0, stream, a, bf);
    else if (d == 128) rc = hs_host::launch_pdl(merge_units<128>, mg, mt, 0, stream, a, bf);
    else rc = hs_host::launch_pdl(merge_units<256>, mg, mt, 0, stream, a, bf);
    if (rc != HS_OK || score == nullptr) return rc;
    // Enough blocks per request for its longest context, within a few waves.
    const int64_t most = hs::max64(1, (int64_t(max_len) + kScoreTokens - 1) / kScoreTokens);
    const int per_row = int(hs::min64(most, hs::max64(1, 16 * int64_t(w.ctas) / rows)));
    return hs_host::launch_pdl(score_kernel, dim3(unsigned(rows) * unsigned(per_row)),
                               dim3(kScoreThreads), 0, stream, a, per_row);
}
