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

// Small calls of few requests with few query heads on a KV head run on the
// warp-level kernel: it starts and ends a unit sooner than the tcgen05 kernel,
// which is ahead where more is streamed and where a cluster's CTAs have very
// few tiles each (and mostly where more query heads share a row; but one to
// eight requests of 2 K to 16 K with 64/8 heads are up to 41 % faster by warps:
// 8 K 19.5 / 13.8).  us in captured graphs, tcgen05 / warps,
// 32/8 heads of 128: one request of 2 K tokens 10.6 / 8.9, 16 K 24.6 / 19.6,
// eight of up to 4 K 18.5 / 16.4, eight of 16 K 88.3 / 92.1, 16 of up to 1 K
// 17.7 / 14.6, 32 of up to 2 K 32.9 / 36.3, 16 of 256 9.1 / 12.0; 64/8 heads:
// one request of 1 K 9.2 / 9.9; 12/12 heads of 64: eight of 1 K 13.6 / 11.8, of
// 8 K 40.8 / 43.8.
constexpr int kWarpRows = 16, kWarpGroup = 4;
constexpr int kWarpTiles = 28;  // tiles of 128 tokens of a KV head per CTA, at most
bool by_warps(const PagedArgs& a, int kv_dtype, int d) {
    if (kv_dtype == HS_E4M3 || d > 128 || a.group > kWarpGroup || a.rows > kWarpRows) return false;
    const int64_t units = int64_t(a.rows) * a.kv_heads, tiles = most_tiles(a, 7);
    const bool clusters = units <= a.ctas && tiles <= (units > 64 ? 4 : 3);
    return !clusters && units * tiles <= int64_t(a.ctas) * kWarpTiles;
}

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kHeadChunk = 256;  // heads whose LSE a scoring block holds at a time

// Where the units of one request lie in the call's runs of tiles.
struct RowPlan {
    Plan pl;
    int way, row_tiles, first_place;
};
// Found by every warp for itself (a lane per request, no barrier).
__device__ __forceinline__ RowPlan row_plan(const PagedArgs& a, int row) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    int n0 = 0, n1 = 0, b0 = 0, b1 = 0, own0 = 0, own1 = 0;
    if (a.cl > 0) return RowPlan{};  // nothing to merge
#pragma unroll 4
    for (int r = lane; r < a.rows; r += 32) {
        const int len = a.seq_lens[r];
        const int t0 = tiling_of(a, len, a.lth[0]).n, t1 = tiling_of(a, len, a.lth[1]).n;
        n0 += places(a, t0);
        n1 += places(a, t1);
        if (r < row) {
            b0 += places(a, t0);
            b1 += places(a, t1);
        }
        if (r == row) {
            own0 = t0;
            own1 = t1;
        }
    }
    n0 = __reduce_add_sync(kAll, n0);
    RowPlan p;
    p.way = way_of(a, n0);
    const bool narrow = p.way != 0;
    p.pl = plan_of(a, p.way, narrow ? __reduce_add_sync(kAll, n1) : n0);
    p.row_tiles = __shfl_sync(kAll, narrow ? own1 : own0, row & 31);
    p.first_place = __reduce_add_sync(kAll, narrow ? b1 : b0) * a.chunks[p.way];
    return p;
}
// The parts that a query head's unit was dealt to: part p (one per CTA) of the
// head is entry at(p) of the partial states.
struct Parts {
    int n;
    int64_t first, rest;
    int64_t step;
    __device__ __forceinline__ int64_t at(int p) const { return p == 0 ? first : rest + p * step; }
};
__device__ __forceinline__ Parts parts_of(const PagedArgs& a, const RowPlan& r, int h) {
    if (a.cl > 0) return Parts{1, 0, 0, 0};
    // hs and gm are powers of two.
    const int lhs = 31 - __clz(a.hs[r.way]), lgm = 31 - __clz(a.gm);
    const int group = a.group, gch = (group + a.gm - 1) >> lgm;
    const int kvh = div_small(h, group), gi = h - kvh * group;
    const int hu = ((kvh & (a.hs[r.way] - 1)) << lgm) + (gi & (a.gm - 1));
    const int start =
        r.first_place + ((kvh >> lhs) * gch + (gi >> lgm)) * places(a, r.row_tiles);
    Parts p{};
    if (r.row_tiles == 0) return p;  // a request without tokens
    const int c0 = run_of(r.pl, start + a.extra);
    const int c1 = run_of(r.pl, start + a.extra + r.row_tiles - 1);
    p.n = c1 - c0 + 1;
    p.step = 2 * int64_t(a.unit_heads_max);
    p.rest = c0 * p.step + hu;
    // Only the first CTA's part can sit in its second slot.
    p.first = p.rest + (start > run_begin(r.pl, c0) ? a.unit_heads_max : 0);
    return p;
}

// Merge of the units whose tiles were dealt to several CTAs (the others were
// written by their CTA): out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// A warp's share is the parts first, first + step, ..: a lane per part for the
// maxima and sums, and the partial rows requested together with them.
template <int D>
struct MergeState {
    static constexpr int V4 = D / 4;                  // float4s of a row
    static constexpr int PL = V4 > 32 ? V4 / 32 : 1;  // float4s of a lane
    float m, l;
    float4 o[PL];
};
template <int D, int AHEAD>
__device__ __forceinline__ MergeState<D> merge_share(const PagedArgs& a, const Parts& parts,
                                                     int first, int step) {
    using S = MergeState<D>;
    const int lane = threadIdx.x & 31;
    S s;
    s.m = -CUDART_INF_F;
    s.l = 0.f;
#pragma unroll
    for (int i = 0; i < S::PL; ++i) s.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = AHEAD / S::PL;  // partial rows requested along with the weights
    for (int p0 = first; p0 < parts.n; p0 += 32 * step) {
        const int n = min(32, (parts.n - p0 + step - 1) / step);
        const int p = p0 + lane * step;
        const float2 ml = p < parts.n
                              ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + parts.at(p))
                              : make_float2(-CUDART_INF_F, 0.f);
        float4 x[kAhead][S::PL];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (k0 + k < n) {
                    const float4* po = reinterpret_cast<const float4*>(
                        a.part_o + parts.at(p0 + (k0 + k) * step) * D);
#pragma unroll
                    for (int i = 0; i < S::PL; ++i)
                        if (S::V4 >= 32 || lane < S::V4) x[k][i] = __ldcg(po + lane + 32 * i);
                }
        };
        load(0);
        float mx = fmaxf(s.m, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        const float keep = exp2f(s.m - ref), w = exp2f(ml.x - ref);
        float l = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        s.l = fmaf(s.l, keep, l);
        s.m = mx;
        if (p0 != first) {
#pragma unroll
            for (int i = 0; i < S::PL; ++i) {
                s.o[i].x *= keep;
                s.o[i].y *= keep;
                s.o[i].z *= keep;
                s.o[i].w *= keep;
            }
        }
        for (int k0 = 0; k0 < n; k0 += kAhead) {
            if (k0 > 0) load(k0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float f = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
                if (k0 + k < n) {
#pragma unroll
                    for (int i = 0; i < S::PL; ++i) {
                        if (S::V4 < 32 && lane >= S::V4) break;
                        s.o[i].x = fmaf(f, x[k][i].x, s.o[i].x);
                        s.o[i].y = fmaf(f, x[k][i].y, s.o[i].y);
                        s.o[i].z = fmaf(f, x[k][i].z, s.o[i].z);
                        s.o[i].w = fmaf(f, x[k][i].w, s.o[i].w);
                    }
                }
            }
        }
    }
    return s;
}

// One warp writes a head's merged state.
template <int D>
__device__ __forceinline__ void write_head(const PagedArgs& a, int64_t qh, int kvh,
                                           const MergeState<D>& s, int out_bf16) {
    using S = MergeState<D>;
    const int lane = threadIdx.x & 31;
    float f = s.l == 0.f ? 0.f : 1.f / s.l;
    if (a.v_scale != nullptr && s.l != 0.f) f *= a.v_scale[kvh];
#pragma unroll
    for (int i = 0; i < S::PL; ++i) {
        if (S::V4 < 32 && lane >= S::V4) break;
        const float4 x = s.o[i];
        const int64_t at = qh * D + 4 * (lane + 32 * i);
        if (out_bf16) {
            __nv_bfloat162 y[2] = {__floats2bfloat162_rn(x.x * f, x.y * f),
                                   __floats2bfloat162_rn(x.z * f, x.w * f)};
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                *reinterpret_cast<const uint2*>(y);
        } else {
            __half2 y[2] = {__floats2half2_rn(x.x * f, x.y * f),
                            __floats2half2_rn(x.z * f, x.w * f)};
            *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) =
                *reinterpret_cast<const uint2*>(y);
        }
    }
    if (lane == 0 && a.lse != nullptr)
        a.lse[qh] = s.l == 0.f ? -CUDART_INF_F : (s.m + log2f(s.l)) * kLn2;
}

// A block takes 8 / wp heads of a request, wp warps (1, 2, 4 or 8) to a head.
template <int D, int AHEAD>
__device__ __forceinline__ void merge_heads(const PagedArgs& a, const RowPlan& plan, int row,
                                            int part, int wp, int out_bf16) {
    using S = MergeState<D>;
    __shared__ float2 ml_s[kMergeWarps];
    __shared__ float4 o_s[kMergeWarps][S::V4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = part * (kMergeWarps / wp) + warp / wp;
    Parts parts{};
    if (h < a.heads) parts = parts_of(a, plan, h);
    // A request without a token has no part: zeros.
    const bool mine = h < a.heads && parts.n != 1;
    hs::pdl_wait();
    S s = merge_share<D, AHEAD>(a, parts.n > 1 ? parts : Parts{}, warp % wp, wp);
    if (wp > 1 && parts.n > 1) {
        if (lane == 0) ml_s[warp] = make_float2(s.m, s.l);
#pragma unroll
        for (int j = 0; j < S::PL; ++j)
            if (S::V4 >= 32 || lane < S::V4) o_s[warp][lane + 32 * j] = s.o[j];
    }
    if (wp > 1) __syncthreads();
    if (!mine || warp % wp != 0) return;
    if (wp > 1 && parts.n > 1) {
        float M = s.m;
        for (int w = 1; w < wp; ++w) M = fmaxf(M, ml_s[warp + w].x);
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        const float own = exp2f(s.m - ref);
        s.l *= own;
#pragma unroll
        for (int j = 0; j < S::PL; ++j) {
            s.o[j].x *= own;
            s.o[j].y *= own;
            s.o[j].z *= own;
            s.o[j].w *= own;
        }
        for (int w = 1; w < wp; ++w) {
            const float f = exp2f(ml_s[warp + w].x - ref);
            s.l = fmaf(f, ml_s[warp + w].y, s.l);
#pragma unroll
            for (int j = 0; j < S::PL; ++j) {
                if (S::V4 < 32 && lane >= S::V4) break;
                const float4 x = o_s[warp + w][lane + 32 * j];
                s.o[j].x = fmaf(f, x.x, s.o[j].x);
                s.o[j].y = fmaf(f, x.y, s.o[j].y);
                s.o[j].z = fmaf(f, x.z, s.o[j].z);
                s.o[j].w = fmaf(f, x.w, s.o[j].w);
            }
        }
        s.m = M;
    }
    write_head<D>(a, int64_t(row) * a.heads + h, div_small(h, a.group), s, out_bf16);
}

// score[r][t] := decay * score[r][t] + sum_h 2^(x[r][h][t] - LSE[r][h]), the
// heads in order; tokens outside the window only decay.  A thread per token,
// sixteen heads' logits in flight; the heads' LSE first, eight lanes to a
// head over its parts, so that this needs no merge to have finished.
__device__ __forceinline__ void score_tokens(const PagedArgs& a, const RowPlan& plan, int row,
                                             int part, int blocks) {
    __shared__ float lse2[kHeadChunk];
    constexpr int kLanes = 8, kAtOnce = kMergeThreads / kLanes;  // lanes of a head, heads at once
    const int tid = threadIdx.x;
    const Tiling vis = tiling_of(a, a.seq_lens[row], 0);
    const int nvis = vis.T - vis.w0 + vis.sc;
    float* score = a.score + int64_t(row) * a.score_stride;
    Parts ahead{};  // of this thread's first head
    if (tid / kLanes < a.heads && (plan.row_tiles > 0 || a.cl > 0)) ahead = parts_of(a, plan, tid / kLanes);
    hs::pdl_wait();
    for (int64_t i0 = int64_t(part) * kMergeThreads; i0 < nvis;
         i0 += int64_t(blocks) * kMergeThreads) {
        const int i = int(i0) + tid;
        float w = 0.f;
        for (int hc = 0; hc < a.heads; hc += kHeadChunk) {
            const int nh = min(kHeadChunk, a.heads - hc);
            if (a.heads > kHeadChunk || i0 == int64_t(part) * kMergeThreads) {
                __syncthreads();
                for (int h0 = 0; h0 < nh; h0 += kAtOnce) {
                    const int h = h0 + tid / kLanes, l = tid % kLanes;
                    float M = -CUDART_INF_F, L = 0.f;
                    if (h < nh) {
                        const Parts parts =
                            h0 == 0 && hc == 0 ? ahead : parts_of(a, plan, hc + h);
                        if (parts.n == 1) {
                            M = __ldcg(a.lse2 + int64_t(row) * a.heads + hc + h);
                            L = l == 0 ? 1.f : 0.f;
                        } else {
#pragma unroll 4
                            for (int p = l; p < parts.n; p += kLanes) {
                                const float2 ml = __ldcg(
                                    reinterpret_cast<const float2*>(a.part_ml) + parts.at(p));
                                const float m = fmaxf(M, ml.x);
                                const float ref = m == -CUDART_INF_F ? 0.f : m;
                                L = fmaf(L, exp2f(M - ref), ml.y * exp2f(ml.x - ref));
                                M = m;
                            }
                        }
                    }
                    const float own = M;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1)
                        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                    L *= exp2f(own - (M == -CUDART_INF_F ? 0.f : M));
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1)
                        L += __shfl_xor_sync(0xffffffffu, L, o);
                    // A head without any weight adds nothing: subtract 0.
                    const float lg = L == 0.f ? -CUDART_INF_F : M + log2f(L);
                    if (l == 0 && h < nh) lse2[h] = lg == -CUDART_INF_F ? 0.f : lg;
                }
                __syncthreads();
            }
            if (i < nvis) {
                const float* x =
                    a.logits + (int64_t(row) * a.heads + hc) * a.logit_stride + i;
#pragma unroll 16
                for (int h = 0; h < nh; ++h)
                    w += exp2f(__ldcg(x + h * a.logit_stride) - lse2[h]);
            }
        }
        if (i < nvis) {
            const int t = i < vis.sc ? i : i - vis.sc + vis.w0;
            score[t] = a.decay == 0.f ? w : fmaf(a.decay, score[t], w);
        }
    }
    // Tokens between the sinks and the window.
    if (a.decay != 1.f)
        for (int64_t t = vis.sc + int64_t(part) * kMergeThreads + tid; t < vis.w0;
             t += int64_t(blocks) * kMergeThreads)
            score[t] = a.decay == 0.f ? 0.f : a.decay * score[t];
}

// What follows the attention: block (row, y) with y < merges joins the parts
// of some heads of a request, the others score its tokens.  The plan depends
// on seq_lens alone, which no longer changes once the attention kernel lets
// this one start, so it is found while that kernel still runs.
template <int D, int AHEAD>
__global__ void __launch_bounds__(kMergeThreads, AHEAD > 4 ? 2 : 4) finish_kernel(const __grid_constant__ PagedArgs a,
                                                               int merges, int wp, int out_bf16) {
    hs::pdl_trigger();
    const RowPlan plan = row_plan(a, blockIdx.x);
    if (int(blockIdx.y) < merges)
        merge_heads<D, AHEAD>(a, plan, blockIdx.x, blockIdx.y, wp, out_bf16);
    else
        score_tokens(a, plan, blockIdx.x, blockIdx.y - merges, gridDim.y - merges);
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

// Tiles (of 16 tokens of a KV head at least) are counted in 31 bits; the
// finishing kernel's grid has a block for up to eight heads in its y dimension.
bool too_large(int32_t rows, int32_t heads, int32_t max_len) {
    return rows > kMaxRows || heads > kMaxHeads || max_len > (1 << 30) ||
           int64_t(rows) * heads * (int64_t(max_len) / 16 + 16) >= (int64_t(1) << 31);
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
    if (bad_shape(rows, heads, kv_heads, d, max_len, window, num_sinks) ||
        too_large(rows, heads, max_len))
        return -1;
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
    if (too_large(rows, heads, max_len)) return HS_ERR_CAPACITY;
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
    a.group = group;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (page_size == (1 << i)) a.page_shift = i;
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
    if (tensor_map_ok(a, kv_dtype, d) && !by_warps(a, kv_dtype, d)) {
        if (kv_dtype == HS_BF16) rc = launch_tc_bf16(a, d, group, stream);
        else if (kv_dtype == HS_FP16) rc = launch_tc_fp16(a, d, group, stream);
        else rc = launch_tc_e4m3(a, d, group, stream);
    } else if (kv_dtype == HS_BF16) rc = launch_bf16(a, d, group, stream);
    else if (kv_dtype == HS_FP16) rc = launch_fp16(a, d, group, stream);
    else rc = launch_e4m3(a, d, group, stream);
    if (rc != HS_OK || (a.cl > 0 && score == nullptr)) return rc;
    // Merging: about half as many warps to a head as its unit has parts (one
    // context over all SMs has 152), within a few blocks an SM.  The kernel
    // chose between the two ways by the lengths; here their bound decides.
    // Scoring: a block per step of tokens where a few waves hold them, else
    // several steps a block.
    const int64_t most = most_places(a);
    const int way = most < a.wide_from || most >= a.wide_to ? 1 : 0;
    const int64_t units = int64_t(rows) * a.chunks[way];
    const int64_t parts = hs::min64(most_places(a, way) / hs::max64(1, units),
                                    w.ctas / hs::max64(1, units) + 2);
    int wp = 1;
    while (wp < kMergeWarps && 2 * wp <= parts &&
           int64_t(rows) * heads * 2 * wp <= 4 * int64_t(w.ctas) * kMergeWarps)
        wp *= 2;
    const int merges = a.cl > 0 ? 0 : (heads * wp + kMergeWarps - 1) / kMergeWarps;
    const int64_t steps = (int64_t(max_len) + kMergeThreads - 1) / kMergeThreads;
    const int scores =
        score == nullptr ? 0
                         : int(hs::max64(1, hs::min64(steps, 16 * int64_t(w.ctas) / rows)));
    const int bf = q_dtype == HS_BF16;
    const dim3 grid{unsigned(rows), unsigned(merges + scores)}, block{kMergeThreads};
    // Sixteen rows in flight a warp where there are many parts (they take the
    // registers of half the blocks: 131 K tokens merge in 5.0 us instead of
    // 7.0, but a batch's 512 blocks in 4.1 instead of 2.7).
    const auto finish = [&](auto narrow, auto deep) {
        return parts > 4 * wp ? hs_host::launch_pdl(deep, grid, block, 0, stream, a, merges, wp, bf)
                              : hs_host::launch_pdl(narrow, grid, block, 0, stream, a, merges, wp, bf);
    };
    if (d == 64) return finish(finish_kernel<64, 4>, finish_kernel<64, 16>);
    if (d == 128) return finish(finish_kernel<128, 4>, finish_kernel<128, 16>);
    return finish(finish_kernel<256, 4>, finish_kernel<256, 16>);
}
