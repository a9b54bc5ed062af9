// hs_prefill.cu -- hs_paged_prefill: argument checks and the attention of a
// chunk of new tokens over a paged cache.
#include <type_traits>

#include "hs_prefill.cuh"

namespace hs_prefill {
namespace {

template <typename T>
__device__ __forceinline__ float widen(T x) {
    return float(x);
}

// A warp per (new token, query head): a lane holds d / 32 elements of the query
// and of the sum, keys one after another with a running maximum.
template <typename Q, typename K, int D>
__global__ void __launch_bounds__(256) simple_kernel(const __grid_constant__ PrefillArgs a) {
    constexpr int N = D / 32;
    hs::pdl_wait();
    hs::pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int token = int(unit / a.heads), h = int(unit % a.heads);
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r < a.rows; r += blockDim.x) {
            const int c0 = a.cu_new[r], c1 = a.cu_new[r + 1];
            if (a.seq_lens[r] > a.max_len || c0 < 0 || c1 < c0 || c1 > a.tokens)
                hs::set_status(a.status, HS_ERR_BAD_INDEX);
        }
    if (token >= a.tokens || a.rows == 0) return;
    int lo = 0, hi = a.rows;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu_new[mid] <= token) lo = mid;
        else hi = mid;
    }
    const Request x = request_of(a, lo);
    if (token < x.first || token >= x.first + x.n) return;
    const int g = h / a.group, pos = x.T - x.n + (token - x.first);
    const Q* q = static_cast<const Q*>(a.q) + token * a.q_stride + int64_t(h) * D + lane * N;
    float qf[N], o[N];
    const float scale = a.scale_log2 * (a.k_scale != nullptr ? a.k_scale[g] : 1.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        qf[i] = widen(q[i]) * scale;
        o[i] = 0.f;
    }
    float m = -CUDART_INF_F, l = 0.f;
    bool bad = false;
    for (int t = 0; t <= pos; ++t) {
        if (a.window > 0 && t <= pos - a.window && t >= a.sinks) {
            t = pos - a.window;
            continue;
        }
        const int b = block_of(a, t), page = a.block_table[lo * a.bt_stride + b];
        if (page < 0 || page >= a.num_pages) {
            bad = true;
            continue;
        }
        const int64_t at = page * a.page_stride + (t - b * a.page_size) * a.row_stride +
                           g * a.head_stride + lane * N;
        const K* k = static_cast<const K*>(a.k) + at;
        const K* v = static_cast<const K*>(a.v) + at;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s = fmaf(qf[i], widen(k[i]), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float mn = fmaxf(m, s), ref = mn == -CUDART_INF_F ? 0.f : mn;
        const float keep = exp2f(m - ref), p = exp2f(s - ref);
        m = mn;
        l = fmaf(l, keep, p);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(p, widen(v[i]), o[i] * keep);
    }
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    const float f = l == 0.f ? 0.f : (a.v_scale != nullptr ? a.v_scale[g] : 1.f) / l;
    const int64_t at = int64_t(token) * a.heads + h;
    Q* out = static_cast<Q*>(a.out) + at * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = Q(l == 0.f ? 0.f : o[i] * f);
    if (lane == 0 && a.lse != nullptr)
        a.lse[at] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

bool too_large(int32_t tokens, int32_t rows, int32_t heads, int32_t max_len) {
    return rows > kMaxRows || heads > kMaxHeads || max_len > (1 << 30) || tokens > (1 << 24);
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
    return 0;
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
    a.window = window;
    a.sinks = num_sinks;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.status = status;
    (void)workspace;
    (void)workspace_bytes;
    const dim3 grid{unsigned((int64_t(tokens) * heads + 7) / 8)};
    const auto launch = [&](auto qt, auto kt) {
        using Q = decltype(qt);
        using K = decltype(kt);
        if (d == 64)
            return hs_host::launch_pdl(simple_kernel<Q, K, 64>, grid, dim3(256), 0, stream, a);
        if (d == 128)
            return hs_host::launch_pdl(simple_kernel<Q, K, 128>, grid, dim3(256), 0, stream, a);
        return hs_host::launch_pdl(simple_kernel<Q, K, 256>, grid, dim3(256), 0, stream, a);
    };
    if (kv_dtype == HS_BF16) return launch(__nv_bfloat16{}, __nv_bfloat16{});
    if (kv_dtype == HS_FP16) return launch(__half{}, __half{});
    return q_dtype == HS_FP16 ? launch(__half{}, __nv_fp8_e4m3{})
                              : launch(__nv_bfloat16{}, __nv_fp8_e4m3{});
}
