// hs_rope.cu -- hs_rope_append: rotary positions on the queries and keys of a
// step's tokens, and the rotated keys and the values into a paged cache.
//
// A pair (a, b) of a head at position p becomes
//   (a cos - b sin, a sin + b cos) * mscale,  angle = 2 pi frac(p * turns / 2^64),
// with turns the pair's turns per position as a 64-bit binary fraction.  The
// product wraps exactly at whole turns, so far positions lose nothing: an
// angle is off by 2 pi (p 2^-65 + 2^-26) at most, of the table's rounding to the
// nearest 2^-64 and of the angle's to fp32 for cospi / sinpi.
//
// Every element is read once and written once with a handful of operations,
// so HBM bounds it.  A CTA takes a token: a thread keeps one place of 16 elements
// of the head for all its heads and moves 16-byte vectors, three rows of them
// asked for before the token's position is known; meanwhile the threads make the
// token's sines and cosines once, each for one pair, and pass them through shared
// memory.  Measured over inputs that change from call to call: 8192 tokens of 32 + 8
// heads of 128, 201 MB, 33.4 us (6.0 TB/s), 4113 tokens of 16 + 4 heads over an E4M3
// cache 14.5, one token 3.3; replays of a captured graph over the same inputs 32.8
// (without the rows ahead and with 128 threads 38.5), 11.1 (46 MB: they stay in the
// L2) and 2.8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "hs_common.cuh"

namespace {

// Threads of a CTA: small CTAs keep more rows in flight on an SM; where there are
// SMs to spare, a token has more of them (one token 2.8 us, by 64 threads 3.6, the
// same inputs again).
constexpr int kThreads = 64, kManyThreads = 256;
constexpr int kMaxDim = 1024;
constexpr int kAhead = 3;  // rows of a thread in flight

struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements from token to token
    const int32_t* positions;
    const int32_t* slot;
    const uint64_t* turns;
    void* q_out;
    void* k_cache;
    void* v_cache;
    int64_t page_stride, row_stride, head_stride;  // elements
    int64_t num_slots;
    int32_t page_size;
    const float* k_scale;
    const float* v_scale;
    int32_t tokens, heads, kv_heads, d, half, interleaved;
    float mscale;
    int32_t* status;
};

template <typename T>
__device__ __forceinline__ float2 widen(uint32_t w) {
    if constexpr (std::is_same_v<T, __half>)
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(float x, float y) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
__device__ __forceinline__ uint32_t narrow_e4m3(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// cos and sin of the pair's angle at position p.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int pair, int p) {
    const int64_t t = int64_t(a.turns[pair] * uint64_t(uint32_t(p)));
    // Half turns in [-1, 1).
    const float x = float(int32_t(t >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * a.mscale, s * a.mscale);
}

// One row (head) of a token.
struct Row {
    char* dst;
    float scale;  // E4M3: the divisor
    bool rotate, e4m3;
};
__device__ __forceinline__ const char* source_of(const RopeArgs& a, int token, int r) {
    const int kv = r - a.heads;
    if (kv < 0) return static_cast<const char*>(a.q) + (token * a.q_stride + int64_t(r) * a.d) * 2;
    const bool key = kv < a.kv_heads;
    return static_cast<const char*>(key ? a.k : a.v) +
           (token * (key ? a.k_stride : a.v_stride) +
            int64_t(key ? kv : kv - a.kv_heads) * a.d) * 2;
}
template <typename T>
__device__ __forceinline__ bool row_of(const RopeArgs& a, int token, int r, int64_t at, bool e4m3,
                                       Row& x) {
    const int kv = r - a.heads;
    if (kv < 0) {
        x.dst = static_cast<char*>(a.q_out) + (token * a.q_out_stride + int64_t(r) * a.d) * 2;
        x.rotate = true;
        x.e4m3 = false;
        x.scale = 1.f;
        return true;
    }
    const bool key = kv < a.kv_heads;
    const int g = key ? kv : kv - a.kv_heads;
    x.dst = static_cast<char*>(key ? a.k_cache : a.v_cache) +
            (at + g * a.head_stride) * (e4m3 ? 1 : 2);
    x.rotate = key;
    x.e4m3 = e4m3;
    const float* s = key ? a.k_scale : a.v_scale;
    x.scale = s != nullptr ? s[g] : 1.f;
    return at >= 0;
}

// Eight elements of the row at element i.
template <typename T>
__device__ __forceinline__ void put8(const Row& x, int i, const float (&f)[8]) {
    if (!x.e4m3) {
        uint4 w;
        w.x = narrow<T>(f[0], f[1]);
        w.y = narrow<T>(f[2], f[3]);
        w.z = narrow<T>(f[4], f[5]);
        w.w = narrow<T>(f[6], f[7]);
        *reinterpret_cast<uint4*>(x.dst + i * 2) = w;
    } else {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x.scale == 1.f ? f[j] : f[j] / x.scale;
        uint2 w;
        w.x = narrow_e4m3(y[0], y[1]) | (narrow_e4m3(y[2], y[3]) << 16);
        w.y = narrow_e4m3(y[4], y[5]) | (narrow_e4m3(y[6], y[7]) << 16);
        *reinterpret_cast<uint2*>(x.dst + i) = w;
    }
}

// VEC: d and the rotated part are multiples of 16; places are 16 elements of a
// head (two runs of eight), else a pair.
template <typename T, bool E4M3, bool VEC>
__global__ void __launch_bounds__(kManyThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 cs[kMaxDim / 2];
    const int tid = threadIdx.x, threads = blockDim.x, token = blockIdx.x;
    const int half = a.half, d = a.d;
    const int rows = (a.q != nullptr ? a.heads : 0) + (a.k != nullptr ? 2 * a.kv_heads : 0);
    const int first = a.q != nullptr ? 0 : a.heads;
    // VEC: the thread's place, its two runs of elements, and its first row.
    const int places = VEC ? d / 16 : 1, per = threads / places;
    const int j = tid % places, r0 = tid / places;
    const bool in = 16 * j < 2 * half;  // its elements are rotated
    const int i0 = !in || a.interleaved ? 16 * j : 8 * j, i1 = in && !a.interleaved ? i0 + half : i0 + 8;
    uint4 w[kAhead][2];
    const auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = base + r0 + k * per;
            if (r0 >= per || r >= rows) break;
            const char* src = source_of(a, token, first + r);
            w[k][0] = *reinterpret_cast<const uint4*>(src + i0 * 2);
            w[k][1] = *reinterpret_cast<const uint4*>(src + i1 * 2);
        }
    };
    hs::pdl_wait();
    hs::pdl_trigger();
    // (A token without a position is read all the same: the rows need not wait
    // for it.)
    if (VEC) load(0);
    const int pos = a.positions[token];
    if (pos < 0) return;
    const int slot = a.slot != nullptr ? a.slot[token] : -1;
    int64_t at = -1;
    if (slot >= 0 && slot < a.num_slots) {
        const int page = slot / a.page_size;
        at = page * a.page_stride + (slot - page * a.page_size) * a.row_stride;
    } else if (slot >= 0 && tid == 0) {
        hs::set_status(a.status, HS_ERR_BAD_INDEX);
    }
    for (int i = tid; i < half; i += threads) cs[i] = turn_of(a, i, pos);
    __syncthreads();
    if constexpr (VEC) {
        if (r0 >= per) return;
        float2 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = in ? cs[8 * j + i] : make_float2(1.f, 0.f);
        for (int base = 0; base < rows; base += kAhead * per) {
            if (base > 0) load(base);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int r = base + r0 + k * per;
                if (r >= rows) break;
                Row x;
                if (!row_of<T>(a, token, first + r, at, E4M3, x)) continue;
                const uint4 w0 = w[k][0], w1 = w[k][1];
                if (!x.e4m3 && !(in && x.rotate)) {
                    *reinterpret_cast<uint4*>(x.dst + i0 * 2) = w0;
                    *reinterpret_cast<uint4*>(x.dst + i1 * 2) = w1;
                    continue;
                }
                float y0[8], y1[8];
                const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p0 = widen<T>(u0[i]), p1 = widen<T>(u1[i]);
                    y0[2 * i] = p0.x;
                    y0[2 * i + 1] = p0.y;
                    y1[2 * i] = p1.x;
                    y1[2 * i + 1] = p1.y;
                }
                if (in && x.rotate) {
                    if (a.interleaved) {
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 c0 = f[i / 2], c1 = f[4 + i / 2];
                            const float a0 = y0[i], b0 = y0[i + 1], a1 = y1[i], b1 = y1[i + 1];
                            y0[i] = a0 * c0.x - b0 * c0.y;
                            y0[i + 1] = a0 * c0.y + b0 * c0.x;
                            y1[i] = a1 * c1.x - b1 * c1.y;
                            y1[i + 1] = a1 * c1.y + b1 * c1.x;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float p = y0[i], q = y1[i];
                            y0[i] = p * f[i].x - q * f[i].y;
                            y1[i] = p * f[i].y + q * f[i].x;
                        }
                    }
                }
                put8<T>(x, i0, y0);
                put8<T>(x, i1, y1);
            }
        }
    } else {
        const int places = d / 2;
        for (int64_t e = tid; e < int64_t(rows) * places; e += threads) {
            const int r = int(e / places), j = int(e - int64_t(r) * places);
            Row x;
            if (!row_of<T>(a, token, first + r, at, E4M3, x)) continue;
            const bool in = j < half;
            const int i0 = in && !a.interleaved ? j : 2 * j;
            const int i1 = in && !a.interleaved ? j + half : i0 + 1;
            const T* src = reinterpret_cast<const T*>(source_of(a, token, first + r));
            float p = float(src[i0]), q = float(src[i1]);
            if (in && x.rotate) {
                const float2 f = cs[j];
                const float y = p * f.x - q * f.y;
                q = p * f.y + q * f.x;
                p = y;
            }
            if (x.e4m3) {
                const uint32_t w = narrow_e4m3(p / x.scale, q / x.scale);
                x.dst[i0] = char(w & 255u);
                x.dst[i1] = char(w >> 8);
            } else {
                const uint32_t w = narrow<T>(p, q);
                reinterpret_cast<uint16_t*>(x.dst)[i0] = uint16_t(w);
                reinterpret_cast<uint16_t*>(x.dst)[i1] = uint16_t(w >> 16);
            }
        }
    }
}

}  // namespace

extern "C" int hs_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, int32_t dtype, int32_t tokens,
                              int32_t heads, int32_t kv_heads, int32_t d, const int32_t* positions,
                              const int32_t* slot, const int64_t* turns, int32_t rot,
                              int32_t interleaved, float mscale, void* q_out, int64_t q_out_stride,
                              void* k_cache, void* v_cache, int32_t kv_dtype, int64_t page_stride,
                              int64_t row_stride, int64_t head_stride, int32_t num_pages,
                              int32_t page_size, const float* k_scale, const float* v_scale,
                              int32_t* status, hs_stream_t stream) {
    if (tokens < 0 || heads < 0 || kv_heads < 0 || d <= 0 || rot < 0 || rot > d || q_stride < 0 ||
        k_stride < 0 || v_stride < 0 || q_out_stride < 0 || page_stride < 0 || row_stride < 0 ||
        head_stride < 0 || num_pages < 0 || dtype < HS_BF16 || dtype > HS_FP16 ||
        kv_dtype < HS_BF16 || kv_dtype > HS_E4M3)
        return HS_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > kMaxDim || rot % 2 != 0 || (kv_dtype != HS_E4M3 && kv_dtype != dtype) ||
        (kv_dtype != HS_E4M3 && (k_scale != nullptr || v_scale != nullptr)))
        return HS_ERR_UNSUPPORTED;
    if (int64_t(heads) + 2 * int64_t(kv_heads) > 1 << 20) return HS_ERR_CAPACITY;
    const bool has_q = q != nullptr, has_kv = k != nullptr;
    if (tokens == 0 || (!has_q && !has_kv)) return HS_OK;
    if (positions == nullptr || (rot > 0 && turns == nullptr) || (has_q && q_out == nullptr) ||
        has_kv != (v != nullptr) ||
        (has_kv && (slot == nullptr || k_cache == nullptr || v_cache == nullptr || page_size <= 0)))
        return HS_ERR_INVALID_ARG;
    // Rows that are written must not overlap.
    if ((has_q && tokens > 1 && q_out_stride < int64_t(heads) * d) ||
        (has_kv && ((num_pages > 1 && page_stride < d) || (page_size > 1 && row_stride < d) ||
                    (kv_heads > 1 && head_stride < d))))
        return HS_ERR_INVALID_ARG;
    const auto al = [](const void* p, uintptr_t n) {
        return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
    };
    const int64_t per16 = kv_dtype == HS_E4M3 ? 16 : 8;  // cache elements of 16 bytes
    if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(q_out, 16) || q_stride % 8 || k_stride % 8 ||
        v_stride % 8 || q_out_stride % 8 || !al(k_cache, 16) || !al(v_cache, 16) ||
        (has_kv && (page_stride % per16 || row_stride % per16 || head_stride % per16)) ||
        !al(positions, 4) || !al(slot, 4) || !al(turns, 8) || !al(k_scale, 4) || !al(v_scale, 4) ||
        !al(status, 4))
        return HS_ERR_MISALIGNED;
    RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out_stride = q_out_stride;
    a.positions = positions;
    a.slot = has_kv ? slot : nullptr;
    a.turns = reinterpret_cast<const uint64_t*>(turns);
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_stride = page_stride;
    a.row_stride = row_stride;
    a.head_stride = head_stride;
    a.num_slots = has_kv ? int64_t(num_pages) * page_size : 0;
    a.page_size = page_size;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.tokens = tokens;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.d = d;
    a.half = rot / 2;
    a.interleaved = interleaved;
    a.mscale = mscale;
    a.status = status;
    // Other parts of a head than whole vectors go pair by pair.
    const bool vec = d % 16 == 0 && rot % 16 == 0;
    const int threads = tokens <= hs_host::num_sms() ? kManyThreads : kThreads;
    const auto launch = [&](auto type, auto e4m3) {
        using T = decltype(type);
        constexpr bool E = decltype(e4m3)::value;
        return vec ? hs_host::launch_pdl(rope_kernel<T, E, true>, dim3(unsigned(tokens)),
                                         dim3(unsigned(threads)), 0, stream, a)
                   : hs_host::launch_pdl(rope_kernel<T, E, false>, dim3(unsigned(tokens)),
                                         dim3(unsigned(threads)), 0, stream, a);
    };
    if (kv_dtype == HS_E4M3)
        return dtype == HS_FP16 ? launch(__half{}, std::true_type{})
                                : launch(__nv_bfloat16{}, std::true_type{});
    return dtype == HS_FP16 ? launch(__half{}, std::false_type{})
                            : launch(__nv_bfloat16{}, std::false_type{});
}
