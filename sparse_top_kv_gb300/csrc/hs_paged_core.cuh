// hs_paged_core.cuh -- the warp-level attention kernel of hs_paged_decode for
// one cache type (included by one translation unit per type): small calls of
// few requests, and caches that tensor maps or the tcgen05 kernel do not take
// (pages that are no multiple of 16 tokens, broadcast strides, E4M3 heads of
// 64).  Bound by latency in small calls (one request of 1 K tokens, 32/8 heads
// of 128: 8.5 us with the merge), by HBM in large ones (64 requests of 8 K in
// pages of 12: 321 us, 6.7 TB/s).
//
// Math, per request and query head h of KV head g, over the visible tokens:
//   x_t = scale * k_scale_g * (q_h . K_t),  m = max_t x_t,
//   l = sum_t 2^((x_t - m) log2 e),  out_h = v_scale_g / l * sum_t 2^(..) V_t,
// as running (m, l, sum) states, exact under merging (the split-KV rule of
// hs_merge_states).
//
// A warp owns one KV head of its unit and streams every ts-th block of 16
// tokens through a private ring of cp.async stages (16-byte chunks, XOR-
// swizzled so that ldmatrix meets no bank conflict); tokens outside the
// context or on a bad page are zero-filled without being read and get weight
// 0, so what stands there (NaN included) never matters.  The query heads of
// the KV head are the M dimension of warp-level MMAs: S = Q K^T, whose
// accumulators are in place the A fragment of O += P V.  P is carried as a
// rounded part and the rounding's remainder, so the weights keep twice the
// operand's precision: up to 8 query heads leave rows 8..15 of the fragment
// free and the remainder rides there at no cost; 9..16 heads take a second
// product.  fp16 weights are scaled by 2^15, so that they lose 2^-40 of the
// largest and not 2^-25 (a remainder in rows of its own by 2^12 more: 2^-52);
// bf16 has fp32's exponents.  E4M3 codes are widened exactly to fp16 (the
// query row is scaled by a power of two into fp16's range, undone on the
// logits).
#pragma once

#include "hs_paged.cuh"

namespace hs_paged {
namespace core {

// Places per CTA from which units take several heads.  us with one head / several:
// 64 requests of 2 K tokens (27 places) 89.3 / 94.2, one of 128 K 86.8 / 91.8, 64
// of 32 K (430 places) 1269 / 1227; E4M3 heads of 64, 64 requests of 4 K (64
// places) 108 / 92.
constexpr int kTilesForWide = 64;
// Places that a unit's start and end count for (us at 0 / 1 / 4: eight requests
// of 1 K tokens 16.4 / 15.1 / 15.9, 64 of 510 38.7 / 35.5 / 37.4).
constexpr int kExtra = 1;

enum Kind { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };

template <int KV, int D, int GH_>
struct Cfg {
    static constexpr int GH = GH_;            // fragment halves in use by heads
    static constexpr int GM = 8 * GH_;        // query heads of a unit per KV head
    static constexpr int kElt = KV == kE4m3 ? 1 : 2;
    static constexpr int kRow = D * kElt;     // bytes of one K (or V) row
    static constexpr int kTile = kKey * kRow;
    static constexpr int kStage = 2 * kTile;
    static constexpr int kWarps = kStage >= 16384 ? 4 : 8;
    // Ring stages: as many as about 192 KB hold, at most 8.
    static constexpr int kFit = 196608 / (kWarps * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kThreads = kWarps * 32;
    static constexpr size_t kRing = size_t(kWarps) * kStages * kStage;
    static constexpr size_t kRed = size_t(kWarps) * GM * (D + 2) * sizeof(float);
    static constexpr size_t kBody = kRing > kRed ? kRing : kRed;
    static constexpr int kChunks = kRow / 16;          // 16-byte chunks of a row
    static constexpr int kRowsPerCopy = 32 / kChunks;  // rows of one warp-wide copy
    static constexpr int kCopies = kKey / kRowsPerCopy;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// m16n8k16, fp32 accumulators.  Fragment ownership, g = lane / 4, t = lane %
// 4: A a0 = (g, 2t..), a1 = (g + 8, 2t..), a2 = (g, 2t + 8..), a3 = (g + 8,
// 2t + 8..); B b0 = (2t.., g), b1 = (2t + 8.., g); C c0, c1 = (g, 2t..),
// c2, c3 = (g + 8, 2t..).
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&d)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&d)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm2t(uint32_t addr, uint32_t (&d)[2]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(d[0]), "=r"(d[1])
                 : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

// Two E4M3 codes (low 16 bits) -> two fp16 values, exact (NaN stays NaN).
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    const __half2 h = __half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3));
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if constexpr (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
template <bool BF>
__device__ __forceinline__ float2 unpack(uint32_t u) {
    if constexpr (BF) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Byte offset of 16-byte chunk `c` of token row `key` in a tile: rows of 128
// bytes and more permute their chunks by the row so that 8 rows of one column
// (ldmatrix), or two rows of four columns (E4M3 K), meet distinct banks.
template <int ROW>
__device__ __forceinline__ uint32_t at(int key, int c) {
    if constexpr (ROW >= 128) return uint32_t(key * ROW + ((c ^ (key & 7)) * 16));
    else return uint32_t(key * ROW + ((c ^ ((key >> 1) & 3)) * 16));  // 64-byte rows
}

template <int KV, int D, int GH>
__global__ void __launch_bounds__(Cfg<KV, D, GH>::kThreads, 1)
paged_kernel(const __grid_constant__ PagedArgs a) {
    using C = Cfg<KV, D, GH>;
    constexpr bool BF = KV == kBf16;
    constexpr int NW = C::kWarps, S = C::kStages, GM = C::GM;
    constexpr int NT = D / 8;
    // Scales of the weights' two parts (the second's relative to the first's).
    constexpr float kP = BF ? 1.f : 32768.f, kLo = BF || GH == 2 ? 1.f : 4096.f;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char* body = smem;                                      // ring / reduction
    uint32_t* live_s = reinterpret_cast<uint32_t*>(smem + C::kBody);  // [NW][S]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;

    hs::pdl_wait();
    hs::pdl_trigger();

    const int group = a.heads / a.kv_heads;
    const int gch = (group + GM - 1) / GM;
    const int cta = blockIdx.x;
    const Run rn = make_run(a, cta);
    if (cta == 0) report_lengths(a);
    if (rn.run <= 0) return;
    const int way = rn.way, lth = a.lth[way];
    const int hsn = a.hs[way], ts = NW / hsn;
    const int hl = warp % hsn, tg = warp / hsn;
    const uint32_t ring = hs::smem_u32(body) + uint32_t(warp) * (S * C::kStage);
    uint32_t* live_w = live_s + warp * S;
    const int cc = lane % C::kChunks, cr = lane / C::kChunks;
    const int mi = lane >> 3, r8 = lane & 7;
    bool bad = false;

    Cursor c = cursor_at(a, rn);
    for (bool begin = true; c.left > 0; begin = false) {
        // ---- One segment: the tiles of one unit in this run ----------------
        const int row = c.row;
        const Tiling vis = c.v;
        const int tile0 = c.tile, steps = min(c.left, vis.n - tile0);
        const bool whole = steps == vis.n;
        const int slot = 2 * cta + (tile0 == 0 && !begin ? 1 : 0);
        const int kvh0 = c.chunk / gch * hsn, gc = c.chunk % gch;
        const int kvh = kvh0 + hl;
        const int Gc = min(GM, group - gc * GM);
        const int h0 = kvh * group + gc * GM;

        // ---- Query fragments ---------------------------------------------
        uint32_t qa[D / 16][2 * GH];
        float qs[GH];  // factor of the row's logits, log2 units
        {
            const float ksc = a.k_scale != nullptr ? a.k_scale[kvh] : 1.f;
#pragma unroll
            for (int hh = 0; hh < GH; ++hh) {
                const int hr = g + 8 * hh;
                const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                                     int64_t(row) * a.q_stride +
                                     int64_t(h0 + min(hr, Gc - 1)) * D;
                qs[hh] = a.scale_log2 * ksc;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    // 16-bit caches: dims 2t, 2t+1 and 2t+8, 2t+9 of the block
                    // of 16; E4M3: the permutation that its 16-byte loads of K
                    // meet (below), the same on both sides of the product.
                    if constexpr (KV != kE4m3) {
                        const uint32_t* p = reinterpret_cast<const uint32_t*>(qp + ks * 16);
                        qa[ks][hh] = hr < Gc ? p[t] : 0u;
                        qa[ks][GH + hh] = hr < Gc ? p[4 + t] : 0u;
                    } else {
                        const int d0 = (ks >> 2) * 64 + t * 16 + (ks & 3) * 4;
                        const uint2 u = hr < Gc ? *reinterpret_cast<const uint2*>(qp + d0)
                                                : make_uint2(0u, 0u);
                        qa[ks][hh] = u.x;
                        qa[ks][GH + hh] = u.y;
                    }
                }
                if constexpr (KV == kE4m3) {
                    if (!a.q_is_half) {
                        // bf16 query: bring the row's largest magnitude to
                        // [2^13, 2^14) and round to fp16.  An element 2^-27 of
                        // the largest still has its 8 bits; smaller ones lose
                        // at most 2^-39 of it.
                        float mx = 0.f;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float2 f = unpack<true>(qa[ks][GH * j + hh]);
                                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
                            }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        int e = 0;
                        if (mx > 0.f && mx < CUDART_INF_F) e = 13 - ilogbf(mx);
                        e = min(max(e, -120), 120);
                        const float up = exp2f(float(e));
                        qs[hh] *= exp2f(float(-e));
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float2 f = unpack<true>(qa[ks][GH * j + hh]);
                                qa[ks][GH * j + hh] = pack<false>(f.x * up, f.y * up);
                            }
                    }
                }
            }
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m[GH], l[GH];
#pragma unroll
        for (int hh = 0; hh < GH; ++hh) {
            m[hh] = -CUDART_INF_F;
            l[hh] = 0.f;
        }

        // ---- Stream the tokens --------------------------------------------
        const int32_t* table = a.block_table + int64_t(row) * a.bt_stride;
        const char* kb = static_cast<const char*>(a.k) + int64_t(kvh) * a.head_stride * C::kElt;
        const char* vb = static_cast<const char*>(a.v) + int64_t(kvh) * a.head_stride * C::kElt;
        // Lane l < 16 looks up token l of a step: its page one step before it
        // is needed.
        auto block_token = [&](int j) {  // first token of this warp's block of a step
            Cursor x = c;
            x.tile = tile0 + j;
            return tile_token(x, lth) + tg * kKey;
        };
        auto token = [&](int j) {  // -1: not attended to
            const int tok = block_token(j) + (lane & 15);
            return j < steps && visible(vis, tok) ? tok : -1;
        };
        int tok_n = token(0);
        int page_n = tok_n >= 0 ? table[block_of(a, tok_n)] : -1;
        auto issue = [&](int j) {
            const int tok = tok_n;
            int page = page_n;
            tok_n = token(j + 1);
            page_n = tok_n >= 0 ? table[block_of(a, tok_n)] : -1;
            if (page >= a.num_pages || (tok >= 0 && page < 0)) bad = true;
            const bool ok = tok >= 0 && page >= 0 && page < a.num_pages;
            const int64_t off =
                ok ? (int64_t(page) * a.page_stride + int64_t(tok - block_of(a, tok) * a.page_size) * a.row_stride) *
                         C::kElt
                   : -1;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            if (lane == 0) live_w[j % S] = mask;
            const uint32_t st = ring + uint32_t(j % S) * C::kStage;
#pragma unroll
            for (int i = 0; i < C::kCopies; ++i) {
                const int key = i * C::kRowsPerCopy + cr;
                const int64_t ko = __shfl_sync(0xffffffffu, off, key);
                const uint32_t nb = ko >= 0 ? 16u : 0u;
                const int64_t src = ko >= 0 ? ko + cc * 16 : 0;
                const uint32_t dst = st + at<C::kRow>(key, cc);
                cp16(dst, kb + src, nb);
                cp16(dst + C::kTile, vb + src, nb);
            }
        };
#pragma unroll
        for (int j = 0; j < S - 1; ++j) {
            if (j < steps) issue(j);
            cp_commit();
        }
        for (int j = 0; j < steps; ++j) {
            if (j + S - 1 < steps) issue(j + S - 1);
            cp_commit();
            cp_wait<S - 1>();
            __syncwarp();
            const uint32_t kt = ring + uint32_t(j % S) * C::kStage;
            const uint32_t vt = kt + C::kTile;
            const uint32_t mask = live_w[j % S];

            // S = Q K^T: n-tile 0 = tokens 0..7, n-tile 1 = tokens 8..15.
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (KV != kE4m3) {
                const int key = r8 + (mi >> 1) * 8;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t b[4];
                    ldsm4(kt + at<C::kRow>(key, 2 * ks + (mi & 1)), b);
                    const uint32_t a1 = GH == 2 ? qa[ks][1] : 0u;
                    const uint32_t a3 = GH == 2 ? qa[ks][2 * GH - 1] : 0u;
                    mma<BF>(s0, qa[ks][0], a1, qa[ks][GH], a3, b[0], b[1]);
                    mma<BF>(s1, qa[ks][0], a1, qa[ks][GH], a3, b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int kb4 = 0; kb4 < D / 64; ++kb4) {
                    const uint4 x0 = lds128(kt + at<C::kRow>(g, kb4 * 4 + t));
                    const uint4 x1 = lds128(kt + at<C::kRow>(g + 8, kb4 * 4 + t));
                    const uint32_t y0[4] = {x0.x, x0.y, x0.z, x0.w};
                    const uint32_t y1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int ks = kb4 * 4 + u;
                        const uint32_t a1 = GH == 2 ? qa[ks][1] : 0u;
                        const uint32_t a3 = GH == 2 ? qa[ks][2 * GH - 1] : 0u;
                        mma<BF>(s0, qa[ks][0], a1, qa[ks][GH], a3, widen(y0[u]),
                                widen(y0[u] >> 16));
                        mma<BF>(s1, qa[ks][0], a1, qa[ks][GH], a3, widen(y1[u]),
                                widen(y1[u] >> 16));
                    }
                }
            }

            // Running softmax of head rows g (and g + 8) over this lane's
            // four tokens 2t, 2t + 1, 2t + 8, 2t + 9.
            uint32_t ph[GH][2], plo[GH][2];  // [.][0] tokens 2t.., [1] 2t + 8..
            float alpha[GH];
            bool grow = false;
#pragma unroll
            for (int hh = 0; hh < GH; ++hh) {
                float x[4] = {s0[2 * hh], s0[2 * hh + 1], s1[2 * hh], s1[2 * hh + 1]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i >> 1) * 8 + 2 * t + (i & 1);
                    x[i] = (mask >> key) & 1u ? x[i] * qs[hh] : -CUDART_INF_F;
                }
                if (a.logits != nullptr && g + 8 * hh < Gc) {
                    float* lp = a.logits +
                                (int64_t(row) * a.heads + h0 + g + 8 * hh) * a.logit_stride;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = block_token(j) + (i >> 1) * 8 + 2 * t + (i & 1);
                        if (visible(vis, tok)) lp[visible_index(vis, tok)] = x[i];
                    }
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[hh], mx);
                // No finite logit yet: subtract 0, every weight stays 0 (a NaN
                // logit stays NaN).
                const float ref = mn == -CUDART_INF_F ? 0.f : mn;
                alpha[hh] = m[hh] == mn ? 1.f : exp2f(m[hh] - ref);
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = exp2f(x[i] - ref);
                l[hh] = l[hh] * alpha[hh] + ((p[0] + p[1]) + (p[2] + p[3]));
                m[hh] = mn;
                grow |= alpha[hh] != 1.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x0 = p[2 * i] * kP, x1 = p[2 * i + 1] * kP;
                    ph[hh][i] = pack<BF>(x0, x1);
                    const float2 f = unpack<BF>(ph[hh][i]);
                    plo[hh][i] = pack<BF>((x0 - f.x) * kLo, (x1 - f.y) * kLo);
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
                // Rows 8..15: the second half of the heads, or (GH = 1) the
                // remainders of the same heads.
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= alpha[0];
                    o[n][1] *= alpha[0];
                    o[n][2] *= alpha[GH - 1];
                    o[n][3] *= alpha[GH - 1];
                }
            }
            auto pv = [&](float (&c)[4], uint32_t b0, uint32_t b1) {
                if constexpr (GH == 1) {
                    mma<BF>(c, ph[0][0], plo[0][0], ph[0][1], plo[0][1], b0, b1);
                } else {
                    mma<BF>(c, ph[0][0], ph[GH - 1][0], ph[0][1], ph[GH - 1][1], b0, b1);
                    mma<BF>(c, plo[0][0], plo[GH - 1][0], plo[0][1], plo[GH - 1][1], b0, b1);
                }
            };
            // O += P V.
            if constexpr (KV != kE4m3) {
                const int key = r8 + (mi & 1) * 8;
#pragma unroll
                for (int np = 0; np < D / 16; ++np) {
                    uint32_t b[4];
                    ldsm4t(vt + at<C::kRow>(key, 2 * np + (mi >> 1)), b);
                    pv(o[2 * np], b[0], b[1]);
                    pv(o[2 * np + 1], b[2], b[3]);
                }
            } else {
                // A transposed 8 x 8 matrix of 16-bit units: lane (g, t) gets
                // dims 2g, 2g + 1 of tokens 2t, 2t + 1 (bytes d0 d1 of the
                // first, then of the second).  Even dims make one n-tile, odd
                // dims the next.
                const int key = r8 + (mi & 1) * 8;
#pragma unroll
                for (int np = 0; np < D / 32; ++np) {
                    uint32_t b[4];
                    ldsm4t(vt + at<C::kRow>(key, 2 * np + (mi >> 1)), b);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t e0 = widen(__byte_perm(b[2 * u], 0u, 0x4420));
                        const uint32_t e1 = widen(__byte_perm(b[2 * u + 1], 0u, 0x4420));
                        const uint32_t f0 = widen(__byte_perm(b[2 * u], 0u, 0x4431));
                        const uint32_t f1 = widen(__byte_perm(b[2 * u + 1], 0u, 0x4431));
                        pv(o[4 * np + 2 * u], e0, e1);
                        pv(o[4 * np + 2 * u + 1], f0, f1);
                    }
                }
            }
            __syncwarp();  // every lane's reads of this stage precede its refill
        }
        cp_wait<0>();

        // ---- Merge the ts warps of each KV head, write the unit's state -----
#pragma unroll
        for (int hh = 0; hh < GH; ++hh) {
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
        }
        __syncthreads();  // the ring becomes the reduction's buffer
        float* so = reinterpret_cast<float*>(body);  // [NW][GM][D]
        float* sml = so + NW * GM * D;               // [NW][GM][2]
        // A head's sum from its two rows of a fragment, or its one.
        auto sum = [&](const float (&c)[4], int hh, int j) {
            return (GH == 1 ? fmaf(c[2 + j], 1.f / kLo, c[j]) : c[2 * hh + j]) * (1.f / kP);
        };
#pragma unroll
        for (int hh = 0; hh < GH; ++hh) {
            if (g + 8 * hh < Gc) {
                float* dst = so + (warp * GM + g + 8 * hh) * D;
                if constexpr (KV != kE4m3) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        *reinterpret_cast<float2*>(dst + n * 8 + 2 * t) =
                            make_float2(sum(o[n], hh, 0), sum(o[n], hh, 1));
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        *reinterpret_cast<float4*>(dst + n * 8 + 4 * t) =
                            make_float4(sum(o[n], hh, 0), sum(o[n + 1], hh, 0),
                                        sum(o[n], hh, 1), sum(o[n + 1], hh, 1));
                    }
                }
                if (t == 0) {
                    sml[(warp * GM + g + 8 * hh) * 2] = m[hh];
                    sml[(warp * GM + g + 8 * hh) * 2 + 1] = l[hh];
                }
            }
        }
        __syncthreads();
        for (int e = tid; e < hsn * Gc * D; e += C::kThreads) {
            const int d = e % D, hg = (e / D) % Gc, hk = e / (D * Gc);
            float M = -CUDART_INF_F;
            for (int q = 0; q < ts; ++q) M = fmaxf(M, sml[((q * hsn + hk) * GM + hg) * 2]);
            const float ref = M == -CUDART_INF_F ? 0.f : M;
            float L = 0.f, O = 0.f;
            for (int q = 0; q < ts; ++q) {
                const int s = (q * hsn + hk) * GM + hg;
                const float f = exp2f(sml[2 * s] - ref);
                L = fmaf(f, sml[2 * s + 1], L);
                O = fmaf(f, so[s * D + d], O);
            }
            const int kv = kvh0 + hk;
            if (whole) {
                const int64_t qh = int64_t(row) * a.heads + kv * group + gc * GM + hg;
                float r = L == 0.f ? 0.f : O / L;
                if (a.v_scale != nullptr && L != 0.f) r *= a.v_scale[kv];
                const bool bf = KV == kBf16 || (KV == kE4m3 && !a.q_is_half);
                if (bf) static_cast<__nv_bfloat16*>(a.out)[qh * D + d] = __float2bfloat16_rn(r);
                else static_cast<__half*>(a.out)[qh * D + d] = __float2half_rn(r);
                if (d == 0) {
                    const float lg = L == 0.f ? -CUDART_INF_F : M + log2f(L);
                    if (a.lse != nullptr) a.lse[qh] = lg * kLn2;
                    if (a.lse2 != nullptr) a.lse2[qh] = lg;
                }
            } else {
                const int64_t s = int64_t(slot) * a.unit_heads_max + hk * GM + hg;
                a.part_o[s * D + d] = O;
                if (d == 0) {
                    a.part_ml[2 * s] = M;
                    a.part_ml[2 * s + 1] = L;
                }
            }
        }
        __syncthreads();  // the reduction's buffer becomes the next unit's ring
        next_segment(c, a, rn.chunks, lth);
    }
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
}

template <int KV, int D, int GH>
int launch_one(PagedArgs& a, hs_stream_t stream) {
    using C = Cfg<KV, D, GH>;
    auto kern = paged_kernel<KV, D, GH>;
    set_ways(a, C::kWarps, C::kWarps * kKey, C::GM, kTilesForWide, kExtra);
    constexpr size_t smem = C::kBody + C::kWarps * C::kStages * 4;
    static int smem_set[64] = {};
    const int rc =
        hs_host::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem, smem_set);
    if (rc != HS_OK) return rc;
    return hs_host::launch_pdl(kern, dim3(a.ctas), dim3(C::kThreads), smem, stream, a);
}

template <int KV>
int launch_kind(PagedArgs& a, int d, int group, hs_stream_t stream) {
    if (group <= 8) {
        if (d == 64) return launch_one<KV, 64, 1>(a, stream);
        if (d == 128) return launch_one<KV, 128, 1>(a, stream);
        return launch_one<KV, 256, 1>(a, stream);
    }
    if (d == 64) return launch_one<KV, 64, 2>(a, stream);
    if (d == 128) return launch_one<KV, 128, 2>(a, stream);
    return launch_one<KV, 256, 2>(a, stream);
}

}  // namespace core
}  // namespace hs_paged
