// hs_paged_tc.cuh -- the attention kernel of hs_paged_decode on the 5th-
// generation tensor cores, fed by TMA (included by one translation unit per
// cache type; pages of a multiple of 16 tokens, rows of 128 bytes and more).
//
// Math, per request and query head h of KV head g, over the visible tokens:
//   x_t = scale * k_scale_g * (q_h . K_t),  p_t = 2^((x_t - m) log2 e),
//   l = sum p_t,  out_h = v_scale_g / l * sum p_t V_t,
// as (m, l, sum) states, exact under merging (the rule of hs_merge_states).
//
// The operator reads every cached byte once and does 4 * (query heads per KV
// head) flops with an element, so HBM bounds it; everything here serves to
// keep TMA loads in flight without a pause.
//  * A tile is 128 cache rows: hs KV heads x 128 / hs tokens, so that one TMA
//    box takes all heads of a run of tokens and DRAM is read in long pieces
//    (one head's row at a time: 351 instead of 336 us over a bf16 batch of up
//    to 64 K tokens, 122 instead of 88 over E4M3 rows of 128 bytes, both
//    before their weights had six parts).  Rows of
//    a tile: [run of bt tokens][head][token of the run], so that a K step of
//    PV holds one head (E4M3 pages of 16: a box per head, [head][token]).
//  * One elected lane per run issues the boxes into a K ring and a V ring in
//    128-byte-swizzled blocks; the loads run ahead over the ends of units.
//  * S^T[128 rows x queries] = K Q^T takes the queries of all hs heads as N;
//    only the entries where the row's head is the query's own are used.  The
//    rest is wasted work that the tensor cores have to spare.
//  * Softmax: one thread per row, against a reference maximum that moves only
//    when a logit exceeds it by 2^8 (a vote), so the common tile needs no
//    reduction; exponent sums stay per thread until the unit ends.  A tile's
//    softmax is one chain of dependent steps (0.6 us, E4M3 0.75 us, as long as
//    the tile's loads), so two groups of four warps take the tiles in turn,
//    each with its own maximum, sums and output accumulators, joined when the
//    unit ends.
//  * QK and PV are issued by a warp each: one thread issuing both was the
//    bound at first (16 products a tile at 80 to 100 cycles each).
//  * O^T[D x queries] += V^T P^T, V as an MN-major view of its tile, K = the
//    16 (E4M3: 32) rows of one head, one accumulator per head.  P is carried
//    as several parts in columns of their own: two bf16 or fp16 ones, six E4M3
//    ones, scaled so that small weights keep their bits too (Cfg::up): behind
//    an attention sink without a value they are all of the output.
//  * E4M3 caches are multiplied as they are (kind::f8f6f4): the query, scaled
//    by a power of two, becomes several E4M3 parts (each the rounding of 16
//    times the remainder before it: two hold the 8 bits of a bf16 query,
//    three the 11 of an fp16 one, down to about 2^-14 and 2^-15 of its row's
//    largest element; smaller ones are off by 2^-22 and 2^-26 of that); each
//    part has columns of its own and the parts are summed in fp32 with their
//    weights 16^-i.
// Every wait is bounded (HS_ERR_TIMEOUT in the status word on expiry).
#pragma once

#include <cuda.h>

#include "hs_paged.cuh"
#include "hs_pair.cuh"
#include "hs_shared.h"
#include "hs_tcgen05.cuh"

namespace hs_paged {
namespace tc {

enum Kind { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };

constexpr int kRows = 128;           // cache rows of a tile = M of the QK product
constexpr int kBlk = kRows * 128;    // one block: 128 rows x 128 bytes
constexpr int kSoftThreads = 128;    // one softmax group: a thread per row
constexpr int kGroups = 2;
constexpr int kTmaWarp = 8, kQkWarp = 9, kPvWarp = 10, kQWarp = 11;
constexpr int kThreads = 384;
constexpr int kSoftBar = 1;          // named barriers of the groups: 1, 2
constexpr int kBothBar = 3;          // and of both
constexpr int kMaskRing = 16;        // tiles whose loaded runs are remembered
constexpr float kThresh = 8.f;       // log2 headroom before O is rescaled
constexpr int kTmemCols = 512;
constexpr int kBarBytes = 5120;      // shared-memory budget of Bars
// Places per CTA from which the units of a deal take several heads (the
// shorter calls here are dealt where their bound on the lengths is long).  32/8 heads of 128, bf16,
// us with all heads / one head to a unit: one request of 1 K tokens 10.8 / 10.8,
// 4 K 14.2 / 12.8, 16 K 18.1 / 20.0, eight of 1 K 14.6 / 16.8, of 2 K 17.1 /
// 21.7, 32 of 512 17.9 / 23.3.
constexpr int kTilesForWide = 2;
// A long 16-bit context or two alone on the GPU is cut by single heads again:
// the 256-byte pieces of a head cost little there, and a head's merge joins a
// few parts instead of 152 (us, all heads / one: 24 K tokens 25.8 / 26.5, 32 K
// 34.6 / 31.1, 128 K 93.1 / 90.2, two of 32 K 52.5 / 51.4, four 90.7 / 91.3).
// E4M3 heads are 128-byte pieces: never (64 requests of up to 8 K 88 / 122, with
// four parts to a weight).
constexpr int kWideAlone = 2;        // requests x chunks of heads
constexpr int kTilesAlone = 12;      // places per CTA

constexpr int kMaxCluster = 8;  // the largest portable cluster
constexpr int kMaxUnit = 64;    // queries of a unit

__device__ __forceinline__ float2 peer_load2(uint32_t addr, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(hs::pair::mapa(addr, uint32_t(rank)))
                 : "memory");
    return v;
}

// Tiles of a CTA whose cluster takes a unit, at most, and their bytes.
constexpr int kTilesOfUnit = 8;
constexpr int kUnitBytes = 512 * 1024;

struct TcArgs {
    PagedArgs p;
    int32_t bt[2];     // tokens of a run (a box): they lie in one page
    int32_t split[2];  // runs shorter than a K step of PV: one box per head
    uint64_t timeout_ns;
};

// QP: E4M3 parts of the query.
template <int KV, int D, int GH, int QP>
struct Cfg {
    static constexpr bool kE4 = KV == kE4m3;
    static constexpr int GM = 8 * GH;                    // query heads per KV head and unit
    static constexpr int kElt = kE4 ? 1 : 2;
    static constexpr int kBlkDims = 128 / kElt;          // dims of a block
    static constexpr int kBlocks = D / kBlkDims;         // blocks of a K (or V) tile
    static constexpr int kSubBlocks = kE4 ? 1 : (kBlocks < 2 ? 1 : 2);  // 128 dims of V
    static constexpr int kSub = kSubBlocks * kBlk;       // one ring unit
    static constexpr int kSubs = kBlocks / kSubBlocks;   // ring units of a tile
    static constexpr int kQParts = kE4 ? QP : 1;
    static constexpr int kQBufs = kE4 ? 2 : 1;  // the E4M3 parts take time to make
    static constexpr int kPParts = kE4 ? 6 : 2;
    // Weights p <= 2^kThresh are carried as parts c_i of the operand's type, p =
    // sum c_i / s_i: each the rounding of s_i times what the parts before it leave,
    // with s_0 = up(-1) and s_(i+1) = s_i up(i).
    //  bf16: has fp32's exponents; two parts keep p to 2^-17.
    //  fp16: s_0 brings the largest p to 2^15, the remainder has a scale of its
    //    own: p to 2^-23, and to 2^-44 in all (below 2^-25 without the scales).
    //  E4M3: 4 bits and a sign each, so s_i grows by 2^5: the first four keep p
    //    >= 2^-6 to 2^-19 and leave 2^-25 of smaller ones.  The last two start
    //    there (large weights' remainders saturate in them, which does no harm):
    //    p to 2^-35, or 2^-10 of itself below 2^-25, down to 2^-48.  (64 requests
    //    of up to 8 K tokens: 90.4 us, 89.0 with four parts 2^4 apart, which lose
    //    p < 2^-22.)
    static constexpr float up(int i) {
        return kE4 ? (i < 0 ? 1.f : i == 3 ? 262144.f : 32.f)
                   : KV == kFp16 ? (i < 0 ? 128.f : 4096.f) : 1.f;
    }
    static constexpr int NH = GM * kQParts;              // query columns of a head
    static constexpr int NP = GM * kPParts;              // output columns of a head
    static constexpr int kStep = 32 / kElt;              // rows of a PV K step
    static constexpr int kPBytes = NP * kRows * kElt;    // P^T: rows of 64 (E4M3: 128) cache rows
    // Most heads of a tile: as many as leave the accumulators within TMEM and
    // at least three units in each ring.
    static constexpr int q_rows(int hs) { return hs * NH < 16 ? 16 : (hs * NH + 15) / 16 * 16; }
    static constexpr int cols(int hs) { return 2 * q_rows(hs) + kGroups * kSubs * hs * NP; }
    static constexpr int units(int hs) {
        return (227 * 1024 - 1024 - kBarBytes - kQBufs * q_rows(hs) * D * kElt - 2 * kPBytes) /
               (2 * kSub);
    }
    static constexpr bool fits(int hs) { return cols(hs) <= kTmemCols && units(hs) >= 3; }
    static constexpr int kHsMax = fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1;
    static_assert(fits(kHsMax), "TMEM columns and ring units");
    static constexpr int kQBytes = q_rows(kHsMax) * D * kElt;
    static constexpr int kFit = units(kHsMax);
    static constexpr int NS = kFit > 8 ? 8 : kFit;       // units of each ring
    // A unit's start and end in tiles: 2.6 us at an SM's share of the bandwidth.
    static constexpr int kExtra = 2 * kSubs * kSub > 98304 ? 1 : 131072 / (2 * kSubs * kSub);
    static constexpr int kKOff = 0;
    static constexpr int kVOff = kKOff + NS * kSub;
    static constexpr int kQOff = kVOff + NS * kSub;
    static constexpr int kPOff = kQOff + kQBufs * kQBytes;
    static constexpr int kBarOff = kPOff + 2 * kPBytes;
    static_assert(kHsMax * GM <= kMaxUnit && kHsMax * GM * D * 4 <= kQOff, "a cluster's parts");
};

struct Bars {
    uint64_t kfull[8], kempty[8], vfull[8], vempty[8];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t q_full[2], q_empty, o_free, drain[2];
    uint32_t tmem_base;
    volatile int32_t abort;
    float2 join_ml[kMaxUnit];           // [head, query] the cluster's CTAs read each other's
    uint32_t loaded[kMaskRing];         // runs of a tile that were loaded
    alignas(16) float red[kGroups][8][16];  // per 16 rows: maxima or sums
    // By head * GM + query:
    float alpha[kGroups][kMaxUnit];     // rescale factors
    float m[kGroups][kMaxUnit];         // epilogue: the groups' references
    float weight[kGroups][kMaxUnit];    // and their factors of the output
    float qscale[4][kMaxUnit];          // E4M3: factor of each query's logits, by segment
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

// 4-D tensor map coordinates: dim, token of the page, KV head, page.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int tok,
                                         int head, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(tok), "r"(head), "r"(page), "r"(hs::smem_u32(bar))
        : "memory");
}

// Whether the phase with `parity` has completed (no wait).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(hs::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

template <int KV>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t acc) {
    if constexpr (KV == kE4m3)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        hs::tc::mma_bf16(d, a, b, idesc, acc);
}

// Instruction descriptor: fp32 accumulators; types by kind (bf16 1, fp16 0,
// E4M3 0); B K-major.
template <int KV>
__device__ __forceinline__ uint32_t idesc(int N, int a_mn_major) {
    const uint32_t fmt = KV == kBf16 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (uint32_t(a_mn_major) << 15) |
           (uint32_t(N >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
    if constexpr (N == 8) {
        hs::tc::tmem_ld8(addr, v);
    } else if constexpr (N % 16 == 0) {
#pragma unroll
        for (int c = 0; c < N; c += 16) {
            float t[16];
            hs::tc::tmem_ld16(addr + c, t);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[c + i] = t[i];
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 8) {
            float t[8];
            hs::tc::tmem_ld8(addr + c, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c + i] = t[i];
        }
    }
}

// Two fp32 values to E4M3 codes (the first in the low byte) and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    return __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// 2^x (PTX ex2.approx.ftz: within 2 ulp; 0 below -126, where a weight no
// longer counts against the sum's 1).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// E4M3 parts of the queries of a segment: step `it` makes 512 / D rows (head
// hl, query gi) of the unit, a lane 16 dims of one.  A function of its own, so
// that its two callers share the instructions.
template <int D, int GH, int QP>
__device__ __noinline__ void query_parts(const PagedArgs& a, Bars& B, unsigned char* qbuf, int nq,
                                         int hsn, int row, int chunk, int seg, int it) {
    constexpr int GM = 8 * GH, NH = GM * QP, kL = D / 16;
    const int lane = threadIdx.x & 31;
    const int group = a.heads / a.kv_heads, gch = (group + GM - 1) / GM;
    const int kvh0 = chunk / gch * hsn, gc = chunk % gch;
    const int Gc = min(GM, group - gc * GM);
    const int ch = lane % kL, n = it * (32 / kL) + lane / kL, hl = n / GM, gi = n % GM;
    uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (gi < Gc) {
        const uint4* p = reinterpret_cast<const uint4*>(
            static_cast<const char*>(a.q) +
            (int64_t(row) * a.q_stride + int64_t((kvh0 + hl) * group + gc * GM + gi) * D +
             ch * 16) * 2);
        raw[0] = *p;
        raw[1] = p[1];
    }
    float x[16];
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                           raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = QP == 3 ? __half22float2(*reinterpret_cast<const __half2*>(&w[i]))
                                 : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    float mx = 0.f;
    bool odd = false;  // not finite: shows as NaN
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        mx = fmaxf(mx, fabsf(x[i]));
        odd |= !(fabsf(x[i]) < CUDART_INF_F);
    }
#pragma unroll
    for (int o = kL / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // Largest magnitude to [2^7, 2^8), by two factors (their product may lie
    // outside fp32's range).
    int e = 0;
    if (mx > 0.f && mx < CUDART_INF_F)
        e = max(7 - (int(__float_as_uint(mx) >> 23) - 127), -126);
    const int ea = e / 2, eb = e - ea;
    const float up = pow2(ea), up2 = pow2(eb);
    uint32_t code[QP][4];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float r0 = x[i] * up * up2, r1 = x[i + 1] * up * up2;
#pragma unroll
        for (int k = 0; k < QP; ++k) {
            const uint32_t cc = odd ? 0x7f7fu : to_e4m3x2(r0, r1);
            code[k][i >> 2] = (i & 2) ? code[k][i >> 2] | (cc << 16) : cc;
            if (k + 1 < QP) {
                const float2 f = from_e4m3x2(cc);
                r0 = (r0 - f.x) * 16.f;
                r1 = (r1 - f.y) * 16.f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < QP; ++k) {
        const int m = hl * NH + k * GM + gi;
        *reinterpret_cast<uint4*>(qbuf + (ch >> 3) * nq * 128 + m * 128 +
                                  (((ch & 7) ^ (m & 7)) << 4)) =
            make_uint4(code[k][0], code[k][1], code[k][2], code[k][3]);
    }
    if (ch == 0) {
        float f = a.scale_log2 * pow2(-ea) * pow2(-eb);
        if (a.k_scale != nullptr) f *= a.k_scale[kvh0 + hl];
        B.qscale[seg & 3][hl * GM + gi] = f;
    }
}

template <int KV, int D, int GH, int QP>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ TcArgs ta, const __grid_constant__ CUtensorMap kmap0,
                const __grid_constant__ CUtensorMap vmap0,
                const __grid_constant__ CUtensorMap kmap1,
                const __grid_constant__ CUtensorMap vmap1) {
    using C = Cfg<KV, D, GH, QP>;
    constexpr int GM = C::GM, NS = C::NS;
    constexpr bool E4 = C::kE4;
    const PagedArgs& a = ta.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& B = *reinterpret_cast<Bars*>(smem + C::kBarOff);
    const uint32_t sb = hs::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t tmo = ta.timeout_ns;
    const volatile int* abort_flag = &B.abort;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            hs::mbar_init(&B.kfull[i], 1);
            hs::mbar_init(&B.kempty[i], 1);
            hs::mbar_init(&B.vfull[i], 1);
            hs::mbar_init(&B.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            hs::mbar_init(&B.s_full[i], 1);
            hs::mbar_init(&B.p_full[i], kSoftThreads);
            hs::mbar_init(&B.pv_done[i], 1);
        }
        for (int i = 0; i < C::kQBufs; ++i) {
            hs::mbar_init(&B.q_full[i], E4 ? kGroups * kSoftThreads : 32);
        }
        hs::mbar_init(&B.q_empty, 1);
        hs::mbar_init(&B.o_free, kGroups * kSoftThreads);
        hs::mbar_init(&B.drain[0], 1);
        hs::mbar_init(&B.drain[1], 1);
        B.abort = 0;
        hs::fence_mbar_init();
    }
    if (warp == kTmaWarp && lane < 4) {
        const CUtensorMap* m = lane == 0 ? &kmap0 : lane == 1 ? &vmap0 : lane == 2 ? &kmap1 : &vmap1;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (warp == kPvWarp) {
        hs::tc::tmem_alloc(&B.tmem_base, kTmemCols);
        hs::tc::tmem_relinquish();
    }
    // The rows of queries that a unit does not have stay zero.
    if constexpr (E4) {
        constexpr int kBytes = C::kPOff - C::kQOff;
        for (int i = tid; i < kBytes / 16; i += kThreads)
            reinterpret_cast<uint4*>(smem + C::kQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
        hs::fence_proxy_async_shared();
    }
    hs::tc::fence_before_sync();
    __syncthreads();
    hs::tc::fence_after_sync();
    hs::pdl_wait();
    hs::pdl_trigger();

    const int group = a.heads / a.kv_heads;
    const int gch = (group + GM - 1) / GM;
    const int cta = blockIdx.x;
    const int cl = a.cl, rank = cl > 1 ? int(hs::pair::cta_rank()) : 0;
    const Run rn = cl > 0 ? unit_run(a, cl > 1 ? cta / cl : cta, rank) : make_run(a, cta);
    const int way = rn.way, chunks = rn.chunks, run = rn.run;
    const Cursor start = cursor_at(a, rn);
    if (cta == 0) report_lengths(a);
    const uint32_t tmem = B.tmem_base;
    const int hsn = a.hs[way], bt = ta.bt[way];
    // hs and bt are powers of two.
    const int lhs = 31 - __clz(hsn), lbt = 31 - __clz(bt);
    const int lth = a.lth[way];          // log2 of the tokens of a tile
    const int runs = 1 << (lth - lbt);   // runs of a tile
    const bool split = ta.split[way] != 0;
    const int lrow = split ? lth : lbt;  // log2 of a head's neighbouring rows
    const int nq = max(16, (hsn * C::NH + 15) / 16 * 16);  // N of the QK product
    const uint32_t o_col = uint32_t(2 * nq);
    const int ocols = hsn * C::NP;       // output columns of 128 dims

    if (run <= 0) {
        // Nothing to do: straight to the tear-down.
    } else if (warp == kTmaWarp) {
        // ------------------------------- loads -------------------------------
        const CUtensorMap* kmap = way == 0 ? &kmap0 : &kmap1;
        const CUtensorMap* vmap = way == 0 ? &vmap0 : &vmap1;
        Cursor c = start;
        bool ok = true, bad = false;
        int kseq = 0, vseq = 0, t = 0;
        // Lane i: run i % runs of the tile (and head i / runs, if the boxes are
        // split); its page is looked up a tile ahead.
        const int run_i = lane & (runs - 1), head_i = lane >> (lth - lbt);
        const bool lane_in = head_i < (split ? hsn : 1);
        const uint32_t lane_row =
            split ? uint32_t((head_i << lth) + (run_i << lbt)) : uint32_t(run_i << (lhs + lbt));
        const uint32_t box = uint32_t(split ? bt : hsn * bt) * 128u;  // bytes of a block's box
        auto lookup = [&](const Cursor& x, int& tok) {
            tok = tile_token(x, lth) + (run_i << lbt);
            if (!lane_in || !any_visible(x.v, tok, bt)) return -2;
            return a.block_table[int64_t(x.row) * a.bt_stride + block_of(a, tok)];
        };
        int tok_n, page_n = lookup(c, tok_n);
        for (; ok;) {
            const int tok = tok_n, page = page_n;
            const int head0 = c.chunk / gch * hsn + (split ? head_i : 0);
            const bool more = c.left > 1;
            advance(c, a, chunks, lth);
            if (more) page_n = lookup(c, tok_n);
            const bool want = page >= 0 && page < a.num_pages;
            if (page != -2 && !want) bad = true;
            const uint32_t loaded = __ballot_sync(0xffffffffu, want);
            const uint32_t bytes = uint32_t(__popc(loaded)) * box * C::kSubBlocks;
            const int at = tok - block_of(a, tok) * a.page_size;
            // Read by the softmax of this tile (its logits follow these
            // loads), at most NS + 3 tiles behind.
            if (lane == 0) B.loaded[t % kMaskRing] = loaded;
            ++t;
            auto fill = [&](uint64_t* full, uint64_t* empty, int off, const CUtensorMap* map,
                            int& seq) {
                for (int s = 0; s < C::kSubs; ++s, ++seq) {
                    const int slot = seq % NS;
                    if (!__all_sync(0xffffffffu,
                                    hs::mbar_wait_bounded(&empty[slot], ((seq / NS) & 1) ^ 1, tmo,
                                                          abort_flag)))
                        return false;
                    if (lane == 0) hs::mbar_arrive_expect_tx(&full[slot], bytes);
                    __syncwarp();
                    if (want) {
                        const uint32_t dst = sb + off + slot * C::kSub + lane_row * 128;
#pragma unroll
                        for (int b = 0; b < C::kSubBlocks; ++b)
                            tma_load(dst + b * kBlk, map, (s * C::kSubBlocks + b) * C::kBlkDims,
                                     at, head0, page, &full[slot]);
                    }
                }
                return true;
            };
            ok = fill(B.kfull, B.kempty, C::kKOff, kmap, kseq) &&
                 fill(B.vfull, B.vempty, C::kVOff, vmap, vseq);
            if (!more) break;
        }
        if (!ok) {
            hs::set_status(a.status, HS_ERR_TIMEOUT);
            B.abort = 1;
            // No copy may outlive the CTA: wait for every unit in flight.
            for (int s = max(0, kseq - NS); s < kseq; ++s)
                hs::mbar_wait_bounded(&B.kfull[s % NS], (s / NS) & 1, tmo, nullptr);
            for (int s = max(0, vseq - NS); s < vseq; ++s)
                hs::mbar_wait_bounded(&B.vfull[s % NS], (s / NS) & 1, tmo, nullptr);
        }
        if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    } else if (warp == kQkWarp) {
        // ---------------------------- S^T = K Q^T -----------------------------
        if (lane == 0) {
            const uint32_t id = idesc<KV>(nq, 0);
            // Descriptors of the first tile; others are an offset (in units
            // of 16 bytes) away.
            const uint64_t k_desc = hs::tc::sdesc_sw128(sb + C::kKOff, 16, 1024);
            const uint64_t q_desc = hs::tc::sdesc_sw128(sb + C::kQOff, 16, 1024);
            Cursor c = start;
            bool ok = true;
            int slot = 0, qb = 0;
            uint32_t phase = 0;
            for (int t = 0, seg = 0; t < run; ++t) {
                if (c.first) {
                    qb = seg % C::kQBufs;
                    ok = ok && hs::mbar_wait_bounded(&B.q_full[qb], (seg / C::kQBufs) & 1, tmo,
                                                     abort_flag);
                    ++seg;
                }
                // The softmax of two tiles ago has read this S buffer.
                if (t >= 2)
                    ok = ok && hs::mbar_wait_bounded(&B.p_full[t & 1], ((t - 2) >> 1) & 1, tmo,
                                                     abort_flag);
                const uint32_t d = tmem + uint32_t((t & 1) * nq);
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    ok = ok && hs::mbar_wait_bounded(&B.kfull[slot], phase, tmo, abort_flag);
                    if (!ok) break;
                    hs::tc::fence_after_sync();
                    const uint64_t kd = k_desc + uint32_t(slot * (C::kSub >> 4));
                    const uint64_t qd =
                        q_desc + uint32_t(qb * (C::kQBytes >> 4) + s * C::kSubBlocks * nq * 8);
#pragma unroll
                    for (int b = 0; b < C::kSubBlocks; ++b) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma<KV>(d, kd + uint32_t(b * (kBlk >> 4) + kk * 2),
                                    qd + uint32_t(b * nq * 8 + kk * 2), id,
                                    (s | b | kk) ? 1u : 0u);
                    }
                    hs::tc::mma_commit(&B.kempty[slot]);
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                hs::tc::mma_commit(&B.s_full[t & 1]);
                if (!E4 && last_of_segment(c)) hs::tc::mma_commit(&B.q_empty);
                if (t + 1 < run) advance(c, a, chunks, lth);
            }
            if (!ok) {
                hs::set_status(a.status, HS_ERR_TIMEOUT);
                B.abort = 1;
            }
            // Every product issued has completed before TMEM is freed.
            hs::tc::mma_commit(&B.drain[0]);
            hs::mbar_wait_bounded(&B.drain[0], 0, tmo, nullptr);
        }
        __syncwarp();
    } else if (warp == kPvWarp) {
        // -------------------------- O^T += V^T P^T -----------------------------
        if (lane == 0) {
            constexpr int kStep = C::kStep, kSteps = kRows / kStep;
            const uint32_t id = idesc<KV>(C::NP, 1);
            const uint64_t v_desc = hs::tc::sdesc_sw128(sb + C::kVOff, kBlk, 1024);
            const uint64_t p_desc = hs::tc::sdesc_sw128(sb + C::kPOff, 16, 1024);
            // Output column of each K step's head, and the steps that hold a
            // head's first rows.
            uint32_t col[kSteps], starts = 0;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                const int r = kk * kStep;
                col[kk] = tmem + o_col + uint32_t((r >> lrow) & (hsn - 1)) * C::NP;
                if (r < (hsn << lrow) && (r & ((1 << lrow) - 1)) == 0) starts |= 1u << kk;
            }
            Cursor c = start;
            bool ok = true;
            int slot = 0, t0 = 0;
            uint32_t phase = 0;
            for (int t = 0, seg = 0; t < run; ++t) {
                if (c.first) {
                    // The epilogue of the segment before has read the output.
                    if (seg > 0)
                        ok = ok && hs::mbar_wait_bounded(&B.o_free, (seg - 1) & 1, tmo, abort_flag);
                    ++seg;
                    t0 = t;
                }
                ok = ok && hs::mbar_wait_bounded(&B.p_full[t & 1], (t >> 1) & 1, tmo, abort_flag);
                // A group's first tile of the segment starts its output.
                const uint32_t fresh = t - t0 < kGroups ? starts : 0u;
                const uint64_t pd = p_desc + uint32_t((t & 1) * (C::kPBytes >> 4));
#pragma unroll
                for (int s = 0; s < C::kSubs; ++s) {
                    ok = ok && hs::mbar_wait_bounded(&B.vfull[slot], phase, tmo, abort_flag);
                    if (!ok) break;
                    hs::tc::fence_after_sync();
                    const uint64_t vd = v_desc + uint32_t(slot * (C::kSub >> 4));
                    const uint32_t d = uint32_t(((t & 1) * C::kSubs + s) * ocols);
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk)
                        mma<KV>(d + col[kk], vd + uint32_t(kk * kStep * 8),
                                pd + uint32_t(E4 ? kk * 2 : (kk >> 2) * (C::NP * 8) + (kk & 3) * 2),
                                id, ((fresh >> kk) & 1u) ^ 1u);
                    hs::tc::mma_commit(&B.vempty[slot]);
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                hs::tc::mma_commit(&B.pv_done[t & 1]);
                if (t + 1 < run) advance(c, a, chunks, lth);
            }
            if (!ok) {
                hs::set_status(a.status, HS_ERR_TIMEOUT);
                B.abort = 1;
            }
            hs::tc::mma_commit(&B.drain[1]);
            hs::mbar_wait_bounded(&B.drain[1], 0, tmo, nullptr);
        }
        __syncwarp();
    } else if (warp == kQWarp) {
        // ------------------- queries (E4M3: the softmax warps) -------------------
        if constexpr (!E4) {
            Cursor c = start;
            bool ok = true;
            for (int seg = 0; c.left > 0; ++seg) {
                if (seg > 0 && !__all_sync(0xffffffffu,
                                           hs::mbar_wait_bounded(&B.q_empty, (seg - 1) & 1, tmo,
                                                                 abort_flag))) {
                    ok = false;
                    break;
                }
                const int kvh0 = c.chunk / gch * hsn, gc = c.chunk % gch;
                const int Gc = min(GM, group - gc * GM);
                const char* q = static_cast<const char*>(a.q) + int64_t(c.row) * a.q_stride * 2;
                constexpr int kCh = D / 8;  // 16-byte chunks of a query row
                for (int e = lane; e < nq * kCh; e += 32) {
                    const int n = e / kCh, ch = e % kCh;
                    const int hl = n / GM, gi = n % GM;
                    const bool in = hl < hsn && gi < Gc;
                    const int h = (kvh0 + min(hl, hsn - 1)) * group + gc * GM + min(gi, Gc - 1);
                    hs::tc::cp_async16(sb + C::kQOff + (ch >> 3) * uint32_t(nq) * 128 + n * 128 +
                                           (((ch & 7) ^ (n & 7)) << 4),
                                       q + int64_t(h) * D * 2 + ch * 16, in ? 16u : 0u);
                }
                hs::tc::cp_async_wait_all();
                hs::fence_proxy_async_shared();
                hs::mbar_arrive(&B.q_full[0]);
                next_segment(c, a, chunks, lth);
            }
            if (!ok) {
                hs::set_status(a.status, HS_ERR_TIMEOUT);
                B.abort = 1;
            }
        }
    } else {
        // ------------------------- softmax and epilogue ------------------------
        const int wg = warp >> 2;                // group: tiles t with t % 2 == wg
        const int r = tid & 127;                 // row of the tile, and TMEM lane
        const int hl = (r >> lrow) & (hsn - 1);  // its head in the unit
        const int rt = (r >> (lhs + lrow) << lrow) + (r & ((1 << lrow) - 1));  // its token
        const int run_r = rt >> lbt;             // and that token's run
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        // Heads of the warp's two half warps.
        const int hA = ((warp & 3) * 32 >> lrow) & (hsn - 1);
        const int hB = ((warp & 3) * 32 + 16 >> lrow) & (hsn - 1);
        const uint32_t s_addr = tmem + lane_base + uint32_t(wg * nq);
        const uint32_t o_addr = tmem + lane_base + o_col;
        const uint32_t o_own = o_addr + uint32_t(wg * C::kSubs * ocols);
        const uint32_t p_own = sb + C::kPOff + wg * C::kPBytes;
        // This row's place in P^T: K-major rows of 128 bytes, 64 (E4M3: 128)
        // cache rows each.
        const int p_col = E4 ? r : (r & 63) * 2;
        const uint32_t p_row =
            p_own + (E4 ? 0u : uint32_t(r >> 6) * (C::NP * 128)) + uint32_t(p_col & 15);
        const uint32_t p_chunk = uint32_t(p_col >> 4);
        auto put16 = [&](int n, uint16_t x) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                             p_row + n * 128 + ((p_chunk ^ uint32_t(n & 7)) << 4)),
                         "h"(x)
                         : "memory");
        };
        auto put8 = [&](int n, uint32_t x) {
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(
                             p_row + n * 128 + ((p_chunk ^ uint32_t(n & 7)) << 4)),
                         "r"(x)
                         : "memory");
        };
        // The j-th group of 16 rows that belong to this row's head, j < 8 / hs.
        auto rows_of = [&](int j) {
            const int lg = lrow - 4;  // log2 of a head's neighbouring groups
            return ((((j >> lg) << lhs) + hl) << lg) + (j & ((1 << lg) - 1));
        };
        bool fail = false;
        // A wait that gives up lets the CTA run to its end at once (every
        // later wait sees the flag), so that all its barriers are met.
        auto wait = [&](uint64_t* bar, int parity) {
            if (!hs::mbar_wait_bounded(bar, uint32_t(parity), tmo, abort_flag)) {
                fail = true;
                B.abort = 1;
            }
            __syncwarp();
        };
        Cursor c = start;
        // E4M3: the parts of a segment's queries, a step of rows per warp.  The
        // buffer's last reader, the segment before last, is done by then.
        auto make_parts = [&](const Cursor& x, int seg) {
            if constexpr (E4) {
                const int Gc = min(GM, group - x.chunk % gch * GM);
                constexpr int kStepRows = 512 / D;
                for (int it = warp; it * kStepRows < hsn * GM; it += kGroups * 4)
                    if (it * kStepRows % GM < Gc)
                        query_parts<D, GH, QP>(a, B, smem + C::kQOff + (seg & 1) * C::kQBytes, nq,
                                               hsn, x.row, x.chunk, seg, it);
                __syncwarp();
                hs::fence_proxy_async_shared();
                hs::mbar_arrive(&B.q_full[seg & 1]);
            }
        };
        make_parts(c, 0);
        for (int t = 0, seg = 0; t < run; ++seg) {
            // ---- One segment: the tiles of one unit in this run ----------------
            const int row = c.row;
            const int kvh0 = c.chunk / gch * hsn, gc = c.chunk % gch;
            const int Gc = min(GM, group - gc * GM);
            const Tiling v = c.v;
            const int tile0 = c.tile, n = min(c.left, v.n - tile0), t0 = t;
            const bool whole = n == v.n && cl <= 1;
            if (E4 && c.left > n) {
                Cursor x = c;
                next_segment(x, a, chunks, lth);
                make_parts(x, seg + 1);
            }
            const int slot = 2 * cta + (tile0 == 0 && t > 0 ? 1 : 0);
            float mref[GM], l[GM];
#pragma unroll
            for (int i = 0; i < GM; ++i) {
                mref[i] = -CUDART_INF_F;
                l[i] = 0.f;
            }
            bool own = false;  // this group has had a tile of the segment
            for (; t < t0 + n; ++t, advance(c, a, chunks, lth)) {
                if ((t & 1) != wg) continue;
                const int tok = tile_token(c, lth) + rt;
                wait(&B.s_full[wg], (t >> 1) & 1);
                hs::tc::fence_after_sync();
                const bool seen = visible(v, tok);
                const bool valid = seen && ((B.loaded[t % kMaskRing] >> run_r) & 1u);
                float x[GM];
#pragma unroll
                for (int k = 0; k < C::kQParts; ++k) {
                    float s[GM];
                    tmem_ld<GM>(s_addr + hA * C::NH + k * GM, s);
                    if (hB != hA) {
                        float s2[GM];
                        tmem_ld<GM>(s_addr + hB * C::NH + k * GM, s2);
                        hs::tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < GM; ++i) s[i] = lane < 16 ? s[i] : s2[i];
                    } else {
                        hs::tc::tmem_wait_ld();
                    }
                    constexpr float kPart[3] = {1.f, 0.0625f, 0.00390625f};
#pragma unroll
                    for (int i = 0; i < GM; ++i)
                        x[i] = k == 0 ? s[i] : fmaf(s[i], kPart[k], x[i]);
                }
#pragma unroll
                for (int i = 0; i < GM; ++i) {
                    x[i] *= E4 ? B.qscale[seg & 3][hl * GM + i] : a.scale_log2;
                    if (!valid) x[i] = -CUDART_INF_F;
                }
                if (a.logits != nullptr && seen) {
                    const int i = visible_index(v, tok);
                    float* lp = a.logits +
                                (int64_t(row) * a.heads + (kvh0 + hl) * group + gc * GM) *
                                    a.logit_stride + i;
#pragma unroll
                    for (int g = 0; g < GM; ++g)
                        if (g < Gc) lp[g * a.logit_stride] = x[g];
                }
                bool grow = !own;
#pragma unroll
                for (int i = 0; i < GM; ++i) grow |= i < Gc && x[i] > mref[i] + kThresh;
                // The group's P buffer and output: its product before is done.
                if (t >= kGroups) wait(&B.pv_done[wg], ((t - kGroups) >> 1) & 1);
                if (hs::pair::named_sync_or(kSoftBar + wg, kSoftThreads, grow)) {
                    // New reference maxima: the largest logits so far.
                    float mx[GM];
#pragma unroll
                    for (int i = 0; i < GM; ++i) mx[i] = x[i];
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < GM; ++i)
                            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
                    if (hsn < 8) {
                        if ((lane & 15) == 0)
#pragma unroll
                            for (int i = 0; i < GM; i += 4)
                                *reinterpret_cast<float4*>(&B.red[wg][r >> 4][i]) =
                                    make_float4(mx[i], mx[i + 1], mx[i + 2], mx[i + 3]);
                        hs::pair::named_sync(kSoftBar + wg, kSoftThreads);
                        for (int j = 0; j < (8 >> lhs); ++j) {
                            const float* q = B.red[wg][rows_of(j)];
#pragma unroll
                            for (int i = 0; i < GM; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(q + i);
                                mx[i] = fmaxf(mx[i], f.x);
                                mx[i + 1] = fmaxf(mx[i + 1], f.y);
                                mx[i + 2] = fmaxf(mx[i + 2], f.z);
                                mx[i + 3] = fmaxf(mx[i + 3], f.w);
                            }
                        }
                    }
                    if (own) {
                        // Rescale what has been summed.
#pragma unroll
                        for (int i = 0; i < GM; ++i) {
                            const float mn = fmaxf(mref[i], mx[i]);
                            const float al = mn == mref[i] ? 1.f : ex2(mref[i] - mn);
                            l[i] *= al;
                            mref[i] = mn;
                            if (rt == 0) B.alpha[wg][hl * GM + i] = al;
                        }
                        hs::pair::named_sync(kSoftBar + wg, kSoftThreads);
                        hs::tc::fence_after_sync();
#pragma unroll 1
                        for (int cb = 0; cb < C::kSubs * ocols; cb += 8) {
                            float o[8];
                            hs::tc::tmem_ld8(o_own + uint32_t(cb), o);
                            hs::tc::tmem_wait_ld();
                            const int oc = cb % ocols;
                            const float* al = &B.alpha[wg][oc / C::NP * GM + oc % GM];
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= al[i];
                            hs::tc::tmem_st8(o_own + uint32_t(cb), o);
                        }
                        hs::tc::tmem_wait_st();
                    } else {
#pragma unroll
                        for (int i = 0; i < GM; ++i) mref[i] = mx[i];
                    }
                }
                own = true;
#pragma unroll
                for (int i = 0; i < GM; i += 2) {
                    if (i >= Gc) break;
                    // Without a finite logit so far: subtract 0, every weight
                    // stays 0 (a NaN logit stays NaN).
                    const float p = ex2(x[i] - (mref[i] == -CUDART_INF_F ? 0.f : mref[i]));
                    const float p2 =
                        ex2(x[i + 1] - (mref[i + 1] == -CUDART_INF_F ? 0.f : mref[i + 1]));
                    l[i] += p;
                    l[i + 1] += p2;
                    float r0 = p * C::up(-1), r1 = p2 * C::up(-1);
#pragma unroll
                    for (int k = 0; k < C::kPParts; ++k) {
                        float2 f;
                        if constexpr (KV == kBf16) {
                            const __nv_bfloat162 c = __floats2bfloat162_rn(r0, r1);
                            f = __bfloat1622float2(c);
                            put16(k * GM + i, __bfloat16_as_ushort(c.x));
                            put16(k * GM + i + 1, __bfloat16_as_ushort(c.y));
                        } else if constexpr (KV == kFp16) {
                            const __half2 c = __floats2half2_rn(r0, r1);
                            f = __half22float2(c);
                            put16(k * GM + i, __half_as_ushort(c.x));
                            put16(k * GM + i + 1, __half_as_ushort(c.y));
                        } else {
                            const uint32_t c = to_e4m3x2(r0, r1);
                            f = from_e4m3x2(c);
                            put8(k * GM + i, c);
                            put8(k * GM + i + 1, c >> 8);
                        }
                        r0 = (r0 - f.x) * C::up(k);
                        r1 = (r1 - f.y) * C::up(k);
                    }
                }
                // Rows that are not attended to hold anything (places behind
                // the context, pages that were not loaded): their V becomes 0,
                // so that the weight 0 times it is 0.
                if (!valid) {
                    for (int s = 0; s < C::kSubs; ++s) {
                        const int seq = t * C::kSubs + s, at = seq % NS;
                        // A parity tells two neighbouring phases apart: the
                        // unit's load before this one has to be known to be
                        // complete.  pv_done says so up to tile t - 2; a unit
                        // that tile t - 1 used last is waited for.
                        bool full = true;
                        if (NS < 2 * C::kSubs && s >= NS - C::kSubs && seq >= NS)
                            full = hs::mbar_wait_bounded(&B.vempty[at], (seq / NS - 1) & 1, tmo,
                                                         abort_flag);
                        if (!full ||
                            !hs::mbar_wait_bounded(&B.vfull[at], (seq / NS) & 1, tmo, abort_flag)) {
                            fail = true;
                            B.abort = 1;
                        }
                        unsigned char* vr = smem + C::kVOff + at * C::kSub + r * 128;
#pragma unroll
                        for (int b = 0; b < C::kSubBlocks; ++b)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                reinterpret_cast<uint4*>(vr + b * kBlk)[(i + lane) & 7] =
                                    make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                __syncwarp();
                hs::fence_proxy_async_shared();
                hs::tc::fence_before_sync();
                hs::mbar_arrive(&B.p_full[wg]);
            }

            // ---- The segment's state: join the groups, write it -----------------
            // The groups' last products of the segment.
            if (own) {
                const int tl = ((t - 1) & 1) == wg ? t - 1 : t - 2;
                wait(&B.pv_done[wg], (tl >> 1) & 1);
            }
            hs::tc::fence_after_sync();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < GM; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if ((lane & 15) == 0)
#pragma unroll
                for (int i = 0; i < GM; i += 4)
                    *reinterpret_cast<float4*>(&B.red[wg][r >> 4][i]) =
                        make_float4(l[i], l[i + 1], l[i + 2], l[i + 3]);
            if (rt == 0)
#pragma unroll
                for (int i = 0; i < GM; ++i) B.m[wg][hl * GM + i] = mref[i];
            hs::pair::named_sync(kBothBar, kGroups * kSoftThreads);
            // A thread per query of the unit: both groups' sums, the unit's
            // maximum, and the factors that join their outputs.
            const int e = tid;
            if (e < hsn * GM) {
                const int h = e / GM, i = e % GM;
                float lw[kGroups];
#pragma unroll
                for (int w = 0; w < kGroups; ++w) {
                    lw[w] = 0.f;
                    const int lg = lrow - 4;
                    for (int j = 0; j < (8 >> lhs); ++j)
                        lw[w] += B.red[w][((((j >> lg) << lhs) + h) << lg) + (j & ((1 << lg) - 1))][i];
                }
                const float m0 = B.m[0][e], m1 = B.m[1][e];
                const float M = fmaxf(m0, m1), ref = M == -CUDART_INF_F ? 0.f : M;
                const float f0 = exp2f(m0 - ref), f1 = exp2f(m1 - ref);
                const float L = fmaf(f0, lw[0], f1 * lw[1]);
                float inv = 1.f;
                if (i < Gc) {
                    if (whole) {
                        const int64_t qh =
                            int64_t(row) * a.heads + (kvh0 + h) * group + gc * GM + i;
                        const float lg = L == 0.f ? -CUDART_INF_F : M + log2f(L);
                        if (a.lse != nullptr) a.lse[qh] = lg * kLn2;
                        if (a.lse2 != nullptr) a.lse2[qh] = lg;
                        inv = L == 0.f ? 0.f : 1.f / L;
                        if (a.v_scale != nullptr && L != 0.f) inv *= a.v_scale[kvh0 + h];
                    } else if (cl > 0) {
                        B.join_ml[h * GM + i] = make_float2(M, L);
                    } else {
                        const int64_t k = int64_t(slot) * a.unit_heads_max + e;
                        a.part_ml[2 * k] = M;
                        a.part_ml[2 * k + 1] = L;
                    }
                }
                inv *= 1.f / C::up(-1);
                B.weight[0][e] = f0 * inv;
                B.weight[1][e] = f1 * inv;
            }
            hs::pair::named_sync(kBothBar, kGroups * kSoftThreads);
            // A CTA of a cluster has one segment: its rings are free by now.
            float* joined = reinterpret_cast<float*>(smem);
            // A segment of one tile leaves the other group's output unwritten.
            const bool has0 = n > 1 || (t0 & 1) == 0, has1 = n > 1 || (t0 & 1) == 1;
            const bool bf = KV == kBf16 || (E4 && !a.q_is_half);
            for (int sh = wg; sh < (C::kSubs << lhs); sh += kGroups) {
                const int s = sh >> lhs, h = sh & (hsn - 1);
                const int d = s * 128 + r;
                float O[GM];
#pragma unroll
                for (int i = 0; i < GM; ++i) O[i] = 0.f;
#pragma unroll
                for (int w = 0; w < kGroups; ++w) {
                    if (!(w == 0 ? has0 : has1)) continue;
                    // The parts from the last to the first, a few at a time.
                    constexpr int kAt = C::NP <= 48 ? C::kPParts : C::kPParts / 2;
                    float sum[GM];
#pragma unroll
                    for (int k0 = C::kPParts - kAt; k0 >= 0; k0 -= kAt) {
                        float o[kAt * GM];
                        tmem_ld<kAt * GM>(o_addr + uint32_t((w * C::kSubs + s) * ocols + h * C::NP +
                                                            k0 * GM), o);
                        hs::tc::tmem_wait_ld();
#pragma unroll
                        for (int k = kAt - 1; k >= 0; --k)
#pragma unroll
                            for (int i = 0; i < GM; ++i)
                                sum[i] = k0 + k + 1 == C::kPParts
                                             ? o[k * GM + i]
                                             : fmaf(sum[i], 1.f / C::up(k0 + k), o[k * GM + i]);
                    }
#pragma unroll
                    for (int i = 0; i < GM; ++i)
                        O[i] = fmaf(sum[i], B.weight[w][h * GM + i], O[i]);
                }
                if (d >= D) continue;
                const int64_t qh = int64_t(row) * a.heads + (kvh0 + h) * group + gc * GM;
                const int64_t at = whole ? qh * D + d
                                         : (int64_t(slot) * a.unit_heads_max + h * GM) * D + d;
#pragma unroll
                for (int i = 0; i < GM; ++i) {
                    if (i >= Gc) break;
                    if (cl > 1)
                        joined[(h * GM + i) * D + d] = O[i];
                    else if (!whole)
                        a.part_o[at + i * D] = O[i];
                    else if (bf)
                        static_cast<__nv_bfloat16*>(a.out)[at + i * D] = __float2bfloat16_rn(O[i]);
                    else
                        static_cast<__half*>(a.out)[at + i * D] = __float2half_rn(O[i]);
                }
            }
            hs::tc::fence_before_sync();
            hs::mbar_arrive(&B.o_free);
            // The states are read: the next segment may write its own.
            hs::pair::named_sync(kBothBar, kGroups * kSoftThreads);
        }
        if (fail) hs::set_status(a.status, HS_ERR_TIMEOUT);
    }
    hs::tc::fence_before_sync();
    __syncthreads();
    hs::tc::fence_after_sync();
    if (warp == kPvWarp) hs::tc::tmem_dealloc(tmem, kTmemCols);
    if (cl > 1 || (cl == 1 && run == 0)) {
        // The cluster joins its parts, each CTA some pairs of dims; a request
        // without a token has none: zeros.
        if (cl > 1) hs::pair::cluster_sync();
        const int kvh0 = start.chunk / gch * hsn, gc = start.chunk % gch, tiles = start.v.n;
        const int Gc = min(GM, group - gc * GM);
        const int64_t qh0 = int64_t(start.row) * a.heads + kvh0 * group + gc * GM;
        const int pairs = hsn * Gc * (D / 2), share = (pairs + cl - 1) / cl;
        const int end = min(pairs, (rank + 1) * share);
        const uint32_t ml_at = hs::smem_u32(B.join_ml), o_at = hs::smem_u32(smem);
        for (int p = rank * share + tid; p < end; p += kThreads) {
            const int d = p % (D / 2) * 2, h = p / (D / 2) / Gc, i = p / (D / 2) - h * Gc;
            const int e = h * GM + i;
            float2 ml[kMaxCluster], o[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                ml[c] = make_float2(-CUDART_INF_F, 0.f);
                o[c] = make_float2(0.f, 0.f);
                // (CTAs without a tile have written nothing.)
                if (c < cl && tiles * (c + 1) / cl > tiles * c / cl) {
                    ml[c] = peer_load2(ml_at + e * 8, c);
                    o[c] = peer_load2(o_at + (e * D + d) * 4, c);
                }
            }
            float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, ml[c].x);
            const float ref = M == -CUDART_INF_F ? 0.f : M;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) {
                const float f = exp2f(ml[c].x - ref);
                L = fmaf(f, ml[c].y, L);
                sum.x = fmaf(f, o[c].x, sum.x);
                sum.y = fmaf(f, o[c].y, sum.y);
            }
            float inv = L == 0.f ? 0.f : 1.f / L;
            if (a.v_scale != nullptr && L != 0.f) inv *= a.v_scale[kvh0 + h];
            const int64_t qh = qh0 + h * group + i;
            sum.x *= inv;
            sum.y *= inv;
            if (KV == kBf16 || (E4 && !a.q_is_half))
                reinterpret_cast<__nv_bfloat162*>(a.out)[(qh * D + d) / 2] =
                    __floats2bfloat162_rn(sum.x, sum.y);
            else
                reinterpret_cast<__half2*>(a.out)[(qh * D + d) / 2] =
                    __floats2half2_rn(sum.x, sum.y);
            if (d == 0) {
                const float lg = L == 0.f ? -CUDART_INF_F : M + log2f(L);
                if (a.lse != nullptr) a.lse[qh] = lg * kLn2;
                if (a.lse2 != nullptr) a.lse2[qh] = lg;
            }
        }
        if (cl > 1) hs::pair::cluster_sync();  // no CTA ends while its parts are read
    }
}

// Tensor map of a cache: dims (head dim, token of the page, KV head, page).
int encode_map(CUtensorMap* m, int kv, const void* base, const PagedArgs& a, int d, int bt,
               int hs_box);

inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&attr)[2], int units, int cl,
                                         size_t smem) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cl);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(units) * unsigned(cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Sets a.cl, and returns the way whose units clusters take (1 where none do).
// Clusters take the units where all of them fit the GPU at once and the bound
// on the lengths leaves each CTA few tiles; then nothing is dealt, merged or
// launched behind (us, dealt / by clusters: one request of 128 tokens 8.1 /
// 6.2, 1 K 10.7 / 8.8, 4 K 13.9 / 11.6, 8 K 19.1 / 14.9; 16 requests of 128
// 11.0 / 7.9, of 1 K 22.9 / 18.2; 64 of 64 16.3 / 10.3; 16 with a window of
// 256 14.0 / 9.4).  With more tiles a ragged batch would wait for its longest
// request (24 of up to 5001 tokens and 256-wide heads: 38.3 / 33.5 where all
// are that long, but 21.7 dealt where they are half of it on average).
inline int cluster_way(PagedArgs& a, const void* kern, size_t smem, int tile_bytes,
                       int (&resident)[64][kMaxCluster + 1]) {
    int dev = 0;
    a.cl = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    const int64_t few = hs::min64(kTilesOfUnit, kUnitBytes / tile_bytes);
    for (int way = 1; way >= 0 && a.cl == 0; --way) {
        const int64_t units = int64_t(a.rows) * a.chunks[way], tiles = most_tiles(a, a.lth[way]);
        if (units > a.ctas || tiles > few * kMaxCluster) continue;
        int64_t best = INT64_MAX;
        for (int cl = 1; cl <= kMaxCluster && units * cl <= a.ctas; ++cl) {
            // In halves of a tile's time: a join takes as long as 2.5 tiles,
            // or 4.5 where the unit has several heads.
            const int64_t each = hs::max64(1, (tiles + cl - 1) / cl);
            const int64_t cost = 2 * each + (cl == 1 ? 0 : a.hs[way] == 1 ? 5 : 9);
            if (each > few || cost >= best) continue;
            const auto ask = [&] {
                int n = 0;
                cudaLaunchAttribute attr[2];
                const cudaLaunchConfig_t cfg = cluster_config(attr, 1, cl, smem);
                if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0)
                    return n;
                cudaGetLastError();
                return -1;
            };
            if (cl > 1 && units > hs_host::ask_once(&resident[dev][cl], ask)) continue;
            best = cost;
            a.cl = cl;
        }
        if (a.cl > 0) return way;
    }
    return 1;
}

template <int KV, int D, int GH, int QP>
int launch_one(PagedArgs& a, hs_stream_t stream) {
    using C = Cfg<KV, D, GH, QP>;
    constexpr int GM = C::GM;
    TcArgs t{};
    set_ways(a, C::kHsMax, kRows, GM, kTilesForWide, C::kExtra);
    if (C::kElt == 2 && a.rows * a.chunks[0] <= kWideAlone)
        a.wide_to = int64_t(a.ctas) * kTilesAlone;
    for (int i = 0; i < 2; ++i) {
        t.bt[i] = kRows / a.hs[i];
        while (a.page_size % t.bt[i]) t.bt[i] /= 2;
        t.split[i] = a.hs[i] > 1 && t.bt[i] < C::kStep;
    }
    t.timeout_ns = hs::kWaitTimeoutNs;
    auto kern = paged_tc_kernel<KV, D, GH, QP>;
    constexpr size_t smem = size_t(C::kBarOff) + sizeof(Bars) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static int smem_set[64] = {};
    int rc = hs_host::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem, smem_set);
    if (rc != HS_OK) return rc;
    static int resident[64][kMaxCluster + 1] = {};
    const int only = cluster_way(a, reinterpret_cast<const void*>(kern), smem,
                                 2 * C::kSubs * C::kSub, resident);
    // Small calls surely take one way: two descriptors instead of four.
    const bool both = a.cl == 0 && a.hs[0] != 1 && most_places(a) >= a.wide_from;
    CUtensorMap m[4];
    for (int i = 0; i < 2; ++i) {
        if (!both && i != only) continue;
        rc = encode_map(&m[2 * i], KV, a.k, a, D, t.bt[i], t.split[i] ? 1 : a.hs[i]);
        if (rc == HS_OK)
            rc = encode_map(&m[2 * i + 1], KV, a.v, a, D, t.bt[i], t.split[i] ? 1 : a.hs[i]);
        if (rc != HS_OK) return rc;
    }
    if (!both) {
        const int other = 1 - only;
        m[2 * other] = m[2 * only];
        m[2 * other + 1] = m[2 * only + 1];
        t.bt[other] = t.bt[only];
        t.split[other] = t.split[only];
        a.hs[other] = a.hs[only];
        a.lth[other] = a.lth[only];
        a.chunks[other] = a.chunks[only];
    }
    t.p = a;
    if (a.cl <= 1) {
        const int ctas = a.cl == 0 ? a.ctas : a.rows * a.chunks[1];
        return hs_host::launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, t, m[0], m[1],
                                   m[2], m[3]);
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(attr, a.rows * a.chunks[1], a.cl, smem);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    if (cudaLaunchKernelEx(&cfg, kern, t, m[0], m[1], m[2], m[3]) != cudaSuccess) {
        cudaGetLastError();
        return HS_ERR_CUDA;
    }
    return HS_OK;
}

template <int KV, int QP>
int launch_kind(PagedArgs& a, int d, int group, hs_stream_t stream) {
    if constexpr (KV != kE4m3) {
        if (d == 64)
            return group <= 8 ? launch_one<KV, 64, 1, QP>(a, stream)
                              : launch_one<KV, 64, 2, QP>(a, stream);
    }
    if (d == 128)
        return group <= 8 ? launch_one<KV, 128, 1, QP>(a, stream)
                          : launch_one<KV, 128, 2, QP>(a, stream);
    return group <= 8 ? launch_one<KV, 256, 1, QP>(a, stream)
                      : launch_one<KV, 256, 2, QP>(a, stream);
}

}  // namespace tc
}  // namespace hs_paged
