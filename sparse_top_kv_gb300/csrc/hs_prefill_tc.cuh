// hs_prefill_tc.cuh -- the attention kernel of hs_paged_prefill on the 5th-
// generation tensor cores (included by one translation unit per cache type).
//
// Math, per new token i and query head h of KV head g, over the cached tokens t
// that the token's position attends to:
//   x_t = scale * k_scale_g * (q . K_t),  p_t = 2^((x_t - m) log2 e),
//   l = sum p_t,  out = v_scale_g / l * sum p_t V_t,
// as (m, l, sum) states, exact under merging (the rule of hs_merge_states).
//
// 4 d flops per (query, token) and head: the tensor cores bound long chunks, HBM
// and latency few tokens.
//  * A query tile is 128 rows of (new token, query head of the KV head), so that
//    a K tile of 128 cached tokens serves every head that shares it, and the
//    causal edge is 128 / group tokens wide.  Two query tiles share the K and V
//    tiles, and the tensor cores work on one while the other is in its softmax;
//    heads of 256 (whose two outputs TMEM does not hold) and few tokens over
//    E4M3 caches have units of one, whose tokens two warpgroups share.
//  * S[queries x tokens] = Q K^T from shared memory into TMEM; P goes back into
//    TMEM as the A operand of O += P V, V an MN-major view of its tile.  A thread
//    per query row: no shuffle in the softmax, and P, O and the statistics of a
//    row never leave their lane.
//  * Softmax against a reference maximum that moves only when a logit exceeds it
//    by 2^kThresh, so that O is rescaled a few times a unit.
//  * P is rounded once to the type of V's products: bf16, or fp16 raised by
//    2^kShift, so that weights down to 2^-25 of the reference keep 11 bits and
//    smaller ones 2^-36 of it.  The sums l are of unrounded weights, in fp32.
//  * E4M3 caches become fp16 in shared memory (exact), bf16 queries fp16 of
//    their row's largest magnitude 2^14 (elements down to 2^-28 of it exact).
//  * Loads: caches whose pages hold runs of 8 tokens by TMA, E4M3 ones into a
//    stage, from which four warps convert them; others by 128 threads, a batch of
//    loads ahead of the stores.  K and V of a unit's first tile go ahead of its
//    queries, and page numbers are looked up a tile ahead.
//  * Entries of V that are not finite must not meet a weight of 0.  Where some
//    query of the unit does not see some token of a tile, rows that no query
//    sees become 0, and rows with entries that are not finite too; those are
//    added to the queries that do see them, one by one.
// Code is fetched like data: the kernel's is as large as the instruction cache,
// and what a unit runs once (masks, plan, output) costs its fetch.  So whatever is
// not a tile's main path is short, shared or rolled.
//
// Measured, 32/8 heads of 128 if nothing else is said.  Over inputs that change from
// call to call: 2048 tokens over 32 K in bf16 0.75 to 0.79 ms (1.4 PFLOP/s of 1.9
// measured; the power cap lowers the clocks), 16 requests of 5 tokens over up to 8 K
// 63 us (4.5 TB/s of 6.8), chunks of up to 512 tokens over up to 8 K of E4M3 200 us
// (0.87 PFLOP/s: the conversion), 16/1 heads of 256 over up to 5 K 91 us (0.76: rings
// of 1.25 tiles).  Replays of a captured graph over the same inputs: 2048 tokens over
// 32 K 0.69 to 0.71 ms (1.5), over 4 K 91 us, over 16 K of E4M3 434 us (1.2), 16/2 heads
// of 256 over 8 K 225 to 234 us (1.05).  (Here and below, figures of other sizes than the first four
// are of replays.)
// Every wait is bounded (HS_ERR_TIMEOUT in the status word on expiry).
#pragma once

#include <cuda.h>

#include "hs_pair.cuh"
#include "hs_prefill.cuh"
#include "hs_shared.h"
#include "hs_tcgen05.cuh"

namespace hs_prefill {
namespace tc {

enum Kind { kBf16 = 0, kFp16 = 1, kE4m3 = 2 };

constexpr int kThreads = 512;
constexpr int kQkWarp = 8, kPvWarp = 9;
constexpr int kTmaWarp = 10;   // or the queries
constexpr int kPlanWarp = 11;  // the run's units, one after another
constexpr int kQThreads = 32;
constexpr int kUnitRing = 4;   // units that the roles may be apart
constexpr int kLoadWarp = 12;  // to 15: V's rows or the loads, and the outputs
constexpr int kLoadBar = 1;    // named barrier of the loading threads
constexpr int kBlk = kTile * 128;  // 128 rows x 128 bytes
constexpr int kTmemCols = 512;

struct TcArgs {
    PrefillArgs p;
    int32_t bt;  // tokens of a run (a TMA box): they lie in one page
    uint64_t timeout_ns;
};

// Who loads K and V.
enum Loads { kTma = 0, kThreadsLoad = 1 };

template <int KV, int D, int LD, int QT>
struct Cfg {
    static constexpr int kKind = KV, kD = D;
    static constexpr bool kE4 = KV == kE4m3, kByTma = LD == kTma;
    static constexpr bool kConvert = kE4 && kByTma;        // E4M3 units pass through a stage
    static constexpr int NQ = QT;                          // query tiles of a unit
    static_assert(QT == 1 || D < 256, "two outputs of 256 dims do not fit TMEM");
    static constexpr int kDims = D < 128 ? D : 128;        // dims of a ring unit
    static constexpr int kSubs = D / kDims;                // ring units of a tile
    static constexpr int kUnit = kTile * kDims * 2;
    static constexpr int kQTile = kTile * D * 2;
    // Ring units: what shared memory holds.
    static constexpr int NS = D == 64 ? 8 : (kByTma && !kConvert ? 5 : 4) + (D == 128 && QT == 1 ? 1 : 0);
    static constexpr int kStages = kConvert ? 2 : 0, kStage = kTile * kDims;
    static constexpr int kOddWords = kConvert ? 16 : 4;
    static constexpr int kRing = 8;        // tiles whose loaded tokens are remembered
    static constexpr int kSegRing = QT == 1 ? 4 : 2;  // units whose query scales are
    static constexpr int kRingOff = NQ * kQTile;       // (queries first)
    static constexpr int kStageOff = kRingOff + NS * kUnit;
    static constexpr int kBarOff = kStageOff + kStages * kStage;
    // TMEM columns.  Two query tiles: one S for both, a P of each, an O of each.
    // One: two S buffers, P in the first half of each half of them, and O.
    static constexpr uint32_t kPCol = 128, kOCol = 256;
    // Registers of a thread, by warpgroup: 2 * soft + products + loads = 512.
    static constexpr int kSoftRegs = kByTma ? 176 : 168, kMmaRegs = kByTma ? 64 : 72,
                         kLoadRegs = kByTma ? 96 : 104;
    static_assert(2 * kSoftRegs + kMmaRegs + kLoadRegs == 65536 / 128, "register shares");
    // Log2 headroom before the reference moves, and what P is raised by.
    static constexpr float kThresh = KV == kBf16 ? 8.f : 4.f;
    static constexpr float kShift = KV == kBf16 ? 0.f : 11.f;
};

// One unit's share of a run, as the roles of the CTA see it: written to a ring by
// one warp (all of them finding it for themselves made 144 KB of code, more than
// an SM's instruction cache, and 2 us of a unit's time).
struct Seg {
    int32_t n;               // this run's tiles; 0: no more units
    int32_t row, kvh;
    int32_t first, m;        // its first new token, and how many
    int32_t p0;              // position of the first query
    int32_t i0, ns, tw;      // first tile; tiles of the sinks; first tile of the rest
    int32_t slot;            // of the partial state, -1: the unit is whole
};
template <typename C>
struct Bars {
    uint64_t kfull[C::NS], vfull[C::NS], ready[C::NS], empty[C::NS];
    uint64_t sfull[2], sempty[2], unit_full[kUnitRing], unit_free[kUnitRing];
    uint64_t q_raw, q_full, q_empty, s_full[2], s_free[2], p_full[2], pv_done[2], l_full[2], o_free[2], drain[2];
    uint64_t pair[C::NQ == 1 ? 4 : 1];  // of warps that share rows
    Seg unit[kUnitRing];
    uint32_t tmem_base;
    volatile int32_t abort;
    alignas(16) uint32_t loaded[C::kRing][4];     // tokens of a tile that were loaded
    int2 tile[C::kRing];                          // its first token; whether some query does not see all of it
    // Rows of V that were taken out, by ring unit (where threads convert, what each
    // of four warps has found, to be joined).
    alignas(16) uint32_t odd[C::kRing][C::kSubs][C::kOddWords / 4][4];
    float factor[C::NQ][kTile];                   // of each row's output; 0: nothing was attended to
    int8_t qexp[C::kE4 ? C::kSegRing : 1][C::kE4 ? C::NQ * kTile : 1];  // queries are raised by 2^qexp
    int64_t offset[C::kByTma ? 1 : 2][C::kByTma ? 1 : kTile];  // rows of a tile in the cache, -1: none
};

__device__ __forceinline__ int token_of(const Seg& s, int i) {
    const int j = s.i0 + i;
    return (j < s.ns ? j : j - s.ns + s.tw) * kTile;
}
// Whether any query of the unit sees token t.
__device__ __forceinline__ bool any_sees(const PrefillArgs& a, const Seg& s, int t) {
    return t < s.p0 + s.m && (a.window == 0 || t > s.p0 - a.window || t < a.sinks);
}
// Whether any of them sees any of the tokens [t, t + n).
__device__ __forceinline__ bool any_sees(const PrefillArgs& a, const Seg& s, int t, int n) {
    return t < s.p0 + s.m && (a.window == 0 || t + n - 1 > s.p0 - a.window || t < a.sinks);
}
// Whether every query of the unit sees every token of the tile from t on.
__device__ __forceinline__ bool all_see(const PrefillArgs& a, const Seg& s, int t) {
    return t + kTile - 1 <= s.p0 &&
           (a.window == 0 || t > s.p0 + s.m - 1 - a.window || t + kTile <= a.sinks);
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int tok,
                                         int head, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(tok), "r"(head), "r"(page), "r"(hs::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, int x, int head,
                                           int token, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(head), "r"(token), "r"(hs::smem_u32(bar))
        : "memory");
}
// Products and commits are issued by the whole warp, converged, for one elected
// lane, four products to a statement: with a lane of its own in a branch, the
// operands' way to uniform registers made each product 110 cycles' work, twice
// what the tensor cores take for it.
// D(tmem) (+)= A(smem desc) B(smem desc), four K steps of 16 (32 bytes apart).
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// D(tmem) (+)= A(tmem) B(smem desc, 16 rows of 128 bytes a K step), four steps.
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            hs::smem_u32(bar))
        : "memory");
}
// kind::f16, fp32 accumulators, A K-major (or in TMEM), M = 128.
template <int KV>
__host__ __device__ constexpr uint32_t idesc(int N, int b_mn_major) {
    return (1u << 4) | ((KV == kBf16 ? 1u : 0u) << 7) | ((KV == kBf16 ? 1u : 0u) << 10) |
           (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
}

// 32 lanes x 32 columns of 32 bit.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(x) : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
    return r;
}
template <int N>
__device__ __forceinline__ void set_max_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 2^x (PTX ex2.approx.ftz: within 2 ulp; 0 below -126, where a weight no longer
// counts against the sum's 1).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N]) {
    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int c = 4; c < N - 4; c += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], v[c + 2 * j], v[c + 2 * j + 1]);
    mx[0] = max3(mx[0], v[N - 4], v[N - 3]);
    mx[1] = max3(mx[1], v[N - 2], v[N - 1]);
    return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
}
template <int KV>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (KV == kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// x if `bit` is set in bits, else -inf.  (The compiler's own: ten instructions.)
__device__ __forceinline__ float keep_if(float x, uint32_t bits, uint32_t bit) {
    float r;
    asm("{\n\t.reg .pred p;\n\t.reg .b32 t;\n\tand.b32 t, %2, %3;\n\tsetp.ne.u32 p, t, 0;\n\t"
        "selp.f32 %0, %1, 0fFF800000, p;\n\t}"
        : "=f"(r)
        : "f"(x), "r"(bits), "r"(bit));
    return r;
}
// The low n bits (n outside [0, 32] as the nearest).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
    return uint32_t(h.x) | (uint32_t(h.y) << 16);
}
// Whether any of the 16 bytes' entries is not finite.
template <int KV>
__device__ __forceinline__ bool not_finite(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KV == kE4m3) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) any |= ((u[i] >> j) & 0x7fu) == 0x7fu;
        } else {
            constexpr uint32_t e = KV == kBf16 ? 0x7f80u : 0x7c00u;
            any |= (u[i] & e) == e || ((u[i] >> 16) & e) == e;
        }
    }
    return any;
}
// Element i of a cache row as fp32.
template <int KV>
__device__ __forceinline__ float element(const void* row, int i) {
    if constexpr (KV == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(row)[i]);
    else if constexpr (KV == kFp16) return __half2float(static_cast<const __half*>(row)[i]);
    else return float(static_cast<const __nv_fp8_e4m3*>(row)[i]);
}

// Ring unit u of the CTA's tile t: first those of K, then those of V.
template <typename C>
__device__ __forceinline__ int unit_of(int t, bool v, int u) {
    return (2 * t + (v ? 1 : 0)) * C::kSubs + u;
}
// The barriers of K's units and of V's count those alone: loads may land in
// another order than they were issued in, and a parity tells only neighbouring
// phases apart, so who waits has to have seen the phase before.
template <typename C>
__device__ __forceinline__ int turn_of(int t, int u) {
    return t * C::kSubs + u;
}

// As hs::mbar_wait_bounded, in a dozen instructions (there are many waits).
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                             uint32_t abort_flag) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 t0, t;\n\t.reg .b32 f;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE%=;\n\t"
        "mov.u64 t0, %%globaltimer;\n"
        "AGAIN%=:\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE%=;\n\t"
        "ld.volatile.shared::cta.b32 f, [%4];\n\t"
        "setp.ne.b32 q, f, 0;\n\t"
        "@q bra DONE%=;\n\t"
        "mov.u64 t, %%globaltimer;\n\t"
        "sub.u64 t, t, t0;\n\t"
        "setp.gt.u64 q, t, %3;\n\t"
        "@!q bra AGAIN%=;\n"
        "DONE%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "l"(timeout_ns), "r"(abort_flag)
        : "memory");
    return ok != 0;
}

// What every role of the CTA knows.
template <typename C>
struct Cta {
    const TcArgs& ta;
    const PrefillArgs& a;
    Bars<C>& B;
    unsigned char* smem;
    uint32_t sb, tmem;
    __device__ __forceinline__ bool wait(uint64_t* bar, int phase) const {
        return wait_bounded(hs::smem_u32(bar), uint32_t(phase & 1), ta.timeout_ns,
                            hs::smem_u32(const_cast<int32_t*>(&B.abort)));
    }
    // By all lanes of a warp.
    __device__ __forceinline__ bool wait_all(uint64_t* bar, int phase) const {
        return __all_sync(0xffffffffu, wait(bar, phase));
    }
    // The product of query tile w's n-th P is done.
    __device__ __forceinline__ bool pv_wait(int w, int n) const {
        return C::NQ == 2 ? wait_all(&B.pv_done[w], n) : wait_all(&B.pv_done[n & 1], n >> 1);
    }
    // The k-th unit of the run (all lanes); false: no more, or ok = false.
    __device__ __forceinline__ bool next_unit(int k, Seg& s, bool& ok) const {
        if (!ok) return false;
        ok = wait_all(&B.unit_full[k % kUnitRing], k / kUnitRing);
        if (!ok) return false;
        s = B.unit[k % kUnitRing];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) hs::mbar_arrive(&B.unit_free[k % kUnitRing]);
        return s.n > 0;
    }
    // Tokens of the CTA's tile t that a query at position pos sees.
    __device__ __forceinline__ void see(int t, int pos, uint32_t (&vis)[4]) const {
        const uint4 ld = *reinterpret_cast<const uint4*>(B.loaded[t & (C::kRing - 1)]);
        const int t0 = B.tile[t & (C::kRing - 1)].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = t0 + 32 * j;
            vis[j] = low_bits(pos + 1 - b) & (j == 0 ? ld.x : j == 1 ? ld.y : j == 2 ? ld.z : ld.w);
            if (a.window > 0)
                vis[j] &= ~low_bits(pos - a.window + 1 - b) | low_bits(a.sinks - b);
        }
    }
    __device__ __forceinline__ void give_up() const {
        hs::set_status(a.status, HS_ERR_TIMEOUT);
        B.abort = 1;
    }
};

// Rows of V that were taken out of a tile, into a row's output: P stands until the
// next one is written, O has the other rows' products.  Apart from the softmax's
// code and registers: it hardly ever runs.
template <int KV, int D, int WORDS, bool SPLIT>
__device__ __noinline__ void add_odd_rows(const PrefillArgs* ap, const uint32_t* odd, uint4 vis,
                                          int t0, int row, int kvh, uint32_t o_addr,
                                          uint32_t p_addr, int u) {
    constexpr int kDims = D < 128 ? D : 128;
    const PrefillArgs& a = *ap;
    odd += u * WORDS;
#pragma unroll 1
    for (int j = 0; j < kTile; ++j) {
        uint32_t word = 0;
        for (int g = 0; g < WORDS; g += 4) word |= odd[g + (j >> 5)];
        if (!((word >> (j & 31)) & 1u)) continue;
        // (Split softmax: the second half's weights are 32 columns further.)
        const uint32_t pw = tmem_ld1(p_addr + uint32_t((j >> 1) + (SPLIT && j >= 64 ? 32 : 0)));
        hs::tc::tmem_wait_ld();
        const uint32_t h = (j & 1) ? pw >> 16 : pw & 0xffffu;
        const float p = KV == kBf16 ? __uint_as_float(h << 16)
                                    : __half2float(__ushort_as_half(uint16_t(h)));
        const uint32_t vw = j < 32 ? vis.x : j < 64 ? vis.y : j < 96 ? vis.z : vis.w;
        const bool sees = (vw >> (j & 31)) & 1u;
        const int tk = t0 + j, b = block_of(a, tk);
        const int64_t page = a.block_table[row * a.bt_stride + b];
        const void* from = static_cast<const char*>(a.v) +
                           (page * a.page_stride + int64_t(tk - b * a.page_size) * a.row_stride +
                            kvh * a.head_stride) * (KV == kE4m3 ? 1 : 2);
#pragma unroll 1
        for (int c = u * kDims; c < (u + 1) * kDims; c += 16) {
            float o[16];
            hs::tc::tmem_ld16(o_addr + uint32_t(c), o);
            hs::tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (sees) o[e] = fmaf(p, element<KV>(from, c + e), o[e]);
            hs::tc::tmem_st16(o_addr + uint32_t(c), o);
            hs::tc::tmem_wait_st();
        }
    }
}
template <typename C>
__device__ __forceinline__ void softmax_role(const Cta<C>& cx) {
    static_assert(C::NQ == 2 && C::kSubs == 1, "two query tiles");
    constexpr int NS = C::NS, KV = C::kKind, D = C::kD;
    constexpr bool E4 = C::kE4;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int tid = threadIdx.x, warp = tid >> 5;
    const uint32_t tmem = cx.tmem;
    const int w = warp >> 2;   // query tile
    const int r = tid & 127;   // row of the tile, and TMEM lane
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const int tok = r / a.group, hd = r - tok * a.group;  // its new token and query head
    const uint32_t o_addr = tmem + lanes + C::kOCol + uint32_t(w * 128);
    bool ok = true;
    int t = 0, mine = 0;  // the CTA's tiles, this query tile's
    int own = 0;          // units with this query tile
    Seg s;
    for (int unit = 0; cx.next_unit(unit, s, ok); ++unit) {
        const int n = s.n;
        if (w * a.tq >= s.m) {  // the second tile of a unit that has one
            t += n;
            continue;
        }
        // The row's position; rows without a query see what the last does.
        const int pos = s.p0 + min(w * a.tq + tok, s.m - 1);
        float as = a.scale_log2;        // its size: the product made the sign
        float off = -CUDART_INF_F;      // reference - kShift
        uint64_t l0 = 0, l1 = 0;        // sums, in pairs
        bool first = true;
        const int last = mine + n;
        for (; mine < last; ++t, ++mine, first = false) {
            const uint32_t s_addr = tmem + lanes;
            const uint32_t p_addr = tmem + lanes + C::kPCol + uint32_t(w * 64);
            ok = ok && cx.wait_all(&B.s_full[w], mine);
            if (!ok) break;
            hs::tc::fence_after_sync();
            float v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, v + c * 32);
            if (first) {
                // (0 would turn masked places into NaN; 2^-126 does not show.)
                if constexpr (E4) {
                    as *= pow2(-B.qexp[unit & (C::kSegRing - 1)][w * kTile + r]);
                    if (a.k_scale != nullptr) as *= a.k_scale[s.kvh];
                }
                as = as == 0.f ? 1.17549435e-38f : fabsf(as);
            }
            const bool part = B.tile[t & (C::kRing - 1)].y != 0;
            hs::tc::tmem_wait_ld();
            hs::tc::fence_before_sync();
            hs::mbar_arrive(&B.s_free[0]);
            if (part) {
                // What this row sees of the tile, 32 tokens at a time.
                uint32_t vis[4];
                cx.see(t, pos, vis);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (__all_sync(0xffffffffu, vis[j] == 0xffffffffu)) continue;
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[32 * j + c] = keep_if(v[32 * j + c], vis[j], 1u << c);
                }
            }
            uint64_t as2, ref2, s0 = 0, s1 = 0;
            const auto refer = [&] {
                // Without a finite logit so far: subtract 0, every weight is
                // 0 (a NaN logit stays NaN).
                const float ref = off == -CUDART_INF_F ? 0.f : off;
                as2 = pair_of(as, as);
                ref2 = pair_of(-ref, -ref);
            };
            const auto weigh = [&](int c) {  // columns [32 c, 32 c + 32)
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const int e = 32 * c + 2 * j;
                    const float2 y = split(fma2(pair_of(v[e], v[e + 1]), as2, ref2));
                    const float2 z = split(fma2(pair_of(v[e + 2], v[e + 3]), as2, ref2));
                    const float2 p = make_float2(ex2(y.x), ex2(y.y)), q = make_float2(ex2(z.x), ex2(z.y));
                    s0 = add2(s0, pair_of(p.x, p.y));
                    s1 = add2(s1, pair_of(q.x, q.y));
                    pk[j] = pack<KV>(p.x, p.y);
                    pk[j + 1] = pack<KV>(q.x, q.y);
                }
                tmem_st16u(p_addr + c * 16, pk);
            };
            // The largest logit, as a reference, moves the old one where it is far
            // above.  (Weights made ahead of it, by the old reference, and made again
            // where it moved: 2 to 8 % slower, whichever part of them.)
            const float top = largest(v) * as - C::kShift;
            const bool grow = top > off + C::kThresh || (off == -CUDART_INF_F && top > off);
            if (mine > 0) {
                ok = ok && cx.pv_wait(w, mine - 1);
                hs::tc::fence_after_sync();
            }
            if (first) {
                if (grow) off = top;
            } else if (__any_sync(0xffffffffu, grow)) {
                // What has been summed is scaled down.
                const float to = grow ? top : off;
                const float al = grow ? (off == -CUDART_INF_F ? 0.f : ex2(off - to)) : 1.f;
                off = to;
                l0 = fma2(l0, pair_of(al, al), 0);
                l1 = fma2(l1, pair_of(al, al), 0);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float o[16];
                    hs::tc::tmem_ld16(o_addr + uint32_t(c), o);
                    hs::tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] *= al;
                    hs::tc::tmem_st16(o_addr + uint32_t(c), o);
                }
            }
            if (!ok) break;
            refer();
            weigh(0);
            weigh(1);
            weigh(2);
            weigh(3);
            l0 = add2(l0, s0);
            l1 = add2(l1, s1);
            hs::tc::tmem_wait_st();
            hs::tc::fence_before_sync();
            hs::mbar_arrive(&B.p_full[w]);
            if (part) {
                // Rows of V that were taken out, into the queries that see them.
                ok = cx.wait_all(&B.ready[t % NS], t / NS);
                const uint4* o = reinterpret_cast<const uint4*>(B.odd[t & (C::kRing - 1)][0]);
                uint32_t any = 0;
#pragma unroll
                for (int g = 0; g < C::kOddWords / 4; ++g) any |= o[g].x | o[g].y | o[g].z | o[g].w;
                if (any != 0 && ok) {
                    ok = cx.pv_wait(w, mine);
                    hs::tc::fence_after_sync();
                    uint32_t vis[4];
                    cx.see(t, pos, vis);
                    add_odd_rows<KV, D, C::kOddWords, false>(
                        &a, &B.odd[t & (C::kRing - 1)][0][0][0],
                        make_uint4(vis[0], vis[1], vis[2], vis[3]), B.tile[t & (C::kRing - 1)].x,
                        s.row, s.kvh, o_addr, p_addr, 0);
                }
                if (!ok) break;
            }
        }
        if (!ok) break;
        // ---- The unit's state: its output is written by another warpgroup ----
        if (own > 0) ok = cx.wait_all(&B.o_free[w], own - 1);
        if (!ok) break;
        ++own;
        const float2 ls = split(add2(l0, l1));
        const float l = ls.x + ls.y;
        const bool live = tok < a.tq && w * a.tq + tok < s.m;
        float f = 1.f;
        if (s.slot < 0) {
            f = l == 0.f ? 0.f : 1.f / l;
            if (a.v_scale != nullptr && l != 0.f) f *= a.v_scale[s.kvh];
            if (live && a.lse != nullptr)
                a.lse[int64_t(s.first + w * a.tq + tok) * a.heads + s.kvh * a.group + hd] =
                    l == 0.f ? -CUDART_INF_F : (off + log2f(l)) * kLn2;
        } else if (live) {
            reinterpret_cast<float2*>(a.part_ml)[int64_t(s.slot) * a.unit_rows + w * kTile + r] =
                make_float2(off, l);
        }
        B.factor[w][r] = f;
        hs::tc::fence_before_sync();
        hs::mbar_arrive(&B.l_full[w]);
    }
    if (!ok) cx.give_up();
}


// A unit of one query tile (a head size of 256, or few new tokens over an E4M3
// cache): each warpgroup has half of a tile's tokens, and of the output's dims where
// it is changed, so that the rows' softmax has all eight warps.  (By four, the other
// idle, it took longer than the tile's products: 2048 tokens over 8 K of E4M3, heads
// of 256, 465 us, now 419.)  Two warps that
// share rows tell each other their largest logits by a column of S, and so have
// one reference.
template <typename C>
__device__ __forceinline__ void softmax_split_role(const Cta<C>& cx) {
    static_assert(C::NQ == 1, "one query tile");
    constexpr int NS = C::NS, KV = C::kKind, D = C::kD;
    constexpr bool E4 = C::kE4;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int w = warp >> 2;   // half
    const int r = tid & 127;   // row of the tile, and TMEM lane
    const uint32_t rows = cx.tmem + (uint32_t((warp & 3) * 32) << 16);
    const int tok = r / a.group, hd = r - tok * a.group;  // its new token and query head
    const uint32_t o_addr = rows + C::kOCol;
    uint64_t* pair = &B.pair[warp & 3];
    bool ok = true;
    int t = 0, met = 0;  // the CTA's tiles; exchanges with the other warp
    // What was written before is the other warp's to read, and its own this one's.
    const auto meet = [&] {
        __syncwarp();
        if (lane == 0) hs::mbar_arrive(pair);
    };
    Seg s;
    for (int unit = 0; cx.next_unit(unit, s, ok); ++unit) {
        // The row's position; rows without a query see what the last does.
        const int pos = s.p0 + min(tok, s.m - 1);
        float as = a.scale_log2;        // its size: the product made the sign
        float off = -CUDART_INF_F;      // reference - kShift
        uint64_t l0 = 0, l1 = 0;        // sums, in pairs
        bool first = true;
        const int last = t + s.n;
        for (; t < last; ++t, first = false) {
            const int x = t & 1;
            const uint32_t s_addr = rows + uint32_t(x * 128 + w * 64);  // and P
            ok = ok && cx.wait_all(&B.s_full[x], t >> 1);
            if (!ok) break;
            hs::tc::fence_after_sync();
            float v[64];
#pragma unroll
            for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + c * 32, v + c * 32);
            if (first) {
                // (0 would turn masked places into NaN; 2^-126 does not show.)
                if constexpr (E4) {
                    as *= pow2(-B.qexp[unit & (C::kSegRing - 1)][r]);
                    if (a.k_scale != nullptr) as *= a.k_scale[s.kvh];
                }
                as = as == 0.f ? 1.17549435e-38f : fabsf(as);
            }
            const bool part = B.tile[t & (C::kRing - 1)].y != 0;
            hs::tc::tmem_wait_ld();
            if (part) {
                uint32_t vis[4];
                cx.see(t, pos, vis);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t see = w == 0 ? vis[j] : vis[2 + j];
                    if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[32 * j + c] = keep_if(v[32 * j + c], see, 1u << c);
                }
            }
            const float own = largest(v) * as - C::kShift;
            tmem_st1(s_addr + 32, own);  // (behind P's columns)
            hs::tc::tmem_wait_st();
            hs::tc::fence_before_sync();
            meet();
            uint64_t s0 = 0, s1 = 0;
            const auto weigh = [&] {
                // Without a finite logit so far: subtract 0, every weight is
                // 0 (a NaN logit stays NaN).
                const float ref = off == -CUDART_INF_F ? 0.f : off;
                const uint64_t as2 = pair_of(as, as), ref2 = pair_of(-ref, -ref);
                s0 = s1 = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const int e = 32 * c + 2 * j;
                        const float2 y = split(fma2(pair_of(v[e], v[e + 1]), as2, ref2));
                        const float2 z = split(fma2(pair_of(v[e + 2], v[e + 3]), as2, ref2));
                        const float2 p = make_float2(ex2(y.x), ex2(y.y)), q = make_float2(ex2(z.x), ex2(z.y));
                        s0 = add2(s0, pair_of(p.x, p.y));
                        s1 = add2(s1, pair_of(q.x, q.y));
                        pk[j] = pack<KV>(p.x, p.y);
                        pk[j + 1] = pack<KV>(q.x, q.y);
                    }
                    tmem_st16u(s_addr + c * 16, pk);
                }
            };
            // Mostly the reference stays, and these weights stand.
            if (!first) weigh();
            ok = cx.wait_all(pair, met++);
            if (!ok) break;
            hs::tc::fence_after_sync();
            const float other = __uint_as_float(tmem_ld1(rows + uint32_t(x * 128 + (1 - w) * 64 + 32)));
            hs::tc::tmem_wait_ld();
            const float top = fmaxf(own, other);
            const bool grow = top > off + C::kThresh || (off == -CUDART_INF_F && top > off);
            if (first) {
                if (grow) off = top;
                weigh();
            } else if (__any_sync(0xffffffffu, grow)) {
                // What has been summed is scaled down.
                const float to = grow ? top : off;
                const float al = grow ? (off == -CUDART_INF_F ? 0.f : ex2(off - to)) : 1.f;
                off = to;
                l0 = fma2(l0, pair_of(al, al), 0);
                l1 = fma2(l1, pair_of(al, al), 0);
                ok = cx.pv_wait(0, t - 1);
                if (!ok) break;
                hs::tc::fence_after_sync();
#pragma unroll 1
                for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += 16) {
                    float o[16];
                    hs::tc::tmem_ld16(o_addr + uint32_t(c), o);
                    hs::tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] *= al;
                    hs::tc::tmem_st16(o_addr + uint32_t(c), o);
                }
                weigh();
            }
            l0 = add2(l0, s0);
            l1 = add2(l1, s1);
            hs::tc::tmem_wait_st();
            hs::tc::fence_before_sync();
            hs::mbar_arrive(&B.p_full[x]);
            if (part && w < C::kSubs) {
                // Rows of V that were taken out, into the queries that see them:
                // a ring unit's dims each.
                const int turn = turn_of<C>(t, w);
                ok = cx.wait_all(&B.ready[turn % NS], turn / NS);
                const uint4* o = reinterpret_cast<const uint4*>(B.odd[t & (C::kRing - 1)][w]);
                uint32_t any = 0;
#pragma unroll
                for (int g = 0; g < C::kOddWords / 4; ++g) any |= o[g].x | o[g].y | o[g].z | o[g].w;
                if (any != 0 && ok) {
                    ok = cx.pv_wait(0, t);
                    hs::tc::fence_after_sync();
                    uint32_t vis[4];
                    cx.see(t, pos, vis);
                    add_odd_rows<KV, D, C::kOddWords, true>(
                        &a, &B.odd[t & (C::kRing - 1)][0][0][0],
                        make_uint4(vis[0], vis[1], vis[2], vis[3]), B.tile[t & (C::kRing - 1)].x,
                        s.row, s.kvh, o_addr, rows + uint32_t(x * 128), w);
                }
                if (!ok) break;
            }
            hs::mbar_arrive(&B.s_free[x]);
        }
        if (!ok) break;
        // ---- The unit's state: its output is written by another warpgroup ----
        if (unit > 0) ok = cx.wait_all(&B.o_free[0], unit - 1);
        if (!ok) break;
        const float2 ls = split(add2(l0, l1));
        float l = ls.x + ls.y;
        if (w == 1) B.factor[0][r] = l;
        meet();
        ok = cx.wait_all(pair, met++);
        if (!ok) break;
        if (w == 0) {
            l += B.factor[0][r];
            const bool live = tok < a.tq && tok < s.m;
            float f = 1.f;
            if (s.slot < 0) {
                f = l == 0.f ? 0.f : 1.f / l;
                if (a.v_scale != nullptr && l != 0.f) f *= a.v_scale[s.kvh];
                if (live && a.lse != nullptr)
                    a.lse[int64_t(s.first + tok) * a.heads + s.kvh * a.group + hd] =
                        l == 0.f ? -CUDART_INF_F : (off + log2f(l)) * kLn2;
            } else if (live) {
                reinterpret_cast<float2*>(a.part_ml)[int64_t(s.slot) * a.unit_rows + r] =
                    make_float2(off, l);
            }
            B.factor[0][r] = f;
        }
        hs::tc::fence_before_sync();
        hs::mbar_arrive(&B.l_full[0]);
    }
    if (!ok) cx.give_up();
}

// -------------------------------- products --------------------------------
// Products and commits are the bound of a warp that issues them all (3600 cycles
// for a pair of tiles whose products take 2048): one issues QK, one PV.  Two
// query tiles share S, whose softmax begins by taking it into registers, and
// have a P each: the QK of one runs ahead of the PV of the other, and a tile has
// the time of both tiles' products for its softmax.  (With S and P of a tile in
// the same columns QK has to wait for PV and the softmax is on the products'
// path.)
constexpr uint32_t kNegateA = 1u << 13;  // of the instruction descriptor
template <typename C>
__device__ __forceinline__ bool qk_role(const Cta<C>& cx) {
    constexpr int NQ = C::NQ, NS = C::NS, kSubs = C::kSubs, KV = C::kKind;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const uint32_t tmem = cx.tmem, sb = cx.sb;
    bool ok = true;
    Seg s;
    const uint64_t q_desc = hs::tc::sdesc_sw128(sb, 16, 1024);
    const uint64_t k_desc = hs::tc::sdesc_sw128(sb + C::kRingOff, 16, 1024);
    int t = 0, segs = 0, n_qk = 0;
    for (; cx.next_unit(segs, s, ok); ++segs) {
        const int n = s.n;
        const int tiles = NQ == 2 && a.tq < s.m ? 2 : 1;
        ok = ok && cx.wait_all(&B.q_full, segs);
        // A negative scale: the products with -Q.
        const bool neg = (a.scale_log2 < 0.f) !=
                         (C::kE4 && a.k_scale != nullptr && a.k_scale[s.kvh] < 0.f);
        const uint32_t id = idesc<KV>(kTile, 0) | (neg ? kNegateA : 0u);
        for (int i = 0; i < n && ok; ++i, ++t) {
            uint32_t at[kSubs];
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
                const int q = turn_of<C>(t, u);
                at[u] = uint32_t(unit_of<C>(t, false, u) % NS * (C::kUnit >> 4));
                ok = ok && cx.wait_all(&B.kfull[q % NS], q / NS);
            }
            for (int w = 0; w < tiles; ++w, ++n_qk) {
                const int x = NQ == 2 ? 0 : t & 1;
                // The last softmax has taken S; or the last product of this
                // buffer's P is done, and its softmax needs P no more.
                if (NQ == 2) {
                    if (n_qk > 0) ok = ok && cx.wait_all(&B.s_free[0], n_qk - 1);
                } else if (t >= 2) {
                    ok = ok && cx.wait_all(&B.pv_done[x], (t - 2) >> 1);
                    ok = ok && cx.wait_all(&B.s_free[x], (t - 2) >> 1);
                }
                hs::tc::fence_after_sync();
                if (!ok) break;
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int b = 0; b < C::kDims / 64; ++b)
                        mma_ss4(tmem + uint32_t(x * 128),
                                q_desc + uint32_t(w * (C::kQTile >> 4) +
                                                  (u * (C::kDims / 64) + b) * (kBlk >> 4)),
                                k_desc + at[u] + uint32_t(b * (kBlk >> 4)), id,
                                (u | b) ? 1u : 0u);
                commit(&B.s_full[NQ == 2 ? w : x]);
            }
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kSubs; ++u) commit(&B.empty[unit_of<C>(t, false, u) % NS]);
            if (i + 1 == n) commit(&B.q_empty);
        }
    }
    return ok;
}
template <typename C>
__device__ __forceinline__ bool pv_role(const Cta<C>& cx) {
    constexpr int NQ = C::NQ, NS = C::NS, kSubs = C::kSubs, KV = C::kKind;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const uint32_t tmem = cx.tmem, sb = cx.sb;
    bool ok = true;
    Seg s;
    constexpr uint32_t id = idesc<KV>(C::kDims, 1);
    const uint64_t v_desc = hs::tc::sdesc_sw128(sb + C::kRingOff, kBlk, 1024);
    int t = 0, done0 = 0, done1 = 0, had0 = 0, had1 = 0;
    for (int unit = 0; cx.next_unit(unit, s, ok); ++unit) {
        const int n = s.n;
        const int tiles = NQ == 2 && a.tq < s.m ? 2 : 1;
        // The outputs before have been read.
        if (had0 > 0) ok = ok && cx.wait_all(&B.o_free[0], had0 - 1);
        if (tiles == 2 && had1 > 0) ok = ok && cx.wait_all(&B.o_free[1], had1 - 1);
        ++had0;
        if (tiles == 2) ++had1;
        for (int i = 0; i < n && ok; ++i, ++t) {
            uint32_t at[kSubs];
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
                const int q = turn_of<C>(t, u);
                at[u] = uint32_t(unit_of<C>(t, true, u) % NS * (C::kUnit >> 4));
                ok = ok && cx.wait_all(&B.ready[q % NS], q / NS);
            }
            for (int w = 0; w < tiles; ++w) {
                const int x = NQ == 2 ? w : t & 1;
                ok = ok && cx.wait_all(&B.p_full[x], NQ == 2 ? (w == 0 ? done0 : done1) : t >> 1);
                hs::tc::fence_after_sync();
                if (!ok) break;
                const bool fresh = i == 0;
                const uint32_t p_col =
                    tmem + (NQ == 2 ? C::kPCol + uint32_t(w * 64) : uint32_t(x * 128));
#pragma unroll
                for (int u = 0; u < kSubs; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma_ts4(tmem + C::kOCol + uint32_t((w + u) * 128),
                                p_col + uint32_t(h * (NQ == 2 ? 32 : 64)),
                                v_desc + at[u] + uint32_t(h * 512), id,
                                fresh && h == 0 ? 0u : 1u);
                commit(&B.pv_done[x]);
                if (w == 0) ++done0;
                else ++done1;
            }
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kSubs; ++u) commit(&B.empty[unit_of<C>(t, true, u) % NS]);
        }
    }
    return ok;
}

// ------------------------------ loads by TMA ------------------------------
// One warp: the queries of each unit, then the K and V units of its tiles, a lane per run of tokens in one page.
template <typename C>
__device__ __forceinline__ bool tma_role(const Cta<C>& cx, const CUtensorMap& qmap,
                                         const CUtensorMap& kmap, const CUtensorMap& vmap) {
    constexpr int kSubs = C::kSubs;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int lane = threadIdx.x & 31, bt = cx.ta.bt;
    const int bt_log = 31 - __clz(bt), runs = kTile >> bt_log;  // a power of two up to 16
    constexpr int kBoxes = C::kConvert ? 1 : C::kDims / 64;
    const uint32_t row_bytes = C::kConvert ? C::kDims : 128;
    const uint32_t box = uint32_t(bt) * row_bytes;
    const uint32_t q_bytes = uint32_t(a.tq * a.group) * 128u * (C::kD / 64);
    uint64_t* q_bar = C::kConvert ? &B.q_raw : &B.q_full;
    bool ok = true, bad = false;
    int t = 0, seq = 0, segs = 0;
    Seg s;
    for (int unit = 0; cx.next_unit(unit, s, ok); ++unit) {
        // A box takes the heads of a KV head for a tile's tokens: its rows are the
        // tile's.  (Tokens of other requests behind a unit's own land in rows that
        // are not written.)
        const auto load_q = [&] {
            if (unit > 0) ok = cx.wait_all(&B.q_empty, unit - 1);
            if (!ok) return;
            segs = unit + 1;
            if (lane == 0) {
                const int tiles = C::NQ == 2 && s.m > a.tq ? 2 : 1;
                hs::mbar_arrive_expect_tx(q_bar, q_bytes * tiles);
                for (int w = 0; w < tiles; ++w)
                    for (int c = 0; c < C::kD / 64; ++c)
                        tma_load_q(cx.sb + w * C::kQTile + c * kBlk, &qmap, c * 64, s.kvh * a.group,
                                   s.first + w * a.tq, q_bar);
            }
            __syncwarp();
        };
        // The first tile's units go ahead of the queries, whose place is free only
        // when the unit before has made its last logits.  (Two ring units: the
        // places of a tile's own are free by then.  More would wait for products
        // behind those logits, or for the converter, which begins with the queries.)
        constexpr int kAhead = kSubs == 1 ? 2 : 1;
        // Whether the lane's run of a tile is needed, and its page: looked up a tile
        // ahead, for it takes as long as a small tile's copies.  (Units that pass
        // through a stage have the time, and were 5 to 10 % slower so.)
        constexpr bool kLookAhead = !C::kConvert;
        bool next_wants = false;
        int next_page = -1;
        const auto look_up = [&](int i) {
            const int tok = token_of(s, i) + lane * bt;
            next_wants = lane < runs && any_sees(a, s, tok, bt);
            if (next_wants) next_page = a.block_table[s.row * a.bt_stride + block_of(a, tok)];
        };
        if (kLookAhead) look_up(0);
        if (unit == 0) load_q();
        for (int i = 0; i < s.n && ok; ++i, ++t) {
            if (!kLookAhead) look_up(i);
            const int t0 = token_of(s, i), tok = t0 + lane * bt;
            const int b = block_of(a, tok), page = next_page;
            const bool wants = next_wants, want = wants && page >= 0 && page < a.num_pages;
            if (wants && !want) bad = true;
            const uint32_t got = __ballot_sync(0xffffffffu, want);
            // (Read by the softmax of this tile, which the ring's units keep less
            // than kRing tiles behind.)
            if (lane < 4) {
                // Runs as tokens, 32 of them a lane.
                uint32_t bits = got >> ((lane * 32) >> bt_log);
                if (bt >= 32) bits = 0u - (bits & 1u);
                else if (bt == 16) bits = (bits & 1u) * 0xffffu + (bits >> 1 & 1u) * 0xffff0000u;
                else bits = ((bits & 15u) * 0x00204081u & 0x01010101u) * 0xffu;
                B.loaded[t & (C::kRing - 1)][lane] = bits;
            }
            if (lane == 4)
                B.tile[t & (C::kRing - 1)] = make_int2(t0, !all_see(a, s, t0) || got != low_bits(runs));
            __syncwarp();
            const uint32_t bytes = uint32_t(__popc(got)) * box * kBoxes;
            const int at = tok - b * a.page_size;
            for (int u = 0; u < 2 * kSubs; ++u, ++seq) {
                uint64_t* full;
                uint32_t dst;
                if constexpr (C::kConvert) {
                    const int slot = u / kSubs;  // one for K, one for V
                    ok = cx.wait_all(&B.sempty[slot], turn_of<C>(t, u % kSubs) + 1);
                    full = &B.sfull[slot];
                    dst = cx.sb + C::kStageOff + slot * C::kStage;
                } else {
                    const int slot = seq % C::NS, turn = turn_of<C>(t, u % kSubs) % C::NS;
                    ok = cx.wait_all(&B.empty[slot], seq / C::NS + 1);
                    full = u < kSubs ? &B.kfull[turn] : &B.vfull[turn];
                    dst = cx.sb + C::kRingOff + slot * C::kUnit;
                }
                if (!ok) break;
                if (lane == 0) hs::mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (want) {
#pragma unroll
                    for (int c = 0; c < kBoxes; ++c)
                        tma_load(dst + lane * box + c * kBlk, u < kSubs ? &kmap : &vmap,
                                 u % kSubs * C::kDims + c * 64, at, s.kvh, page, full);
                }
                if (kLookAhead && u == 0 && i + 1 < s.n) look_up(i + 1);
                if (i == 0 && u == kAhead - 1 && unit > 0) {
                    load_q();
                    if (!ok) {
                        ++seq;
                        break;
                    }
                }
            }
        }
    }
    // No copy may outlive the CTA (where all went well each has been waited for).
    if (!ok) {
        if (segs > 0) hs::mbar_wait_bounded(q_bar, (segs - 1) & 1, cx.ta.timeout_ns, nullptr);
        if constexpr (C::kConvert) {
            for (int q = max(0, seq - 2 * kSubs); q < seq; ++q) {
                const int u = q % (2 * kSubs);
                hs::mbar_wait_bounded(&B.sfull[u / kSubs],
                                      turn_of<C>(q / (2 * kSubs), u % kSubs) & 1,
                                      cx.ta.timeout_ns, nullptr);
            }
        } else {
            for (int q = max(0, seq - C::NS); q < seq; ++q) {
                const int u = q % (2 * kSubs), turn = turn_of<C>(q / (2 * kSubs), u % kSubs);
                hs::mbar_wait_bounded(u < kSubs ? &B.kfull[turn % C::NS] : &B.vfull[turn % C::NS],
                                      (turn / C::NS) & 1, cx.ta.timeout_ns, nullptr);
            }
        }
    }
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    return ok;
}

// --------------------------- queries by threads ---------------------------
// Eight bf16 queries as fp16, raised so that their row's largest magnitude lies in
// [2^14, 2^15) (rows below 2^-112 not as far); a row is CHUNKS neighbouring lanes.
// *up: the power.
template <int CHUNKS>
__device__ __forceinline__ uint4 raise_queries(const uint4& raw, int* up) {
    uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    float f[8], mx = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
        f[2 * i] = y.x;
        f[2 * i + 1] = y.y;
        mx = max3(mx, fabsf(y.x), fabsf(y.y));
    }
#pragma unroll
    for (int o = CHUNKS / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    int e = 0;
    if (mx > 0.f && mx < CUDART_INF_F) e = min(14 - (int(__float_as_uint(mx) >> 23) - 127), 126);
    const float m = pow2(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack<kFp16>(f[2 * i] * m, f[2 * i + 1] * m);
    *up = e;
    return make_uint4(u[0], u[1], u[2], u[3]);
}
// The rows of a unit's queries, by THREADS threads (whole warps): 16-bit ones
// copied, bf16 ones of E4M3 caches made fp16.
template <typename C, int THREADS>
__device__ __forceinline__ void load_queries(const Cta<C>& cx, const Seg& s, int ti, int slot) {
    constexpr int D = C::kD;
    const PrefillArgs& a = cx.a;
    const int lane = ti & 31;
    constexpr int kCh = D / 8;  // 16-byte chunks of a row: a lane each
    constexpr int kRowStep = THREADS / kCh;
    const int ch = lane % kCh, row0 = ti / 32 * (32 / kCh) + lane / kCh;
    // Token and head of a row without a division each.
    const int hstep = kRowStep % a.group, tstep = kRowStep / a.group;
    const int tok0 = row0 / a.group, hd0 = row0 - tok0 * a.group;
    const char* q = static_cast<const char*>(a.q) +
                    (s.first * a.q_stride + int64_t(s.kvh) * a.group * D + ch * 8) * 2;
#pragma unroll 1
    for (int w = 0; w < C::NQ; ++w) {
        int tok = tok0, hd = hd0;
#pragma unroll 1
        for (int r = row0; r < kTile; r += kRowStep) {
            const bool in = tok < a.tq && w * a.tq + tok < s.m;
            const int64_t at = in ? (w * a.tq + tok) * a.q_stride + hd * D : 0;
            const uint32_t dst = w * C::kQTile + (ch >> 3) * kBlk + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
            if constexpr (!C::kE4) {
                hs::tc::cp_async16(cx.sb + dst, q + at * 2, in ? 16u : 0u);
            } else {
                uint4 raw = in ? *reinterpret_cast<const uint4*>(q + at * 2) : make_uint4(0u, 0u, 0u, 0u);
                int e = 0;
                if (!a.q_is_half) raw = raise_queries<kCh>(raw, &e);
                *reinterpret_cast<uint4*>(cx.smem + dst) = raw;
                if (ch == 0) cx.B.qexp[slot & (C::kSegRing - 1)][w * kTile + r] = int8_t(e);
            }
            hd += hstep;
            tok += tstep;
            if (hd >= a.group) {
                hd -= a.group;
                ++tok;
            }
        }
    }
    if constexpr (!C::kE4) hs::tc::cp_async_wait_all();
    hs::fence_proxy_async_shared();
    hs::mbar_arrive(&cx.B.q_full);
}
// The same of queries that have landed in their place, by 128 threads.  (Loaded
// by these: 40000 cycles a unit.)
template <typename C>
__device__ __forceinline__ void convert_queries(const Cta<C>& cx, int tiles, int ti, int slot) {
    constexpr int kCh = C::kD / 8, kRowStep = 128 / kCh;
    const int lane = ti & 31, ch = lane % kCh, row0 = ti / 32 * (32 / kCh) + lane / kCh;
    int8_t* qexp = cx.B.qexp[slot & (C::kSegRing - 1)];
    if (cx.a.q_is_half) {
        for (int n = ti; n < C::NQ * kTile; n += 128) qexp[n] = 0;
    } else {
#pragma unroll 4
        for (int n = row0; n < tiles * kTile; n += kRowStep) {
            const int w = n / kTile, r = n % kTile;
            uint4* at = reinterpret_cast<uint4*>(cx.smem + w * C::kQTile + (ch >> 3) * kBlk + r * 128 +
                                                 (((ch & 7) ^ (r & 7)) << 4));
            int e;
            *at = raise_queries<kCh>(*at, &e);
            if (ch == 0) qexp[n] = int8_t(e);
        }
    }
    hs::fence_proxy_async_shared();
    hs::mbar_arrive(&cx.B.q_full);
}
template <typename C>
__device__ __forceinline__ bool query_role(const Cta<C>& cx) {
    const int ti = threadIdx.x - kTmaWarp * 32;
    bool ok = true;
    Seg s;
    for (int unit = 0; cx.next_unit(unit, s, ok); ++unit) {
        if (unit > 0) ok = cx.wait_all(&cx.B.q_empty, unit - 1);
        if (ok) load_queries<C, kQThreads>(cx, s, ti, unit);
    }
    return ok;
}

// --------------------------------- output ---------------------------------
// The fourth warpgroup writes a unit's output (or partial state) while the
// softmax is at the next unit's tiles.
struct Written {
    int n = 0;              // tiles of the unit; 0: none to write
    int tiles, m, kvh;      // query tiles, tokens
    int first, slot;        // first token; slot of the partial state, -1: whole
    int units[2] = {0, 0}, products[2] = {0, 0};  // of each query tile, up to this unit
};
__device__ __forceinline__ void unit_to_write(const Seg& s, int tiles, Written& d) {
    d.n = s.n;
    d.tiles = tiles;
    d.m = s.m;
    d.kvh = s.kvh;
    d.first = s.first;
    d.slot = s.slot;
#pragma unroll
    for (int w = 0; w < 2; ++w)
        if (w < tiles) {
            ++d.units[w];
            d.products[w] += s.n;
        }
}
template <typename C>
__device__ __forceinline__ bool write_unit(const Cta<C>& cx, const Written& d) {
    constexpr int D = C::kD;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t((r >> 5) * 32) << 16;
    const int tok = r / a.group, hd = r - tok * a.group;
    const bool bf = C::kKind == kBf16 || (C::kE4 && !a.q_is_half);
#pragma unroll 1
    for (int w = 0; w < d.tiles; ++w) {
        if (!cx.wait_all(&B.l_full[w], d.units[w] - 1) || !cx.pv_wait(w, d.products[w] - 1))
            return false;
        hs::tc::fence_after_sync();
        const uint32_t o_addr = cx.tmem + lanes + C::kOCol + uint32_t(w * 128);
        const bool live = tok < a.tq && w * a.tq + tok < d.m;
        const float f = B.factor[w][r];
        const int64_t qh = int64_t(d.first + w * a.tq + tok) * a.heads + d.kvh * a.group + hd;
        uint16_t* to = static_cast<uint16_t*>(a.out) + qh * D;
        float* po = a.part_o + (int64_t(d.slot) * (D / 8) * a.unit_rows + w * kTile + r) * 8;
        // A row per thread: 32 bytes of each of 32 rows at a time.  (Pieces
        // exchanged between lanes for whole lines: five times as long.)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(o_addr + uint32_t(c), o);
            hs::tc::tmem_wait_ld();
            if (c + 32 == D) {
                hs::tc::fence_before_sync();
                hs::mbar_arrive(&B.o_free[w]);
            }
            if (!live) continue;
            if (d.slot >= 0) {
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(o[j + e]);
                    store32(po + int64_t((c + j) / 8) * a.unit_rows * 8, y);
                }
                continue;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = f == 0.f ? 0.f : o[j] * f;
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
                uint32_t y[8];
                if (bf) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = pack<kBf16>(o[j + 2 * e], o[j + 2 * e + 1]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = pack<kFp16>(o[j + 2 * e], o[j + 2 * e + 1]);
                }
                if (a.out_wide) {
                    store32(to + c + j, y);
                } else {
                    reinterpret_cast<uint4*>(to + c + j)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                    reinterpret_cast<uint4*>(to + c + j)[1] = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
        }
    }
    return true;
}

// ------------------------------- rows of V --------------------------------
// 16-bit caches by TMA: V's units pass through here, for the rows that have to
// be cleared.
template <typename C>
__device__ __forceinline__ bool check_role(const Cta<C>& cx) {
    constexpr int NS = C::NS;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int lane = threadIdx.x & 31, j = (threadIdx.x >> 5) & 3;
    bool ok = true;
    int t = 0;
    Written done;
    Seg s;
    bool more = true;
    for (int unit = 0; more; ++unit) {
        more = cx.next_unit(unit, s, ok);
        const int n = more ? s.n : 1;  // (behind the last unit: its output)
        for (int i = 0; i < n && ok; ++i, ++t) {
            for (int u = 0; u < C::kSubs && more; ++u) {
                const int q = unit_of<C>(t, true, u), turn = turn_of<C>(t, u);
                ok = cx.wait_all(&B.vfull[turn % NS], turn / NS);
                if (!ok) break;
                const int2 tile = B.tile[t & (C::kRing - 1)];
                if (tile.y != 0) {
                    const int r = j * 32 + lane;
                    const bool in = any_sees(a, s, tile.x + r) &&
                                    ((B.loaded[t & (C::kRing - 1)][j] >> lane) & 1u);
                    unsigned char* row = cx.smem + C::kRingOff + q % NS * C::kUnit + r * 128;
                    bool odd = false;
                    // (Rolled: fetching the unrolled code took 4000 cycles a unit.)
                    if (in)
#pragma unroll 2
                        for (int c = 0; c < C::kDims / 8; ++c)
                            odd |= not_finite<C::kKind>(*reinterpret_cast<const uint4*>(
                                row + (c >> 3) * kBlk + (((c + lane) & 7) << 4)));
                    const uint32_t all = __ballot_sync(0xffffffffu, odd);
                    if (lane == 0) B.odd[t & (C::kRing - 1)][u][0][j] = all;
                    if (!in || odd)
#pragma unroll 2
                        for (int c = 0; c < C::kDims / 8; ++c)
                            *reinterpret_cast<uint4*>(row + (c >> 3) * kBlk + (((c + lane) & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    hs::fence_proxy_async_shared();
                }
                __syncwarp();
                if (lane == 0) hs::mbar_arrive(&B.ready[turn % NS]);
            }
            // The unit before, while this one's first tile is in its softmax.
            if (ok && i == 0 && done.n > 0) ok = write_unit(cx, done);
        }
        if (more) unit_to_write(s, C::NQ == 2 && a.tq < s.m ? 2 : 1, done);
    }
    return ok;
}

// Eight E4M3 codes as fp16.
__device__ __forceinline__ uint4 widen_codes(const uint2& x) {
    return make_uint4(e4m3x2_to_half2(x.x & 0xffffu), e4m3x2_to_half2(x.x >> 16),
                      e4m3x2_to_half2(x.y & 0xffffu), e4m3x2_to_half2(x.y >> 16));
}
// Lanes of a warp that hold the chunks of this lane's row.
template <int CHUNKS>
__device__ __forceinline__ uint32_t row_lanes(int lane) {
    return CHUNKS >= 32 ? 0xffffffffu : ((1u << (CHUNKS & 31)) - 1u) << (lane / CHUNKS * CHUNKS);
}

// E4M3 caches by TMA: units from the stages (one for K, one for V) to the ring as
// fp16.
template <typename C>
__device__ __forceinline__ bool convert_role(const Cta<C>& cx) {
    constexpr int NS = C::NS, kCh = C::kDims / 16;  // chunks of a row
    constexpr int kStep = kTile / kCh;              // rows of a pass
    static_assert(kStep % 8 == 0, "the swizzle is the same in every pass");
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int lt = threadIdx.x & 127, lane = lt & 31, ch = lt % kCh, r0 = lt / kCh;
    // Its 16 codes make two 16-byte chunks of fp16; half the lanes begin with the
    // second one, for the banks.
    const int swap = ch >= 4 ? 1 : 0, c0 = 2 * ch + swap, c1 = 2 * ch + 1 - swap;
    const int to0 = r0 * 128 + (c0 >> 3) * kBlk + (((c0 & 7) ^ (r0 & 7)) << 4);
    const int to1 = r0 * 128 + (c1 >> 3) * kBlk + (((c1 & 7) ^ (r0 & 7)) << 4);
    const unsigned char* from = cx.smem + C::kStageOff + lt * 16;
    bool ok = true;
    int t = 0;
    Written done;
    Seg s;
    const auto take = [&](int side, uint2 (&x)[kCh][2]) {
#pragma unroll
        for (int p = 0; p < kCh; ++p) {
            const unsigned char* at = from + side * C::kStage + p * kStep * C::kDims;
            x[p][0] = *reinterpret_cast<const uint2*>(at + swap * 8);
            x[p][1] = *reinterpret_cast<const uint2*>(at + 8 - swap * 8);
        }
        hs::mbar_arrive(&B.sempty[side]);
    };
    const auto put = [&](int slot, const uint2 (&x)[kCh][2]) {
        unsigned char* to = cx.smem + C::kRingOff + slot * C::kUnit;
#pragma unroll
        for (int p = 0; p < kCh; ++p) {
            *reinterpret_cast<uint4*>(to + to0 + p * kStep * 128) = widen_codes(x[p][0]);
            *reinterpret_cast<uint4*>(to + to1 + p * kStep * 128) = widen_codes(x[p][1]);
        }
        hs::fence_proxy_async_shared();
    };
    bool more = true;
    for (int unit = 0; more; ++unit) {
        more = cx.next_unit(unit, s, ok);
        if (more) ok = cx.wait_all(&B.q_raw, unit);
        if (!ok) break;
        if (more) convert_queries<C>(cx, C::NQ == 2 && a.tq < s.m ? 2 : 1, lt, unit);
        const int n = more ? s.n : 1;  // (behind the last unit: its output)
        for (int i = 0; i < n && ok; ++i, ++t) {
            // K's units, then V's, whose codes are taken early where a tile has one.
            uint2 x[kCh][2], y[kCh][2];
#pragma unroll
            for (int u = 0; u < C::kSubs && more; ++u) {
                const int turn = turn_of<C>(t, u), seq = unit_of<C>(t, false, u);
                ok = ok && cx.wait_all(&B.sfull[0], turn) &&
                     cx.wait_all(&B.empty[seq % NS], seq / NS + 1);
                if (!ok) break;
                take(0, x);
                if (C::kSubs == 1) {
                    ok = cx.wait_all(&B.sfull[1], turn);
                    take(1, y);
                }
                put(seq % NS, x);
                hs::mbar_arrive(&B.kfull[turn % NS]);
            }
#pragma unroll
            for (int u = 0; u < C::kSubs && more; ++u) {
                const int turn = turn_of<C>(t, u), seq = unit_of<C>(t, true, u);
                if (C::kSubs > 1) {
                    ok = ok && cx.wait_all(&B.sfull[1], turn);
                    if (ok) take(1, y);
                }
                ok = ok && cx.wait_all(&B.empty[seq % NS], seq / NS + 1);
                if (!ok) break;
                const int2 tile = B.tile[t & (C::kRing - 1)];
                if (tile.y != 0) {
                    uint32_t odd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int p = 0; p < kCh; ++p) {
                        const int r = p * kStep + r0;
                        const bool in = any_sees(a, s, tile.x + r) &&
                                        ((B.loaded[t & (C::kRing - 1)][r >> 5] >> (r & 31)) & 1u);
                        const uint32_t bad = __ballot_sync(
                            0xffffffffu, in && not_finite<kE4m3>(make_uint4(
                                                   y[p][0].x, y[p][0].y, y[p][1].x, y[p][1].y)));
                        const bool out = (bad & row_lanes<kCh>(lane)) != 0;
                        if (!in || out) y[p][0] = y[p][1] = make_uint2(0u, 0u);
                        if (out && ch == 0) odd[p * kStep >> 5] |= 1u << (r & 31);
                    }
                    // What each warp has found of its rows: a quarter of every word.
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t all = __reduce_or_sync(0xffffffffu, odd[g]);
                        if (lane == 0) B.odd[t & (C::kRing - 1)][u][lt >> 5][g] = all;
                    }
                }
                put(seq % NS, y);
                hs::mbar_arrive(&B.ready[turn % NS]);
            }
            if (ok && i == 0 && done.n > 0) ok = write_unit(cx, done);
        }
        if (more) unit_to_write(s, C::NQ == 2 && a.tq < s.m ? 2 : 1, done);
    }
    return ok;
}

// Loads by 128 threads: pages without runs of 8 tokens, broadcast strides.
template <typename C>
__device__ __forceinline__ bool load_role(const Cta<C>& cx) {
    constexpr bool E4 = C::kE4;
    constexpr int D = C::kD;
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    unsigned char* smem = cx.smem;
    const int lt = threadIdx.x & 127, lane = lt & 31;
    Seg s;
    constexpr int kElt = E4 ? 1 : 2, kPer = 16 / kElt;  // elements of 16 bytes
    constexpr int kCh = D / kPer;                       // 16-byte chunks of a row
    constexpr int kStep = kTile / kCh;                  // rows of a pass
    constexpr int kPass = kCh < 8 ? kCh : 8;            // passes of a batch
    constexpr int kBatch = kPass * kStep, kBatches = kTile / kBatch;
    const int ch = lt % kCh, r0 = lt / kCh;
    bool ok = true, bad = false;
    int t = 0;
    uint4 buf[2][kPass];
    const auto rows_of = [&](int t, int i) {
        // Row lt of the tile: where it lies in the cache.
        const int tok = token_of(s, i) + lt, b = block_of(a, tok);
        int64_t at = -1;
        if (any_sees(a, s, tok)) {
            const int64_t page = a.block_table[s.row * a.bt_stride + b];
            if (page >= 0 && page < a.num_pages)
                at = page * a.page_stride + int64_t(tok - b * a.page_size) * a.row_stride +
                     s.kvh * a.head_stride;
            else
                bad = true;
        }
        B.offset[t & 1][lt] = at;
        const uint32_t got = __ballot_sync(0xffffffffu, at >= 0);
        if (lane == 0) {
            B.loaded[t & (C::kRing - 1)][lt >> 5] = got;
            for (int u = 0; u < C::kSubs; ++u) B.odd[t & (C::kRing - 1)][u][0][lt >> 5] = 0;
        }
        hs::pair::named_sync(kLoadBar, kTile);
    };
    const auto load = [&](int t, bool v, int batch, uint4 (&x)[kPass]) {
        const char* base = static_cast<const char*>(v ? a.v : a.k) + ch * 16;
#pragma unroll
        for (int j = 0; j < kPass; ++j) {
            const int64_t at = B.offset[t & 1][batch * kBatch + j * kStep + r0];
            x[j] = at >= 0 ? *reinterpret_cast<const uint4*>(base + at * kElt)
                           : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    const auto store = [&](int t, bool v, int batch, uint4 (&x)[kPass], bool part) {
#pragma unroll
        for (int j = 0; j < kPass; ++j) {
            const int r = batch * kBatch + j * kStep + r0;
            if (v && part) {
                // A row's chunks lie in neighbouring lanes of one warp.
                const uint32_t odd = __ballot_sync(0xffffffffu, not_finite<C::kKind>(x[j]));
                const uint32_t mine = (kCh == 32 ? 0xffffffffu : ((1u << (kCh & 31)) - 1u) << (lane / kCh * kCh));
                if (odd & mine) {
                    x[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (ch == 0)
                        for (int u = 0; u < C::kSubs; ++u)
                            atomicOr(&B.odd[t & (C::kRing - 1)][u][0][r >> 5], 1u << (r & 31));
                }
            }
            const int c0 = E4 ? 2 * ch : ch;  // its first chunk of eight 16-bit elements
            const int u = c0 * 8 / C::kDims, cb = c0 - u * (C::kDims / 8);
            unsigned char* dst = smem + C::kRingOff + unit_of<C>(t, v, u) % C::NS * C::kUnit +
                                 (cb >> 3) * kBlk + r * 128;
            if constexpr (E4) {
                const uint4 y = widen_codes(make_uint2(x[j].x, x[j].y)), z = widen_codes(make_uint2(x[j].z, x[j].w));
                *reinterpret_cast<uint4*>(dst + (((cb & 7) ^ (r & 7)) << 4)) = y;
                *reinterpret_cast<uint4*>(dst + ((((cb & 7) + 1) ^ (r & 7)) << 4)) = z;
            } else {
                *reinterpret_cast<uint4*>(dst + (((cb & 7) ^ (r & 7)) << 4)) = x[j];
            }
        }
    };
    const auto wait_empty = [&](int t, bool v) {
        bool fine = ok;
        for (int u = 0; u < C::kSubs; ++u) {
            const int q = unit_of<C>(t, v, u);
            fine = fine && cx.wait(&B.empty[q % C::NS], q / C::NS + 1);
        }
        // All or none go on: they meet at a barrier.
        return !hs::pair::named_sync_or(kLoadBar, kTile, !fine);
    };
    const auto arrive = [&](int t, bool v) {
        hs::fence_proxy_async_shared();
        for (int u = 0; u < C::kSubs; ++u) {
            const int q = turn_of<C>(t, u) % C::NS;
            hs::mbar_arrive(v ? &B.ready[q] : &B.kfull[q]);
        }
    };
    Written done;
    bool run = true;  // alike in all threads
    for (int unit = 0; run; ++unit) {
        // (All or none: they meet at barriers.)
        bool more = cx.next_unit(unit, s, ok);
        run = !hs::pair::named_sync_or(kLoadBar, kTile, !ok);
        if (!run || !more) break;
        rows_of(t, 0);
        load(t, false, 0, buf[0]);
        for (int i = 0; i < s.n && run; ++i, ++t) {
            const uint4 ld = *reinterpret_cast<const uint4*>(B.loaded[t & (C::kRing - 1)]);
            const bool part = !all_see(a, s, token_of(s, i)) ||
                              (ld.x & ld.y & ld.z & ld.w) != 0xffffffffu;
            if (lt == 0) B.tile[t & (C::kRing - 1)] = make_int2(token_of(s, i), part);
            // Batches of K, then of V; each is loaded while the one before it is
            // stored.
#pragma unroll
            for (int j = 0; j < 2 * kBatches; ++j) {
                const bool v = j >= kBatches;
                if (j % kBatches == 0 && run) run = wait_empty(t, v);
                if (j + 1 < 2 * kBatches) {
                    load(t, j + 1 >= kBatches, (j + 1) % kBatches, buf[(j + 1) & 1]);
                } else if (i + 1 < s.n) {
                    rows_of(t + 1, i + 1);
                    load(t + 1, false, 0, buf[0]);
                }
                if (run) {
                    store(t, v, j % kBatches, buf[j & 1], part);
                    if ((j + 1) % kBatches == 0) arrive(t, v);
                }
            }
            // (A warp that gives up says so where all meet next.)
            if (run && i == 0 && done.n > 0) ok = write_unit(cx, done) && ok;
        }
        unit_to_write(s, C::NQ == 2 && a.tq < s.m ? 2 : 1, done);
    }
    ok = ok && run;
    if (ok && done.n > 0) ok = write_unit(cx, done);
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    return ok;
}

// --------------------------------- units ----------------------------------
// Walks the run's units.
template <typename C>
__device__ __forceinline__ bool plan_role(const Cta<C>& cx) {
    const PrefillArgs& a = cx.a;
    Bars<C>& B = cx.B;
    const int lane = threadIdx.x & 31;
    constexpr uint32_t kAll = 0xffffffffu;
    // The run: the call's places, dealt to the CTAs, a lane per request.
    int64_t total = 0;
    bool falls = false, blind = false;
#pragma unroll 2
    for (int r = lane; r < a.rows; r += 32) {
        const Request x = request_of(a, r);
        total += places_of(a, x);
        blind |= x.blind > 0;
        falls |= a.cu_new[r + 1] < a.cu_new[r];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    // Requests that overlap would both write their rows: none does.
    falls = __any_sync(kAll, falls);
    if (falls) total = 0;
    const int64_t per = quotient(total, a.ctas);
    const int rest = int(total - per * a.ctas);
    const int64_t place0 = run_begin(per, rest, blockIdx.x);
    const int64_t place1 = run_begin(per, rest, blockIdx.x + 1);
    // The unit that it begins in.
    int64_t start = 0;
    int row = 0, kvh = 0, block = 0, unit = 0;
    SharedUnit shared{};
    shared.blind = __any_sync(kAll, blind) && !falls;
    if (place0 < place1) {
        for (int64_t before = 0;; row += 32) {
            const int r = row + lane;
            const int64_t own = r < a.rows ? places_of(a, request_of(a, r)) : 0;
            int64_t upto = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(kAll, upto, d);
                if (lane >= d) upto += o;
            }
            upto += before;
            const uint32_t past = __ballot_sync(kAll, upto > place0);
            before = __shfl_sync(kAll, upto, 31);
            if (past != 0) {
                const int at = __ffs(past) - 1;
                start = __shfl_sync(kAll, upto - own, at);
                row += at;
                break;
            }
            if (row + 32 >= a.rows) break;  // (cannot be)
        }
        const Request x = request_of(a, row);
        const int64_t each = places(a, x, blocks_of(a, x.n));
        for (; kvh + 32 < a.kv_heads; kvh += 32)
            if (start + (kvh + 32) * each > place0) break;
        kvh += __popc(__ballot_sync(kAll, kvh + lane + 1 < a.kv_heads &&
                                              start + (kvh + lane + 1) * each <= place0));
        start += kvh * each;
        int hi = blocks_of(a, x.n);
        while (hi - block > 1) {
            const int mid = (block + hi) >> 1;
            if (places(a, x, mid) <= place0 - start) block = mid;
            else hi = mid;
        }
        start += places(a, x, block);
    }
    bool ok = true;
    const auto publish = [&](const Seg& s) {
        if (unit >= kUnitRing)
            ok = cx.wait_all(&B.unit_free[unit % kUnitRing], unit / kUnitRing - 1);
        if (ok && lane == 0) {
            B.unit[unit % kUnitRing] = s;
            hs::mbar_arrive(&B.unit_full[unit % kUnitRing]);
        }
        __syncwarp();
        ++unit;
    };
    if (place0 < place1) {
        Request x = request_of(a, row);
        int blocks = blocks_of(a, x.n);
        while (ok) {
            Seg s;
            s.row = row;
            s.kvh = kvh;
            s.first = x.first + block * a.tb;
            s.m = min(a.tb, x.n - block * a.tb);
            s.p0 = x.T - x.n + block * a.tb;
            const int hi = s.p0 + s.m;  // tokens up to the last query's own
            const int lo = a.window > 0 ? max(0, s.p0 + 1 - a.window) : 0;
            s.tw = min(lo, hi) / kTile;
            const int sc = a.window > 0 ? min(a.sinks, lo) : 0;
            s.ns = min((sc + kTile - 1) / kTile, s.tw);
            const int nt = s.ns + (hi + kTile - 1) / kTile - s.tw;
            const int cost = cost_of(a, x, block);
            s.i0 = tile_at(place0 - start, cost, nt);
            const int i1 = tile_at(place1 - start, cost, nt);
            s.n = i1 - s.i0;
            s.slot = s.i0 == 0 && i1 == nt ? -1 : 2 * int(blockIdx.x) + (start < place0 ? 0 : 1);
            if (s.n > 0) {
                if (start < place0) shared.cont = s.n;
                if (s.slot >= 0 && s.i0 == 0) {
                    shared.valid = 1;
                    shared.slot = s.slot;
                    shared.first = s.first;
                    shared.tokens = s.m;
                    shared.kvh = kvh;
                    for (int c = blockIdx.x + 1;; c += 32) {
                        const uint32_t in = __ballot_sync(
                            kAll, c + lane < a.ctas && run_begin(per, rest, c + lane) < start + cost);
                        shared.last = c - 1 + __popc(in);
                        if (in != kAll) break;
                    }
                }
                publish(s);
            }
            start += cost;
            if (start >= place1) break;
            if (++block < blocks) continue;
            block = 0;
            if (++kvh < a.kv_heads) continue;
            kvh = 0;
            do {  // the next request with a query that attends; there is one
                if (++row >= a.rows) break;
                x = request_of(a, row);
            } while (x.n == 0);
            if (row >= a.rows) break;
            blocks = blocks_of(a, x.n);
        }
    }
    if (ok) {
        Seg end{};
        publish(end);
    }
    if (lane == 0) a.shared[blockIdx.x] = shared;
    return ok;
}

template <int KV, int D, int LD, int QT>
__global__ void __launch_bounds__(kThreads, 1)
prefill_tc_kernel(const __grid_constant__ TcArgs ta, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<KV, D, LD, QT>;
    const PrefillArgs& a = ta.p;
    extern __shared__ __align__(1024) unsigned char smem[];
    Bars<C>& B = *reinterpret_cast<Bars<C>*>(smem + C::kBarOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The swizzled tiles need it (and there is no room to round up).
    if ((hs::smem_u32(smem) & 1023u) != 0) {
        hs::set_status(a.status, HS_ERR_CUDA);
        return;
    }
    constexpr int kHalves = C::NQ == 1 ? 2 : 1;  // warpgroups of a query tile
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            hs::mbar_init(&B.kfull[i], C::kByTma && !C::kConvert ? 1 : kTile);
            hs::mbar_init(&B.vfull[i], 1);
            hs::mbar_init(&B.ready[i], C::kByTma && !C::kConvert ? 4 : kTile);
            hs::mbar_init(&B.empty[i], 1);
        }
        hs::mbar_init(&B.q_full, C::kConvert ? kTile : C::kByTma ? 1 : kQThreads);
        hs::mbar_init(&B.q_raw, 1);
        hs::mbar_init(&B.q_empty, 1);
        for (uint64_t& b : B.pair) hs::mbar_init(&b, 2);
        for (int i = 0; i < 2; ++i) {
            hs::mbar_init(&B.s_full[i], 1);
            hs::mbar_init(&B.s_free[i], kHalves * kTile);
            hs::mbar_init(&B.p_full[i], kHalves * kTile);
            hs::mbar_init(&B.pv_done[i], 1);
            hs::mbar_init(&B.l_full[i], kHalves * kTile);
            hs::mbar_init(&B.o_free[i], kTile);
            hs::mbar_init(&B.drain[i], 1);
            hs::mbar_init(&B.sfull[i], 1);
            hs::mbar_init(&B.sempty[i], kTile);
        }
        for (int i = 0; i < kUnitRing; ++i) {
            hs::mbar_init(&B.unit_full[i], 1);
            hs::mbar_init(&B.unit_free[i], 8 + 3 + 4);  // a warp each
        }
        B.abort = 0;
        hs::fence_mbar_init();
    }
    if (C::kByTma && warp == kTmaWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &kmap : lane == 1 ? &vmap : &qmap)
                     : "memory");
    if (warp == kQkWarp) {
        hs::tc::tmem_alloc(&B.tmem_base, kTmemCols);
        hs::tc::tmem_relinquish();
    }
    hs::tc::fence_before_sync();
    __syncthreads();
    hs::tc::fence_after_sync();
    hs::pdl_wait();
    hs::pdl_trigger();
    if (blockIdx.x == 0)
        for (int r = tid; r < a.rows; r += kThreads) {
            const int c0 = a.cu_new[r], c1 = a.cu_new[r + 1];
            if (a.seq_lens[r] > a.max_len || c0 < 0 || c1 < c0 || c1 > a.tokens)
                hs::set_status(a.status, HS_ERR_BAD_INDEX);
        }
    const Cta<C> cx{ta, a, B, smem, hs::smem_u32(smem), B.tmem_base};
    bool ok = true;
    if (warp < 8) {
        set_max_regs_up<C::kSoftRegs>();
        if constexpr (C::NQ == 2) softmax_role<C>(cx);
        else softmax_split_role<C>(cx);
    } else if (warp < kLoadWarp) {
        set_max_regs_down<C::kMmaRegs>();
        if (warp <= kPvWarp) {
            ok = warp == kQkWarp ? qk_role<C>(cx) : pv_role<C>(cx);
            if (!ok) cx.give_up();
            // Every product issued has completed before TMEM is freed.
            __syncwarp();
            commit(&B.drain[warp - kQkWarp]);
            hs::mbar_wait_bounded(&B.drain[warp - kQkWarp], 0, ta.timeout_ns, nullptr);
            __syncwarp();
        } else if (warp == kPlanWarp) {
            if (!plan_role<C>(cx)) cx.give_up();
        } else if constexpr (C::kByTma) {
            if (!tma_role<C>(cx, qmap, kmap, vmap)) cx.give_up();
        } else {
            if (!query_role<C>(cx)) cx.give_up();
        }
    } else {
        set_max_regs_down<C::kLoadRegs>();
        if constexpr (C::kConvert) ok = convert_role<C>(cx);
        else if constexpr (C::kByTma) ok = check_role<C>(cx);
        else ok = load_role<C>(cx);
        if (!ok) cx.give_up();
    }
    hs::tc::fence_before_sync();
    __syncthreads();
    hs::tc::fence_after_sync();
    if (warp == kQkWarp) hs::tc::tmem_dealloc(cx.tmem, kTmemCols);
}

// Tensor map of a cache: dims (head dim, token of the page, KV head, page).
int encode_map(CUtensorMap* m, const void* base, const PrefillArgs& a, int kv_dtype, int d, int bt);
// Of the queries: dims (head dim, head, token), boxes of a query tile.
int encode_q_map(CUtensorMap* m, const PrefillArgs& a, int dtype, int d);

template <int KV, int D, int LD, int QT>
int launch_one(const PrefillArgs& a, int bt, hs_stream_t stream) {
    using C = Cfg<KV, D, LD, QT>;
    TcArgs t{};
    t.p = a;
    t.bt = bt;
    t.timeout_ns = hs::kWaitTimeoutNs;
    auto kern = prefill_tc_kernel<KV, D, LD, QT>;
    constexpr size_t smem = size_t(C::kBarOff) + sizeof(Bars<C>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static int smem_set[64] = {};
    int rc = hs_host::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem, smem_set);
    if (rc != HS_OK) return rc;
    // The warps' register shares (setmaxnreg) add up to what 128 a thread give.
    static int regs[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return HS_ERR_CUDA;
    const auto ask = [&] {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) == cudaSuccess) return fa.numRegs;
        cudaGetLastError();
        return -1;
    };
    if (hs_host::ask_once(&regs[dev], ask) != 65536 / kThreads) return HS_ERR_UNSUPPORTED;
    CUtensorMap q{}, k{}, v{};
    if (C::kByTma) {
        rc = encode_q_map(&q, a, C::kE4 ? (a.q_is_half ? HS_FP16 : HS_BF16) : KV, D);
        if (rc == HS_OK) rc = encode_map(&k, a.k, a, KV, D, bt);
        if (rc == HS_OK) rc = encode_map(&v, a.v, a, KV, D, bt);
        if (rc != HS_OK) return rc;
    }
    return hs_host::launch_pdl(kern, dim3(unsigned(a.ctas)), dim3(kThreads), smem, stream, t, q, k, v);
}

// bt: tokens of a TMA box, or 0: threads load.
template <int KV>
int launch_kind(const PrefillArgs& a, int d, int bt, hs_stream_t stream) {
    if (d == 256)
        return bt > 0 ? launch_one<KV, 256, kTma, 1>(a, bt, stream)
                      : launch_one<KV, 256, kThreadsLoad, 1>(a, 0, stream);
    if constexpr (KV == kE4m3)
        if (a.unit_rows == kTile)
            return d == 64 ? launch_one<KV, 64, kTma, 1>(a, bt, stream)
                           : launch_one<KV, 128, kTma, 1>(a, bt, stream);
    if (bt > 0)
        return d == 64 ? launch_one<KV, 64, kTma, 2>(a, bt, stream)
                       : launch_one<KV, 128, kTma, 2>(a, bt, stream);
    return d == 64 ? launch_one<KV, 64, kThreadsLoad, 2>(a, 0, stream)
                   : launch_one<KV, 128, kThreadsLoad, 2>(a, 0, stream);
}

}  // namespace tc

}  // namespace hs_prefill
