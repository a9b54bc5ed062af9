// hs_evict.cu -- eviction from a paged KV cache to a budget of tokens by
// running attention scores: which tokens stay (hs_evict_select), the row
// moves that close the holes (hs_evict_move), and both (hs_evict).
//
// A request of T > B tokens keeps the B first ones in the order (protected
// tokens, higher score, lower index).  Attention does not depend on the
// order of the rows, so the kept rows stay where they are: only those at
// indices >= B move, into the holes left below B, the j-th of them into the
// j-th hole.  A steady decode step (T = B + 1) moves at most one row, and no
// source is a destination, so the moves run in any order and in place.
#include <math_constants.h>

#include "hs_common.cuh"

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kDigit = 11;          // bits of a key decided in one pass
constexpr int kBins = 1 << kDigit;
constexpr int kCopies = 4;          // counters of a bin, by lane
static_assert(kBins == 2 * kThreads, "two bins a thread");
constexpr int kMaxCluster = 8;
constexpr int kCacheKeys = 40960;   // keys of a CTA's slice that shared memory keeps
// Tokens a CTA of a cluster should have at least: below that the cluster's
// barriers and remote loads cost what the shorter slice saves (32 requests of
// 32 K tokens: 16.3 us at 8192 and 4096, 18.9 at 16384, 26.1 at 32768).
constexpr int kSliceMin = 8192;
constexpr int kTrimThreads = 1024;
constexpr int kTrimKeys = 16;       // keys a thread of the trimming kernel holds
constexpr int kTrimMost = 8;        // tokens that it evicts at most
constexpr int kPlaces = 0x7fffffff;

struct EvictArgs {
    const float* score;
    int64_t score_stride;
    const int32_t* positions;  // or nullptr: the index itself
    int64_t pos_stride;
    const int32_t* seq_lens;
    const int32_t* next_pos;   // or nullptr: T
    int32_t rows, max_len, budget, recent, sinks;
    float* score_out;
    int64_t score_out_stride;
    int32_t* positions_out;    // or nullptr
    int64_t pos_out_stride;
    int32_t* lens_out;
    int32_t* move_src;         // [rows, cap]
    int32_t* move_dst;
    int32_t* move_count;       // [rows]
    int32_t cap;
    int32_t* status;
};

// ---- Cluster helpers (barrier over the cluster, loads from a peer) ---------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const int* p, uint32_t rank) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(addr)
                 : "r"(hs::smem_u32(p)), "r"(rank));
    return addr;
}
__device__ __forceinline__ int2 peer_load2(const int* p, uint32_t rank) {
    int2 v;
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ int4 peer_load4(const int* p, uint32_t rank) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
}

// Order of scores as unsigned integers: NaN below everything, the two zeros
// equal.
__device__ __forceinline__ uint32_t order_key(float s) {
    if (s != s) return 1u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kProtected = 0xffffffffu;  // above +inf's key

// One cluster per request, each CTA a contiguous slice of its tokens.  The
// B-th largest key is found by its digits of 11 bits from the top: every CTA
// counts its slice's digits (four counters a bin, by lane, since most scores
// share a few exponents), the cluster sums the counts through distributed
// shared memory, and only keys that share the chosen digits are counted
// again.  Protected tokens share one key; where they alone are more than the
// budget, all others get key 0 and the search starts again with the protected
// ones' scores.  Then each warp walks its part of the slice in order: what is kept
// before an index gives the rank of a hole or of a moving row.
__global__ void __launch_bounds__(kThreads)
evict_select_kernel(const __grid_constant__ EvictArgs a, int slice, int cached, int state) {
    extern __shared__ __align__(16) unsigned char smem[];
    int* hist = reinterpret_cast<int*>(smem);              // [kCopies][kBins]
    int* counts = hist + kCopies * kBins;                  // [2][kBins], read by the cluster
    int* totals = counts + 2 * kBins;                      // [4]: gt, eq, gt < B, eq < B (16-byte aligned)
    int* scratch = totals + 4;                             // [32]
    int* pick = scratch + 32;                              // [4]
    int* warp_n = pick + 4;                                // [kWarps][2]
    uint32_t* keys = reinterpret_cast<uint32_t*>(warp_n + 2 * kWarps);  // [slice] if cached
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ncta = cluster_size();
    const int row = blockIdx.x / ncta;

    hs::pdl_trigger();
    hs::pdl_wait();
    const float* score = a.score + int64_t(row) * a.score_stride;
    const int32_t* pos = a.positions ? a.positions + int64_t(row) * a.pos_stride : nullptr;
    float* score_out = a.score_out + int64_t(row) * a.score_out_stride;
    int32_t* pos_out =
        a.positions_out ? a.positions_out + int64_t(row) * a.pos_out_stride : nullptr;
    const bool copy_score = a.score_out != a.score;
    const bool copy_pos = pos_out != nullptr && a.positions_out != a.positions;
    // The first scores and positions are read along with the length (rows
    // hold max_len entries; those past the length are not used).
    constexpr int U = 8;
    float x[U];
    int32_t p[U];
    {
        const int e = min(a.max_len, int(rank) * slice + slice);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = int(rank) * slice + tid + u * kThreads;
            x[u] = i < e ? score[i] : 0.f;
            p[u] = pos != nullptr && i < e ? pos[i] : i;
        }
    }
    const int len = a.seq_lens[row];
    const int next = a.next_pos ? a.next_pos[row] : 0;
    const int T = min(max(len, 0), a.max_len), B = a.budget;
    const int s0 = min(T, int(rank) * slice), s1 = min(T, s0 + slice);
    if (len > a.max_len && rank == 0 && tid == 0) hs::set_status(a.status, HS_ERR_BAD_INDEX);

    if (T <= B) {  // nothing to evict (the same in every CTA of the cluster)
        for (int i = s0 + tid; i < s1; i += kThreads) {
            if (copy_score) score_out[i] = score[i];
            if (copy_pos) pos_out[i] = pos ? pos[i] : i;
        }
        cluster_sync();  // every CTA has read seq_lens (lens_out may be the same array)
        if (rank == 0 && tid == 0) {
            a.lens_out[row] = T;
            a.move_count[row] = 0;
        }
        return;
    }
    const int64_t from = int64_t(a.next_pos ? next : T) - a.recent;  // positions from here on are protected
    bool few = false;  // the budget is too small for the protected tokens
    auto key_of = [&](float s, int p) {
        const bool keep = p < a.sinks || p >= from;
        return keep == few ? order_key(s) : keep ? kProtected : 0u;
    };
    auto make_key = [&](int i) { return key_of(score[i], pos ? pos[i] : i); };
    auto key_at = [&](int i) { return cached ? keys[i - s0] : make_key(i); };

    // ---- The B-th largest key ---------------------------------------------
    uint32_t prefix = 0;  // digits chosen so far
    int need = B;         // keys still wanted among those that share them
    bool all = false;     // every key of the chosen digits is kept
    for (int pass = 0;; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;  // 11, 11 and 10 bits
        const int width = pass < 2 ? kDigit : 10;
        for (int i = tid; i < kCopies * kBins / 4; i += kThreads)
            reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
        int* column = hist + (lane & (kCopies - 1)) * kBins;
        if (pass == 0) {
            // All loads of a batch ahead of its stores (the outputs may be the
            // inputs, so the compiler keeps their order).  What stands below
            // the budget is copied on the way: a hole among it is overwritten
            // by the row that moves there.
            for (int i0 = s0 + tid; i0 < s1; i0 += U * kThreads) {
                if (few || i0 >= int(rank) * slice + U * kThreads) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = i0 + u * kThreads;
                        x[u] = i < s1 ? score[i] : 0.f;
                        p[u] = pos != nullptr && i < s1 ? pos[i] : i;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * kThreads;
                    if (i >= s1) break;
                    const uint32_t k = key_of(x[u], p[u]);
                    if (cached) keys[i - s0] = k;
                    atomicAdd(column + (k >> 21), 1);
                    if (i < B) {
                        if (copy_score) score_out[i] = x[u];
                        if (copy_pos) pos_out[i] = p[u];
                    }
                }
            }
        } else {
#pragma unroll 4
            for (int i = s0 + tid; i < s1; i += kThreads) {
                const uint32_t k = key_at(i);
                if ((k >> (shift + width)) == (prefix >> (shift + width)))
                    atomicAdd(column + ((k >> shift) & ((1u << width) - 1u)), 1);
            }
        }
        __syncthreads();
        // A thread sums two neighbouring bins; the cluster's counts of a pass
        // are read before those of the next but one are written.
        int* mine = counts + (pass & 1) * kBins;
        const int b0 = kBins - 2 * (tid + 1);  // from the largest digit down
        int2 n = make_int2(0, 0);
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            const int2 x = *reinterpret_cast<const int2*>(hist + c * kBins + b0);
            n.x += x.x;
            n.y += x.y;
        }
        if (ncta > 1) {
            *reinterpret_cast<int2*>(mine + b0) = n;
            cluster_sync();
            n = make_int2(0, 0);
            for (uint32_t c = 0; c < ncta; ++c) {
                const int2 x = peer_load2(mine + b0, c);
                n.x += x.x;
                n.y += x.y;
            }
        }
        int sum;
        const int before = hs::block_excl_scan(n.x + n.y, scratch, &sum);
        if (before < need && need <= before + n.y + n.x) {
            const bool low = need > before + n.y;  // the lower of the two bins
            const int upto = before + n.y + (low ? n.x : 0);
            pick[0] = low ? b0 : b0 + 1;
            pick[1] = need - (low ? before + n.y : before);
            pick[2] = need == upto;
        }
        __syncthreads();
        prefix |= uint32_t(pick[0]) << shift;
        need = pick[1];
        all = pick[2] != 0;
        if (all || pass == 2) break;
        if (pass == 0 && !few && pick[0] == kBins - 1) {
            // Only protected tokens have this digit.  (The same in every CTA;
            // all have read the counts before they are written again.)
            few = true;
            prefix = 0;
            need = B;
            pass = -1;
            cluster_sync();
        }
    }
    // Kept: keys above `limit`, and the first `need` of those equal to it.
    // (All keys of the chosen digits kept: those above the one below them;
    // T > B, so some key is smaller and the subtraction does not wrap.)
    const uint32_t limit = all ? prefix - 1u : prefix;
    if (all) need = 0;

    // ---- How many are kept before each warp's part ---------------------------
    const int per_warp = ((slice + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int w0 = min(s1, s0 + warp * per_warp), w1 = min(s1, w0 + per_warp);
    int gt = 0, eq = 0, gt_low = 0, eq_low = 0;
#pragma unroll 4
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? key_at(i) : 0u;
        const bool is_gt = i < w1 && k > limit, is_eq = i < w1 && k == limit;
        gt += is_gt;
        eq += is_eq;
        gt_low += is_gt && i < B;
        eq_low += is_eq && i < B;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    gt_low = __reduce_add_sync(0xffffffffu, gt_low);
    eq_low = __reduce_add_sync(0xffffffffu, eq_low);
    if (tid < 4) totals[tid] = 0;
    __syncthreads();
    if (lane == 0) {
        warp_n[2 * warp] = gt;
        warp_n[2 * warp + 1] = eq;
        atomicAdd(totals, gt);
        atomicAdd(totals + 1, eq);
        atomicAdd(totals + 2, gt_low);
        atomicAdd(totals + 3, eq_low);
    }
    cluster_sync();
    // Lane c < ncta reads CTA c's totals, lane w < kWarps warp w's counts.
    int4 ct = make_int4(0, 0, 0, 0);
    if (lane < int(ncta)) ct = peer_load4(totals, lane);
    const int2 wn = lane < warp ? reinterpret_cast<const int2*>(warp_n)[lane] : make_int2(0, 0);
    const bool earlier = lane < int(rank);
    int gt_before = __reduce_add_sync(0xffffffffu, (earlier ? ct.x : 0) + wn.x);
    int eq_before = __reduce_add_sync(0xffffffffu, (earlier ? ct.y : 0) + wn.y);
    const int low_gt = __reduce_add_sync(0xffffffffu, ct.z);
    const int low_eq = __reduce_add_sync(0xffffffffu, ct.w);
    const int kept_low = low_gt + min(need, low_eq);  // kept below B
    const int moves = B - kept_low;

    // ---- Holes and moving rows, in order -----------------------------------
    int32_t* msrc = a.move_src + int64_t(row) * a.cap;
    int32_t* mdst = a.move_dst + int64_t(row) * a.cap;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < w1;
        const uint32_t k = in ? key_at(i) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && k > limit);
        const uint32_t be = __ballot_sync(0xffffffffu, in && k == limit);
        const int eqr = eq_before + __popc(be & below);
        const bool kept = in && (k > limit || (k == limit && eqr < need));
        const int kb = gt_before + __popc(bg & below) + min(need, eqr);  // kept before i
        if (in) {
            if (i < B) {
                if (!kept) mdst[i - kb] = i;
            } else if (kept) {
                msrc[kb - kept_low] = i;
            } else {
                score_out[i] = 0.f;
            }
        }
        gt_before += __popc(bg);
        eq_before += __popc(be);
    }
    // The lists are complete (and every CTA has read the request's state).
    cluster_sync();
    if (rank == 0 && tid == 0) {
        a.lens_out[row] = B;
        a.move_count[row] = moves;
    }
    if (!state) return;  // the kernel that moves the rows moves these too
    for (int j = int(rank) * kThreads + tid; j < moves; j += int(ncta) * kThreads) {
        const int s = __ldcg(msrc + j), d = __ldcg(mdst + j);
        const float x = score[s];
        score_out[s] = 0.f;
        score_out[d] = x;
        if (pos_out != nullptr) pos_out[d] = pos ? pos[s] : s;
    }
}

struct MoveArgs {
    unsigned char* k;
    unsigned char* v;  // or nullptr
    int64_t page_stride, row_stride, head_stride;  // bytes
    int32_t kv_heads, row_bytes, num_pages, page_size, rows, max_blocks, cap;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;
    int32_t* status;
    // Scores and positions that move along, or nullptr.
    const float* score;
    float* score_out;
    const int32_t* positions;
    int32_t* positions_out;
    int64_t score_stride, score_out_stride, pos_stride, pos_out_stride;
};

// Byte offset of a request's place in the caches, or -1 (a bad page).
__device__ __forceinline__ int64_t place_of(const MoveArgs& a, const int32_t* table, int i) {
    const int b = i / a.page_size;
    if (i < 0 || b >= a.max_blocks) return -1;
    const int page = table[b];
    if (page < 0 || page >= a.num_pages) return -1;
    return page * a.page_stride + (i - b * a.page_size) * a.row_stride;
}

// A warp takes up to 32 moves at a time, a lane looking up one of them (the
// offsets go to shared memory), and copies their rows of all caches as one
// run of 16-byte pieces, a piece per lane and four in flight (four CTAs an SM:
// 8 in flight or 6 CTAs measured 10 % slower, the registers spill).
constexpr int kMoveWarps = 8;
constexpr int kMoveFlight = 4;
__global__ void __launch_bounds__(kMoveWarps * 32, 4)
evict_move_kernel(const __grid_constant__ MoveArgs a, int ctas_per_row) {
    __shared__ longlong2 offs[kMoveWarps][32];
    hs::pdl_trigger();
    hs::pdl_wait();
    const int row = blockIdx.x / ctas_per_row, part = blockIdx.x % ctas_per_row;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = min(max(a.count[row], 0), a.cap);
    const int32_t* src = a.src + int64_t(row) * a.cap;
    const int32_t* dst = a.dst + int64_t(row) * a.cap;
    const int32_t* table = a.block_table + int64_t(row) * a.bt_stride;
    const int warps = ctas_per_row * kMoveWarps;
    // Fewer moves a batch where there are few, so that every warp has some.
    const int batch = min(32, max(1, (n + warps - 1) / warps));
    const int per_head = a.row_bytes / 16, chunks = per_head * a.kv_heads;
    const int pieces = a.v != nullptr ? 2 * chunks : chunks;  // of one move
    const bool dense = a.head_stride == a.row_bytes || a.kv_heads == 1;
    bool bad = false;
    for (int j0 = (part * kMoveWarps + warp) * batch; j0 < n; j0 += warps * batch) {
        const int m = min(n - j0, batch);
        int s = 0, d = 0, p = 0;
        float sc = 0.f;
        if (lane < m) {
            s = __ldcg(src + j0 + lane);
            d = __ldcg(dst + j0 + lane);
            if (a.score_out != nullptr) {
                sc = a.score[row * a.score_stride + s];
                p = a.positions != nullptr ? a.positions[row * a.pos_stride + s] : s;
            }
            longlong2 o;
            o.x = place_of(a, table, s);
            o.y = place_of(a, table, d);
            if (o.x < 0 || o.y < 0) {
                bad = true;
                o.x = -1;
            }
            offs[warp][lane] = o;
        }
        __syncwarp();
        int j = 0, x = lane;  // this lane's next piece: x of move j
        while (x >= pieces) {
            x -= pieces;
            ++j;
        }
        while (__any_sync(0xffffffffu, j < m)) {
            uint4 r[kMoveFlight];
            unsigned char* to[kMoveFlight];
#pragma unroll
            for (int u = 0; u < kMoveFlight; ++u) {
                to[u] = nullptr;
                if (j < m) {
                    const longlong2 o = offs[warp][j];
                    const bool second = x >= chunks;
                    const int y = second ? x - chunks : x;
                    const int64_t at = dense ? int64_t(y) * 16
                                             : (y / per_head) * a.head_stride + (y % per_head) * 16;
                    unsigned char* base = (second ? a.v : a.k) + at;
                    if (o.x >= 0) {
                        r[u] = __ldcs(reinterpret_cast<const uint4*>(base + o.x));
                        to[u] = base + o.y;
                    }
                    x += 32;
                    while (x >= pieces) {
                        x -= pieces;
                        ++j;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kMoveFlight; ++u)
                if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = r[u];
        }
        if (lane < m && a.score_out != nullptr) {
            a.score_out[row * a.score_out_stride + s] = 0.f;
            a.score_out[row * a.score_out_stride + d] = sc;
            if (a.positions_out != nullptr) a.positions_out[row * a.pos_out_stride + d] = p;
        }
        __syncwarp();  // the offsets are read
    }
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
}

// Few tokens too many (max_len - budget <= kTrimMost, a decode step's case):
// one CTA per request holds all keys in registers, finds the evicted tokens
// one at a time as block-wide minima in the order (lower key, higher index),
// and moves the rows itself: one launch, no lists to scan.
__global__ void __launch_bounds__(kTrimThreads)
evict_trim_kernel(const __grid_constant__ EvictArgs a, const __grid_constant__ MoveArgs m) {
    __shared__ unsigned long long best[kTrimThreads / 32];
    __shared__ int out_s[kTrimMost];           // evicted places
    __shared__ int2 move_s[kTrimMost];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x;
    hs::pdl_trigger();
    hs::pdl_wait();
    const int len = a.seq_lens[row];
    const int T = min(max(len, 0), a.max_len), B = a.budget;
    const int E = max(0, T - B);
    const float* score = a.score + int64_t(row) * a.score_stride;
    const int32_t* pos = a.positions ? a.positions + int64_t(row) * a.pos_stride : nullptr;
    float* score_out = a.score_out + int64_t(row) * a.score_out_stride;
    int32_t* pos_out =
        a.positions_out ? a.positions_out + int64_t(row) * a.pos_out_stride : nullptr;
    const bool copy_score = a.score_out != a.score;
    const bool copy_pos = pos_out != nullptr && a.positions_out != a.positions;
    const int64_t from = int64_t(a.next_pos ? a.next_pos[row] : T) - a.recent;
    if (len > a.max_len && tid == 0) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    // (protected, key, inverted index) of this thread's tokens: the smallest is
    // evicted first (no key has all bits set, so ~0 means none).  Kept places
    // below the budget are copied on the way; an evicted one among them is
    // overwritten or zeroed below.
    unsigned long long k[kTrimKeys];
#pragma unroll
    for (int u0 = 0; u0 < kTrimKeys; u0 += 4) {
        if (u0 * kTrimThreads >= T) {
            k[u0] = k[u0 + 1] = k[u0 + 2] = k[u0 + 3] = ~0ull;
            continue;
        }
        // Four loads ahead of their stores (the outputs may be the inputs).
        float x[4];
        int32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = tid + (u0 + u) * kTrimThreads;
            x[u] = i < T ? score[i] : 0.f;
            p[u] = pos != nullptr && i < T ? pos[i] : i;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = tid + (u0 + u) * kTrimThreads;
            const uint32_t keep = p[u] < a.sinks || p[u] >= from;
            const uint64_t key = (uint64_t(keep) << 32) | order_key(x[u]);
            k[u0 + u] = i < T ? (key << 31) | uint32_t(kPlaces - i) : ~0ull;
            if (i < min(T, B)) {
                if (copy_score) score_out[i] = x[u];
                if (copy_pos) pos_out[i] = p[u];
            }
        }
    }
    for (int e = 0; e < E; ++e) {
        unsigned long long low = ~0ull;
#pragma unroll
        for (int u = 0; u < kTrimKeys; ++u)
            if (u * kTrimThreads < T) low = min(low, k[u]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
        if (lane == 0) best[warp] = low;
        __syncthreads();
        low = best[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
        const int i = kPlaces - int(low & kPlaces);
        if (tid == 0) out_s[e] = i;
        // Its owner drops it.
        if ((i & (kTrimThreads - 1)) == tid) {
#pragma unroll
            for (int u = 0; u < kTrimKeys; ++u)
                if (k[u] == low) k[u] = ~0ull;
        }
        __syncthreads();  // best is read, out_s written
    }
    // The j-th kept place from the budget on goes to the j-th hole.
    int moves = 0;
    if (E > 0) {
        int holes = 0;
        for (int e = 0; e < E; ++e) holes += out_s[e] < B;
        moves = holes;
        if (tid < E) {
            const int i = out_s[tid];
            if (i < B) {
                int j = 0;
                for (int e = 0; e < E; ++e) j += out_s[e] < i;
                move_s[j].y = i;
            }
            const int s = B + tid;
            bool kept = true;
            int j = tid;
            for (int e = 0; e < E; ++e) {
                if (out_s[e] == s) kept = false;
                if (out_s[e] >= B && out_s[e] < s) --j;
            }
            if (kept) move_s[j].x = s;
        }
        __syncthreads();
        float x = 0.f;
        int p = 0;
        if (tid < moves) {
            const int2 mv = move_s[tid];
            a.move_src[int64_t(row) * a.cap + tid] = mv.x;
            a.move_dst[int64_t(row) * a.cap + tid] = mv.y;
            x = score[mv.x];
            p = pos ? pos[mv.x] : mv.x;
        }
        __syncwarp();
        if (tid < E) score_out[B + tid] = 0.f;
        if (tid < moves) {
            score_out[move_s[tid].y] = x;
            if (pos_out != nullptr) pos_out[move_s[tid].y] = p;
        }
    }
    if (tid == 0) {
        a.lens_out[row] = min(T, B);
        a.move_count[row] = moves;
    }
    if (m.k == nullptr) return;
    // The rows: a warp per (move, cache, head), 16 bytes a lane.
    const int32_t* table = m.block_table + int64_t(row) * m.bt_stride;
    const int caches = m.v != nullptr ? 2 : 1;
    const int per_head = m.row_bytes / 16;
    bool bad = false;
    for (int w = warp; w < moves * caches * m.kv_heads; w += kTrimThreads / 32) {
        const int h = w % m.kv_heads, c = w / m.kv_heads % caches;
        const int2 mv = move_s[w / (m.kv_heads * caches)];
        const int64_t f = place_of(m, table, mv.x), t = place_of(m, table, mv.y);
        if (f < 0 || t < 0) {
            bad = true;
            continue;
        }
        unsigned char* base = (c ? m.v : m.k) + h * m.head_stride;
        for (int x = lane; x < per_head; x += 32)
            *reinterpret_cast<uint4*>(base + t + x * 16) =
                __ldcs(reinterpret_cast<const uint4*>(base + f + x * 16));
    }
    if (bad) hs::set_status(m.status, HS_ERR_BAD_INDEX);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_select(const EvictArgs& a) {
    if (a.rows < 0 || a.max_len < 0 || a.budget <= 0 || a.recent < 0 || a.sinks < 0 ||
        int64_t(a.recent) + a.sinks > a.budget || a.cap < 0)
        return HS_ERR_INVALID_ARG;
    // Places are counted in 31 bits; a request moves at most this many rows.
    if (a.max_len > (1 << 30)) return HS_ERR_CAPACITY;
    if (a.cap < hs::min64(a.budget, hs::max64(0, int64_t(a.max_len) - a.budget)))
        return HS_ERR_CAPACITY;
    if (a.rows == 0) return HS_OK;
    if (a.score == nullptr || a.seq_lens == nullptr || a.score_out == nullptr ||
        a.lens_out == nullptr || a.move_count == nullptr ||
        (a.cap > 0 && (a.move_src == nullptr || a.move_dst == nullptr)))
        return HS_ERR_INVALID_ARG;
    if (a.score_stride < a.max_len || a.score_out_stride < a.max_len ||
        (a.positions != nullptr && a.pos_stride < a.max_len) ||
        (a.positions_out != nullptr && a.pos_out_stride < a.max_len) ||
        (a.score == a.score_out && a.score_stride != a.score_out_stride) ||
        (a.positions != nullptr && a.positions == a.positions_out &&
         a.pos_stride != a.pos_out_stride))
        return HS_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(a.score), static_cast<const void*>(a.score_out),
                          static_cast<const void*>(a.positions),
                          static_cast<const void*>(a.positions_out),
                          static_cast<const void*>(a.seq_lens),
                          static_cast<const void*>(a.next_pos),
                          static_cast<const void*>(a.lens_out),
                          static_cast<const void*>(a.move_src),
                          static_cast<const void*>(a.move_dst),
                          static_cast<const void*>(a.move_count)})
        if (!aligned(p, 4)) return HS_ERR_MISALIGNED;
    return HS_OK;
}

// Whether every request is within a few tokens of the budget and small enough
// for the trimming kernel (64 requests of 2049 tokens: one launch instead of
// two, 5.65 us a call instead of 16.8).
bool trims(const EvictArgs& a) {
    return int64_t(a.max_len) - a.budget <= kTrimMost && a.max_len <= kTrimThreads * kTrimKeys;
}

int launch_trim(const EvictArgs& a, const MoveArgs& m, hs_stream_t stream) {
    return hs_host::launch_pdl(evict_trim_kernel, dim3(unsigned(a.rows)), dim3(kTrimThreads), 0,
                               stream, a, m);
}

// state: whether the scores and positions move here or with the rows.
int launch_select(const EvictArgs& a, bool state, hs_stream_t stream) {
    // As many CTAs per request as the GPU has free, each with a slice worth
    // a cluster barrier.
    const int64_t sms = hs_host::num_sms();
    int cl = 1;
    while (cl < kMaxCluster && int64_t(a.rows) * cl * 2 <= sms &&
           a.max_len > int64_t(cl) * kSliceMin)
        cl *= 2;
    const int slice = int((int64_t(a.max_len) + cl - 1) / cl);
    const int cached = slice <= kCacheKeys;
    const size_t smem = size_t(kCopies * kBins + 2 * kBins + 4 + 32 + 4 + 2 * kWarps) * 4 +
                        (cached ? size_t(slice) * 4 : 0);
    static int smem_set[64] = {};
    const int rc = hs_host::ensure_dynamic_smem(
        reinterpret_cast<const void*>(evict_select_kernel), smem, smem_set);
    if (rc != HS_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows) * unsigned(cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cl);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a, slice, cached, int(state)) !=
        cudaSuccess) {
        cudaGetLastError();
        return HS_ERR_CUDA;
    }
    return HS_OK;
}

int check_move(const MoveArgs& a) {
    if (a.rows < 0 || a.kv_heads <= 0 || a.row_bytes <= 0 || a.num_pages < 0 ||
        a.page_size <= 0 || a.max_blocks < 0 || a.cap < 0 || a.page_stride < 0 ||
        a.row_stride < 0 || a.head_stride < 0 || a.bt_stride < 0 ||
        int64_t(a.kv_heads) * a.row_bytes > (int64_t(1) << 30))
        return HS_ERR_INVALID_ARG;
    if (a.row_bytes % 16 || a.page_stride % 16 || a.row_stride % 16 || a.head_stride % 16 ||
        !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.block_table, 4) ||
        !aligned(a.src, 4) || !aligned(a.dst, 4) || !aligned(a.count, 4))
        return HS_ERR_MISALIGNED;
    if (a.rows == 0 || a.cap == 0) return HS_OK;
    if (a.k == nullptr || a.block_table == nullptr || a.src == nullptr || a.dst == nullptr ||
        a.count == nullptr || a.k == a.v)
        return HS_ERR_INVALID_ARG;
    return HS_OK;
}

int launch_move(const MoveArgs& a, hs_stream_t stream) {
    if (a.rows == 0 || a.cap == 0) return HS_OK;
    const int64_t most = (int64_t(a.cap) + kMoveWarps - 1) / kMoveWarps;
    const int64_t want = hs::max64(1, 8 * int64_t(hs_host::num_sms()) / a.rows);
    const int per_row = int(hs::min64(most, want));
    return hs_host::launch_pdl(evict_move_kernel, dim3(unsigned(a.rows) * unsigned(per_row)),
                               dim3(kMoveWarps * 32), 0, stream, a, per_row);
}

EvictArgs select_args(const float* score, int64_t score_stride, const int32_t* positions,
                      int64_t pos_stride, const int32_t* seq_lens, const int32_t* next_pos,
                      int32_t rows, int32_t max_len, int32_t budget, int32_t recent,
                      int32_t num_sinks, float* score_out, int64_t score_out_stride,
                      int32_t* positions_out, int64_t pos_out_stride, int32_t* lens_out,
                      int32_t* move_src, int32_t* move_dst, int32_t* move_count, int32_t cap,
                      int32_t* status) {
    return EvictArgs{score, score_stride, positions, pos_stride, seq_lens, next_pos, rows, max_len,
                     budget, recent, num_sinks, score_out, score_out_stride, positions_out,
                     pos_out_stride, lens_out, move_src, move_dst, move_count, cap, status};
}

MoveArgs move_args(void* k, void* v, int64_t page_stride, int64_t row_stride, int64_t head_stride,
                   int32_t kv_heads, int32_t row_bytes, int32_t num_pages, int32_t page_size,
                   const int32_t* block_table, int64_t bt_stride, int32_t max_blocks,
                   const int32_t* src, const int32_t* dst, const int32_t* count, int32_t rows,
                   int32_t cap, int32_t* status) {
    return MoveArgs{static_cast<unsigned char*>(k), static_cast<unsigned char*>(v), page_stride,
                    row_stride, head_stride, kv_heads, row_bytes, num_pages, page_size, rows,
                    max_blocks, cap, block_table, bt_stride, src, dst, count, status,
                    nullptr, nullptr, nullptr, nullptr, 0, 0, 0, 0};
}

}  // namespace

extern "C" int hs_evict_select(const float* score, int64_t score_stride, const int32_t* positions,
                               int64_t pos_stride, const int32_t* seq_lens,
                               const int32_t* next_pos, int32_t rows, int32_t max_len,
                               int32_t budget, int32_t recent, int32_t num_sinks,
                               float* score_out, int64_t score_out_stride, int32_t* positions_out,
                               int64_t pos_out_stride, int32_t* lens_out, int32_t* move_src,
                               int32_t* move_dst, int32_t* move_count, int32_t cap,
                               int32_t* status, hs_stream_t stream) {
    const EvictArgs a = select_args(score, score_stride, positions, pos_stride, seq_lens, next_pos,
                                    rows, max_len, budget, recent, num_sinks, score_out,
                                    score_out_stride, positions_out, pos_out_stride, lens_out,
                                    move_src, move_dst, move_count, cap, status);
    const int rc = check_select(a);
    if (rc != HS_OK || rows == 0) return rc;
    return trims(a) ? launch_trim(a, MoveArgs{}, stream) : launch_select(a, true, stream);
}

extern "C" int hs_evict_move(void* k, void* v, int64_t page_stride, int64_t row_stride,
                             int64_t head_stride, int32_t kv_heads, int32_t row_bytes,
                             int32_t num_pages, int32_t page_size, const int32_t* block_table,
                             int64_t bt_stride, int32_t max_blocks, const int32_t* move_src,
                             const int32_t* move_dst, const int32_t* move_count, int32_t rows,
                             int32_t cap, int32_t* status, hs_stream_t stream) {
    const MoveArgs m = move_args(k, v, page_stride, row_stride, head_stride, kv_heads, row_bytes,
                                 num_pages, page_size, block_table, bt_stride, max_blocks,
                                 move_src, move_dst, move_count, rows, cap, status);
    const int rc = check_move(m);
    return rc != HS_OK ? rc : launch_move(m, stream);
}

extern "C" int hs_evict(const float* score, int64_t score_stride, const int32_t* positions,
                        int64_t pos_stride, const int32_t* seq_lens, const int32_t* next_pos,
                        int32_t rows, int32_t max_len, int32_t budget, int32_t recent,
                        int32_t num_sinks, float* score_out, int64_t score_out_stride,
                        int32_t* positions_out, int64_t pos_out_stride, int32_t* lens_out,
                        int32_t* move_src, int32_t* move_dst, int32_t* move_count, int32_t cap,
                        void* k, void* v, int64_t page_stride, int64_t row_stride,
                        int64_t head_stride, int32_t kv_heads, int32_t row_bytes,
                        int32_t num_pages, int32_t page_size, const int32_t* block_table,
                        int64_t bt_stride, int32_t max_blocks, int32_t* status,
                        hs_stream_t stream) {
    const EvictArgs a = select_args(score, score_stride, positions, pos_stride, seq_lens, next_pos,
                                    rows, max_len, budget, recent, num_sinks, score_out,
                                    score_out_stride, positions_out, pos_out_stride, lens_out,
                                    move_src, move_dst, move_count, cap, status);
    MoveArgs m = move_args(k, v, page_stride, row_stride, head_stride, kv_heads, row_bytes,
                           num_pages, page_size, block_table, bt_stride, max_blocks,
                           move_src, move_dst, move_count, rows, cap, status);
    int rc = check_select(a);
    if (rc == HS_OK) rc = check_move(m);
    if (rc == HS_OK && int64_t(max_blocks) * page_size < max_len) rc = HS_ERR_INVALID_ARG;
    if (rc != HS_OK || rows == 0) return rc;
    if (trims(a)) return launch_trim(a, m, stream);
    // The scores and positions of the rows that move go with them, so that the
    // selection, during which nothing else runs, is shorter (32 latent contexts
    // of 32 K tokens in a captured graph, part of the rows from L2, 39.5 us
    // instead of 40.5; 43.7 where the inputs change).
    m.score = score;
    m.score_out = score_out;
    m.positions = positions;
    m.positions_out = positions_out;
    m.score_stride = score_stride;
    m.score_out_stride = score_out_stride;
    m.pos_stride = pos_stride;
    m.pos_out_stride = pos_out_stride;
    rc = launch_select(a, false, stream);
    return rc != HS_OK ? rc : launch_move(m, stream);
}
