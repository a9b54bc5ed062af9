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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxCluster = 8;
constexpr int kCacheKeys = 40960;   // keys of a CTA's slice that shared memory keeps
constexpr int kSliceMin = 4096;     // tokens a CTA of a cluster should have at least

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
__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
    uint32_t addr;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(addr)
                 : "r"(hs::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Order of scores as unsigned integers: NaN below everything, the two zeros
// equal, protected tokens above +inf.
__device__ __forceinline__ uint32_t order_key(float s, bool keep) {
    if (keep) return 0xffffffffu;
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One cluster per request, each CTA a contiguous slice of its tokens.  The
// B-th largest key is found by its digits of 8 bits from the top: every CTA
// counts its slice's digits (one counter column per lane, so the atomics of a
// warp never meet in a bank), the cluster sums the 256 counts through
// distributed shared memory, and only keys that share the chosen digits are
// counted again.  Then each warp walks its part of the slice in order: what
// is kept before an index gives the rank of a hole or of a moving row.
__global__ void __launch_bounds__(kThreads)
evict_select_kernel(const __grid_constant__ EvictArgs a, int slice, int cached) {
    extern __shared__ __align__(16) unsigned char smem[];
    int* hist = reinterpret_cast<int*>(smem);              // [kBins][32]
    int* counts = hist + kBins * 32;                       // [4][kBins], read by the cluster
    int* totals = counts + 4 * kBins;                      // [4]: gt, eq, gt < B, eq < B
    int* scratch = totals + 4;                             // [32]
    int* pick = scratch + 32;                              // [4]
    int* warp_n = pick + 4;                                // [kWarps][2]
    uint32_t* keys = reinterpret_cast<uint32_t*>(warp_n + 2 * kWarps);  // [slice] if cached
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), ncta = cluster_size();
    const int row = blockIdx.x / ncta;

    hs::pdl_trigger();
    hs::pdl_wait();
    const int len = a.seq_lens[row];
    const int T = min(max(len, 0), a.max_len), B = a.budget;
    const float* score = a.score + int64_t(row) * a.score_stride;
    const int32_t* pos = a.positions ? a.positions + int64_t(row) * a.pos_stride : nullptr;
    float* score_out = a.score_out + int64_t(row) * a.score_out_stride;
    int32_t* pos_out =
        a.positions_out ? a.positions_out + int64_t(row) * a.pos_out_stride : nullptr;
    const bool copy_score = a.score_out != a.score;
    const bool copy_pos = pos_out != nullptr && a.positions_out != a.positions;
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
    const int newest = a.next_pos ? a.next_pos[row] : T;
    const int64_t from = int64_t(newest) - a.recent;  // positions from here on are protected
    auto make_key = [&](int i) {
        const int p = pos ? pos[i] : i;
        return order_key(score[i], p < a.sinks || p >= from);
    };
    auto key_at = [&](int i) { return cached ? keys[i - s0] : make_key(i); };

    // ---- The B-th largest key ---------------------------------------------
    uint32_t prefix = 0;  // digits chosen so far
    int need = B;         // keys still wanted among those that share them
    bool all = false;     // every key of the chosen digits is kept
    int shift = 24;
    for (;; shift -= 8) {
        for (int i = tid; i < kBins * 32; i += kThreads) hist[i] = 0;
        __syncthreads();
        if (shift == 24) {
            constexpr int U = 8;
            for (int i0 = s0 + tid; i0 < s1; i0 += U * kThreads) {
                uint32_t k[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * kThreads;
                    k[u] = i < s1 ? make_key(i) : 0u;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * kThreads;
                    if (i < s1) {
                        if (cached) keys[i - s0] = k[u];
                        atomicAdd(hist + (k[u] >> 24) * 32 + lane, 1);
                    }
                }
            }
        } else {
            for (int i = s0 + tid; i < s1; i += kThreads) {
                const uint32_t k = key_at(i);
                if ((k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(hist + ((k >> shift) & 255u) * 32 + lane, 1);
            }
        }
        __syncthreads();
        int* mine = counts + (shift >> 3) * kBins;
        if (tid < kBins) {
            int n = 0;
#pragma unroll 8
            for (int j = 0; j < 32; ++j) n += hist[tid * 32 + ((j + tid) & 31)];
            mine[tid] = n;
        }
        cluster_sync();
        // Counts of the whole request, from the largest digit down.
        int v = 0;
        if (tid < kBins)
            for (uint32_t c = 0; c < ncta; ++c) v += peer_load(mine + (kBins - 1 - tid), c);
        int sum;
        const int before = hs::block_excl_scan(v, scratch, &sum);
        if (tid < kBins && before < need && need <= before + v) {
            pick[0] = kBins - 1 - tid;
            pick[1] = need - before;
            pick[2] = need == before + v;
        }
        __syncthreads();
        prefix |= uint32_t(pick[0]) << shift;
        need = pick[1];
        all = pick[2] != 0;
        if (all || shift == 0) break;
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
    int gt_before = 0, eq_before = 0, low_gt = 0, low_eq = 0;
    for (uint32_t c = 0; c < ncta; ++c) {
        if (c < rank) {
            gt_before += peer_load(totals, c);
            eq_before += peer_load(totals + 1, c);
        }
        low_gt += peer_load(totals + 2, c);
        low_eq += peer_load(totals + 3, c);
    }
    for (int w = 0; w < warp; ++w) {
        gt_before += warp_n[2 * w];
        eq_before += warp_n[2 * w + 1];
    }
    const int kept_low = low_gt + min(need, low_eq);  // kept below B
    const int moves = B - kept_low;

    // ---- Holes and moving rows, in order -----------------------------------
    int32_t* msrc = a.move_src + int64_t(row) * a.cap;
    int32_t* mdst = a.move_dst + int64_t(row) * a.cap;
    const uint32_t below = (1u << lane) - 1u;
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
                if (!kept) {
                    mdst[i - kb] = i;
                } else {
                    if (copy_score) score_out[i] = score[i];
                    if (copy_pos) pos_out[i] = pos ? pos[i] : i;
                }
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
    __threadfence();
    cluster_sync();
    for (int j = int(rank) * kThreads + tid; j < moves; j += int(ncta) * kThreads) {
        const int s = __ldcg(msrc + j), d = __ldcg(mdst + j);
        const float x = score[s];
        score_out[s] = 0.f;
        score_out[d] = x;
        if (pos_out != nullptr) pos_out[d] = pos ? pos[s] : s;
    }
    if (rank == 0 && tid == 0) {
        a.lens_out[row] = B;
        a.move_count[row] = moves;
    }
    cluster_sync();  // no CTA ends while a peer may still read its shared memory
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
};

// A warp moves one token of one cache at a time, 16 bytes a lane, four loads
// in flight before the stores.
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ MoveArgs a,
                                                         int ctas_per_row) {
    hs::pdl_trigger();
    hs::pdl_wait();
    const int row = blockIdx.x / ctas_per_row, part = blockIdx.x % ctas_per_row;
    const int lane = threadIdx.x & 31;
    const int n = min(max(a.count[row], 0), a.cap);
    const int caches = a.v != nullptr ? 2 : 1;
    const int32_t* table = a.block_table + int64_t(row) * a.bt_stride;
    const int per_head = a.row_bytes / 16, chunks = per_head * a.kv_heads;
    bool bad = false;
    for (int w = part * 8 + (threadIdx.x >> 5); w < n * caches; w += ctas_per_row * 8) {
        const int j = w / caches, c = w % caches;
        const int s = a.src[int64_t(row) * a.cap + j], d = a.dst[int64_t(row) * a.cap + j];
        const int sb = s / a.page_size, db = d / a.page_size;
        int sp = -1, dp = -1;
        if (s >= 0 && sb < a.max_blocks) sp = table[sb];
        if (d >= 0 && db < a.max_blocks) dp = table[db];
        if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
            bad = true;
            continue;
        }
        unsigned char* base = c ? a.v : a.k;
        const unsigned char* from = base + sp * a.page_stride + (s % a.page_size) * a.row_stride;
        unsigned char* to = base + dp * a.page_stride + (d % a.page_size) * a.row_stride;
        for (int x0 = lane; x0 < chunks; x0 += 128) {
            uint4 r[4];
            int64_t off[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int x = x0 + 32 * u;
                off[u] = (x / per_head) * a.head_stride + (x % per_head) * 16;
                if (x < chunks) r[u] = __ldcg(reinterpret_cast<const uint4*>(from + off[u]));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (x0 + 32 * u < chunks) *reinterpret_cast<uint4*>(to + off[u]) = r[u];
        }
    }
    if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_select(const EvictArgs& a) {
    if (a.rows < 0 || a.max_len < 0 || a.budget <= 0 || a.recent < 0 || a.sinks < 0 ||
        int64_t(a.recent) + a.sinks > a.budget || a.cap < 0)
        return HS_ERR_INVALID_ARG;
    // A request moves at most this many rows.
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

int launch_select(const EvictArgs& a, hs_stream_t stream) {
    // As many CTAs per request as the GPU has free, each with a slice worth
    // a cluster barrier.
    const int64_t sms = hs_host::num_sms();
    int cl = 1;
    while (cl < kMaxCluster && int64_t(a.rows) * cl * 2 <= sms &&
           a.max_len > int64_t(cl) * kSliceMin)
        cl *= 2;
    const int slice = int((int64_t(a.max_len) + cl - 1) / cl);
    const int cached = slice <= kCacheKeys;
    const size_t smem = size_t(kBins * 32 + 4 * kBins + 4 + 32 + 4 + 2 * kWarps) * 4 +
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
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a, slice, cached) != cudaSuccess) {
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
    const int64_t most = (int64_t(a.cap) * (a.v != nullptr ? 2 : 1) + 7) / 8;
    const int64_t want = hs::max64(1, 8 * int64_t(hs_host::num_sms()) / a.rows);
    const int per_row = int(hs::min64(most, want));
    return hs_host::launch_pdl(evict_move_kernel, dim3(unsigned(a.rows) * unsigned(per_row)),
                               dim3(256), 0, stream, a, per_row);
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
                    max_blocks, cap, block_table, bt_stride, src, dst, count, status};
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
    return launch_select(a, stream);
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
    const MoveArgs m = move_args(k, v, page_stride, row_stride, head_stride, kv_heads, row_bytes,
                                 num_pages, page_size, block_table, bt_stride, max_blocks,
                                 move_src, move_dst, move_count, rows, cap, status);
    int rc = check_select(a);
    if (rc == HS_OK) rc = check_move(m);
    if (rc == HS_OK && int64_t(max_blocks) * page_size < max_len) rc = HS_ERR_INVALID_ARG;
    if (rc != HS_OK || rows == 0) return rc;
    rc = launch_select(a, stream);
    return rc != HS_OK ? rc : launch_move(m, stream);
}
