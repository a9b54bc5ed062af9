// hs_extend.cu -- hs_paged_extend: requests of a paged cache grow by a step's
// new tokens or give tokens up; pages come from and go to a ring of free ones.
//
// With T tokens held, n asked for (n < 0: given up) and pages of B tokens,
//   need = ceil((T + n) / B) - ceil(T / B) of a request that grows,
//   back = ceil(T / B) - ceil((T + n) / B) of one that shrinks,
// and the requests' shares of the tokens and of the ring are prefix sums over
// the requests in order.
//
// Latency bounds it (a few KB to a few MB): one kernel of one CTA or one
// cluster of CTAs.  Every CTA makes the prefix sums of all requests for itself
// (at most 4096: four to a thread), then takes its share of the tokens and of
// the pages that change hands, finding the request of each by bisection in
// shared memory; a token in a fresh block reads its page from the ring, so
// nothing waits for the table.  The cluster barrier between the two parts lets
// lengths and ring be updated in place.
#include "hs_common.cuh"
#include "hs_pair.cuh"

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxRows = 4096;
constexpr int kPer = kMaxRows / kThreads;  // requests of a thread
constexpr int kMany = 1 << 30;             // prefix sums stop here (saturating)
constexpr int kMaxCluster = 8;

struct ExtendArgs {
    const int32_t* new_lens;
    const int32_t* seq_lens;
    int32_t* table;
    int64_t bt_stride;
    int32_t rows, max_blocks;
    int32_t* ring;
    int32_t pages;
    const int64_t* ring_pos;
    int32_t page_size, max_tokens;
    int32_t* lens_out;
    int32_t* attend_lens;
    int64_t* ring_out;
    int32_t* cu_new;
    int32_t* slot;
    int32_t* row_req;
    int32_t* positions;
    int32_t* status;
};

__device__ __forceinline__ int sat_add(int a, int b) { return min(a + b, kMany); }

// Exclusive saturating prefix sum over the block of kPer consecutive values of
// each thread (each in [0, kMany]); returns the block's total.
__device__ __forceinline__ int scan_rows(int (&v)[kPer], int* scratch) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int x = v[i];
        v[i] = sum;
        sum = sat_add(sum, x);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = sat_add(incl, o);
    }
    const int before = __shfl_up_sync(0xffffffffu, incl, 1);
    __syncthreads();  // scratch may still be read
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int w = scratch[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w = sat_add(w, o);
    }
    const int total = __shfl_sync(0xffffffffu, w, 31);
    const int base = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
    const int mine = sat_add(base, lane == 0 ? 0 : before);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = sat_add(mine, v[i]);
    return total;
}

// The last r of [0, rows) with start[r] <= i.
__device__ __forceinline__ int find(const int* start, int rows, int i) {
    int lo = 0, hi = rows;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int ring_at(int64_t first, int i, int pages) {
    int x = int(first % pages) + i;
    return x >= pages ? x - pages : x;
}

__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const ExtendArgs a) {
    extern __shared__ int shared[];
    int* cu = shared;                       // first token of each request
    int* at = cu + a.rows;                  // first page that it takes
    int* to = at + a.rows;                  // first page that it gives back
    int* lens = to + a.rows;                // tokens held before
    int* grow = lens + a.rows;              // tokens granted; < 0: given up
    __shared__ int scratch[32];
    const int tid = threadIdx.x, B = a.page_size;
    const int cl = gridDim.x, rank = blockIdx.x;
    hs::pdl_wait();
    hs::pdl_trigger();
    const int64_t taken = a.ring_pos[0], returned = a.ring_pos[1];
    // A ring that cannot be: nothing is taken or given back.
    const bool odd = taken < 0 || returned < taken || returned - taken > a.pages;
    const int avail = odd ? 0 : int(returned - taken);
    const int64_t room = int64_t(a.max_blocks) * B;

    int ask[kPer], need[kPer], back[kPer], held[kPer], n[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = tid * kPer + i;
        held[i] = n[i] = 0;
        if (r < a.rows) {
            held[i] = a.seq_lens[r];
            n[i] = a.new_lens[r];
        }
    }
    bool bad = odd;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        // A length that the table cannot hold: the request is left alone.
        if (held[i] > room) {
            bad = true;
            held[i] = -1;
            n[i] = max(n[i], 0);
        } else {
            held[i] = max(held[i], 0);
        }
        ask[i] = min(max(n[i], 0), kMany);
        back[i] = 0;
        if (n[i] < 0 && held[i] > 0 && !odd) {
            const int left = max(0, held[i] + max(n[i], -held[i]));
            back[i] = (held[i] + B - 1) / B - (left + B - 1) / B;
        }
    }
    int own_ask[kPer], own_back[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        own_ask[i] = ask[i];
        own_back[i] = back[i];
    }
    const int tokens = min(scan_rows(ask, scratch), a.max_tokens);
    int given = scan_rows(back, scratch);
    // More than the ring can hold: something else returned them already.
    if (given > a.pages - avail) {
        bad = true;
        given = 0;
    }
    int own_need[kPer];
    bool fits[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        fits[i] = held[i] >= 0 && int64_t(held[i]) + own_ask[i] <= room &&
                  int64_t(ask[i]) + own_ask[i] <= a.max_tokens;
        need[i] = fits[i] ? int((int64_t(held[i]) + own_ask[i] + B - 1) / B - (held[i] + B - 1) / B)
                          : 0;
        own_need[i] = need[i];
    }
    scan_rows(need, scratch);
    bool refused = false;
    int last = 0;  // pages taken up to this thread's last served request
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = tid * kPer + i;
        if (r >= a.rows) continue;
        const bool served = fits[i] && (own_need[i] == 0 || sat_add(need[i], own_need[i]) <= avail);
        if (own_ask[i] > 0 && !served) refused = true;
        cu[r] = min(ask[i], a.max_tokens);
        at[r] = min(need[i], avail);
        to[r] = back[i];
        lens[r] = held[i];
        grow[r] = n[i] > 0 ? (served ? n[i] : 0)
                           : (!odd && given >= own_back[i] ? max(n[i], -max(held[i], 0)) : 0);
        if (served && own_need[i] > 0) last = max(last, need[i] + own_need[i]);
    }
    if (rank == 0) {
        if (bad) hs::set_status(a.status, HS_ERR_BAD_INDEX);
        if (refused) hs::set_status(a.status, HS_ERR_CAPACITY);
    }
    // Pages taken in all: what the last served request's share ends with.
    last = int(__reduce_max_sync(0xffffffffu, unsigned(last)));
    __syncthreads();
    if ((tid & 31) == 0) scratch[tid >> 5] = last;
    __syncthreads();
    const int grown = int(__reduce_max_sync(0xffffffffu, unsigned(scratch[tid & 31])));
    // Every CTA has read the lengths and the ring's ends.
    if (cl > 1) hs::pair::cluster_sync();

    const int step = cl * kThreads, first = rank * kThreads + tid;
    for (int r = first; r < a.rows; r += step) {
        const int g = grow[r], T = lens[r];
        const int now = T < 0 ? a.seq_lens[r] : T + g;
        a.lens_out[r] = now;
        a.attend_lens[r] = g > 0 ? now : 0;
        a.cu_new[r] = cu[r];
    }
    if (first == 0) {
        a.cu_new[a.rows] = tokens;
        a.ring_out[0] = taken + grown;
        a.ring_out[1] = returned + given;
    }
    for (int i = first; i < grown; i += step) {
        const int r = find(at, a.rows, i);
        a.table[r * a.bt_stride + (lens[r] + B - 1) / B + i - at[r]] =
            a.ring[ring_at(taken, i, a.pages)];
    }
    for (int i = first; i < given; i += step) {
        const int r = find(to, a.rows, i);
        a.ring[ring_at(returned, i, a.pages)] =
            a.table[r * a.bt_stride + (lens[r] + grow[r] + B - 1) / B + i - to[r]];
    }
    for (int t = first; t < a.max_tokens; t += step) {
        int r = -1, pos = -1, slot = -1;
        if (t < tokens) {
            r = find(cu, a.rows, t);
            if (grow[r] > 0) {
                pos = lens[r] + t - cu[r];
                const int b = pos / B, have = (lens[r] + B - 1) / B;
                const int page = b < have ? a.table[r * a.bt_stride + b]
                                          : a.ring[ring_at(taken, at[r] + b - have, a.pages)];
                slot = page >= 0 && page < a.pages ? page * B + pos - b * B : -1;
                if (slot < 0) hs::set_status(a.status, HS_ERR_BAD_INDEX);
            } else {
                r = -1;
            }
        }
        a.slot[t] = slot;
        a.row_req[t] = r;
        a.positions[t] = pos;
    }
}

}  // namespace

extern "C" int hs_paged_extend(const int32_t* new_lens, const int32_t* seq_lens,
                               int32_t* block_table, int64_t bt_stride, int32_t rows,
                               int32_t max_blocks, int32_t* free_ring, int32_t num_pages,
                               const int64_t* ring_pos, int32_t page_size, int32_t max_tokens,
                               int32_t* lens_out, int32_t* attend_lens, int64_t* ring_out,
                               int32_t* cu_new, int32_t* slot, int32_t* row_req,
                               int32_t* positions, int32_t* status, hs_stream_t stream) {
    if (rows < 0 || max_blocks < 0 || num_pages < 0 || page_size <= 0 || max_tokens < 0 ||
        bt_stride < 0 || (rows > 1 && bt_stride < max_blocks))
        return HS_ERR_INVALID_ARG;
    if (rows > kMaxRows || num_pages > kMany || max_tokens > kMany ||
        int64_t(num_pages) * page_size > INT32_MAX || int64_t(max_blocks) * page_size > kMany)
        return HS_ERR_CAPACITY;
    if (ring_pos == nullptr || ring_out == nullptr || cu_new == nullptr ||
        (rows > 0 && (new_lens == nullptr || seq_lens == nullptr || lens_out == nullptr ||
                      attend_lens == nullptr || (max_blocks > 0 && block_table == nullptr))) ||
        (num_pages > 0 && free_ring == nullptr) ||
        (max_tokens > 0 && (slot == nullptr || row_req == nullptr || positions == nullptr)))
        return HS_ERR_INVALID_ARG;
    const auto al = [](const void* p, uintptr_t n) {
        return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
    };
    for (const void* p : {(const void*)new_lens, (const void*)seq_lens, (const void*)block_table,
                          (const void*)free_ring, (const void*)lens_out, (const void*)attend_lens,
                          (const void*)cu_new, (const void*)slot, (const void*)row_req,
                          (const void*)positions, (const void*)status})
        if (!al(p, 4)) return HS_ERR_MISALIGNED;
    if (!al(ring_pos, 8) || !al(ring_out, 8)) return HS_ERR_MISALIGNED;
    ExtendArgs a{};
    a.new_lens = new_lens;
    a.seq_lens = seq_lens;
    a.table = block_table;
    a.bt_stride = bt_stride;
    a.rows = rows;
    a.max_blocks = max_blocks;
    a.ring = free_ring;
    a.pages = num_pages;
    a.ring_pos = ring_pos;
    a.page_size = page_size;
    a.max_tokens = max_tokens;
    a.lens_out = lens_out;
    a.attend_lens = attend_lens;
    a.ring_out = ring_out;
    a.cu_new = cu_new;
    a.slot = slot;
    a.row_req = row_req;
    a.positions = positions;
    a.status = status;
    const size_t smem = size_t(rows) * 5 * 4;
    static int smem_set[64] = {};
    const int rc = hs_host::ensure_dynamic_smem(reinterpret_cast<const void*>(extend_kernel), smem,
                                                smem_set);
    if (rc != HS_OK) return rc;
    const int cl = max_tokens > 2 * kThreads ? kMaxCluster : 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cl);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, extend_kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return HS_ERR_CUDA;
    }
    return HS_OK;
}
