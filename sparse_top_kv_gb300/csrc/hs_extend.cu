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
// (at most 4096: one or four to a thread), then takes its share of the tokens
// and of the pages that change hands, finding the request of each by bisection in
// shared memory; a token in a fresh block reads its page from the ring, so
// nothing waits for the table.  The cluster barrier between the two parts lets
// lengths and ring be updated in place.  Measured: 64 requests of one token 4.7
// us (with a 64-bit remainder per token, four requests to a thread and a scan for
// each sum 7.1), 512 requests of up to 1024 tokens 10.4 (15.9).
#include "hs_common.cuh"
#include "hs_pair.cuh"
#include "hs_plan.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxRows = 4096;
constexpr int kAtOnce = 4;                 // tokens of a thread whose pages are read together
constexpr int kMany = 1 << 30;             // most pages or tokens of a call
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
    int32_t page_size, page_shift, max_tokens;  // page_shift: log2, -1: no power of two
    int32_t* lens_out;
    int32_t* attend_lens;
    int64_t* ring_out;
    int32_t* cu_new;
    int32_t* slot;
    int32_t* row_req;
    int32_t* positions;
    int32_t* status;
};

using hs_plan::kSatMax;
using hs_plan::sat_add;

// Exclusive saturating prefix sums over the block of M lists of PER consecutive
// values of each thread (each in [0, kSatMax]); total: the block's.
template <int M, int PER>
__device__ __forceinline__ void scan_rows(int (&v)[M][PER], int (&total)[M], int (*scratch)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl[M], before[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        incl[m] = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = v[m][i];
            v[m][i] = incl[m];
            incl[m] = sat_add(incl[m], x);
        }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int o = __shfl_up_sync(0xffffffffu, incl[m], d);
            if (lane >= d) incl[m] = sat_add(incl[m], o);
        }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        before[m] = __shfl_up_sync(0xffffffffu, incl[m], 1);
        if (lane == 31) scratch[m][warp] = incl[m];
    }
    __syncthreads();
    int w[M];
#pragma unroll
    for (int m = 0; m < M; ++m) w[m] = scratch[m][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int o = __shfl_up_sync(0xffffffffu, w[m], d);
            if (lane >= d) w[m] = sat_add(w[m], o);
        }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        total[m] = __shfl_sync(0xffffffffu, w[m], 31);
        const int base = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w[m], warp - 1);
        const int mine = sat_add(base, lane == 0 ? 0 : before[m]);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[m][i] = sat_add(mine, v[m][i]);
    }
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

// PER: requests of a thread in the prefix sums.
template <int PER>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const ExtendArgs a) {
    extern __shared__ int shared[];
    int* cu = shared;                       // first token of each request
    int* at = cu + a.rows;                  // first page that it takes
    int* to = at + a.rows;                  // first page that it gives back
    int* lens = to + a.rows;                // tokens held before
    int* grow = lens + a.rows;              // tokens granted; < 0: given up
    __shared__ int scratch[4][32];          // (a row for each of the kernel's exchanges)
    __shared__ int found;                   // 1: a request was refused, 2: a state that cannot be
    const int tid = threadIdx.x, B = a.page_size;
    if (tid == 0) found = 0;
    const int cl = gridDim.x, rank = blockIdx.x;
    // Pages of n tokens, and the page of token n.
    const auto page_of = [&](int n) { return a.page_shift >= 0 ? n >> a.page_shift : n / B; };
    const auto pages_of = [&](int n) { return page_of(n + B - 1); };
    hs::pdl_wait();
    hs::pdl_trigger();
    const int64_t taken = a.ring_pos[0], returned = a.ring_pos[1];
    int held[PER], n[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = tid * PER + i;
        held[i] = n[i] = 0;
        if (r < a.rows) {
            held[i] = a.seq_lens[r];
            n[i] = a.new_lens[r];
        }
    }
    // A ring that cannot be: nothing is taken or given back.
    const bool odd = taken < 0 || returned < taken || returned - taken > a.pages;
    const int avail = odd ? 0 : int(returned - taken);
    const int64_t room = int64_t(a.max_blocks) * B;
    // The ring's ends as places.  (A 64-bit remainder for every token took longer
    // than the rest of the step.)
    int take_at = 0, give_at = 0;
    if (!odd && a.pages > 0) {
        take_at = taken >> 32 == 0 ? int(uint32_t(taken) % uint32_t(a.pages)) : int(taken % a.pages);
        give_at = take_at + avail;
        if (give_at >= a.pages) give_at -= a.pages;
    }
    const auto ring_at = [&](int first, int i) {
        const int x = first + i;
        return x >= a.pages ? x - a.pages : x;
    };

    bool bad = odd;
    int asked[2][PER], own_ask[PER], own_back[PER];  // tokens asked for, pages given back
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        // A length that the table cannot hold: the request is left alone.
        if (held[i] > room) {
            bad = true;
            held[i] = -1;
            n[i] = max(n[i], 0);
        } else {
            held[i] = max(held[i], 0);
        }
        own_ask[i] = min(max(n[i], 0), kSatMax);
        own_back[i] = 0;
        if (n[i] < 0 && held[i] > 0 && !odd)
            own_back[i] = pages_of(held[i]) - pages_of(max(0, held[i] + max(n[i], -held[i])));
        asked[0][i] = own_ask[i];
        asked[1][i] = own_back[i];
    }
    int totals[2];
    scan_rows(asked, totals, scratch);
    const int tokens = min(totals[0], a.max_tokens);
    int given = totals[1];
    // More than the ring can hold: something else returned them already.
    if (given > a.pages - avail) {
        bad = true;
        given = 0;
    }
    int need[1][PER], own_need[PER], all_need[1];
    bool fits[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        fits[i] = held[i] >= 0 && int64_t(held[i]) + own_ask[i] <= room &&
                  int64_t(asked[0][i]) + own_ask[i] <= a.max_tokens;
        own_need[i] = need[0][i] = fits[i] ? pages_of(held[i] + own_ask[i]) - pages_of(held[i]) : 0;
    }
    scan_rows(need, all_need, scratch + 2);
    bool refused = false;
    int last = 0;  // pages taken up to this thread's last served request
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = tid * PER + i;
        if (r >= a.rows) continue;
        const bool served = fits[i] && (own_need[i] == 0 || sat_add(need[0][i], own_need[i]) <= avail);
        if (own_ask[i] > 0 && !served) refused = true;
        cu[r] = min(asked[0][i], a.max_tokens);
        at[r] = min(need[0][i], avail);
        to[r] = asked[1][i];
        lens[r] = held[i];
        grow[r] = n[i] > 0 ? (served ? n[i] : 0)
                           : (!odd && given >= own_back[i] ? max(n[i], -max(held[i], 0)) : 0);
        if (served && own_need[i] > 0) last = max(last, need[0][i] + own_need[i]);
    }
    // Pages taken in all: what the last served request's share ends with.
    last = int(__reduce_max_sync(0xffffffffu, unsigned(last)));
    if (bad || refused) atomicMax(&found, bad ? 2 : 1);
    if ((tid & 31) == 0) scratch[3][tid >> 5] = last;
    __syncthreads();
    const int grown = int(__reduce_max_sync(0xffffffffu, unsigned(scratch[3][tid & 31])));
    // One code a call, whichever threads find what: that of the lengths and the ring,
    // then refusals, then pages that are none.
    if (rank == 0 && tid == 0 && found != 0)
        hs::set_status(a.status, found == 2 ? HS_ERR_BAD_INDEX : HS_ERR_CAPACITY);
    const auto no_page = [&] {
        if (found == 0) hs::set_status(a.status, HS_ERR_BAD_INDEX);
    };
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
        a.table[r * a.bt_stride + pages_of(lens[r]) + i - at[r]] = a.ring[ring_at(take_at, i)];
    }
    for (int i = first; i < given; i += step) {
        const int r = find(to, a.rows, i);
        const int page = a.table[r * a.bt_stride + pages_of(lens[r] + grow[r]) + i - to[r]];
        if (page < 0 || page >= a.pages) no_page();
        a.ring[ring_at(give_at, i)] = page;
    }
    // The pages of kAtOnce tokens are read together.  (Four neighbouring tokens
    // with one search and wide stores: no faster.)
    for (int64_t t0 = first; t0 < a.max_tokens; t0 += int64_t(kAtOnce) * step) {
        int req[kAtOnce], pos[kAtOnce], in[kAtOnce], page[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t t = t0 + int64_t(k) * step;
            req[k] = pos[k] = page[k] = -1;
            in[k] = 0;
            if (t >= tokens) continue;
            const int r = find(cu, a.rows, int(t));
            if (grow[r] <= 0) continue;
            req[k] = r;
            pos[k] = lens[r] + int(t) - cu[r];
            const int b = page_of(pos[k]), have = pages_of(lens[r]);
            in[k] = pos[k] - b * B;
            page[k] = b < have ? a.table[r * a.bt_stride + b]
                               : a.ring[ring_at(take_at, at[r] + b - have)];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int64_t t = t0 + int64_t(k) * step;
            if (t >= a.max_tokens) break;
            const bool good = page[k] >= 0 && page[k] < a.pages;
            if (req[k] >= 0 && !good) no_page();
            a.slot[t] = good ? page[k] * B + in[k] : -1;
            a.row_req[t] = req[k];
            a.positions[t] = pos[k];
        }
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
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (page_size == (1 << i)) a.page_shift = i;
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
    // Four requests to a thread only where there are more than 1024: the chain of
    // their sums is the call's time.
    const bool one = rows <= kThreads;
    auto kern = one ? extend_kernel<1> : extend_kernel<kMaxRows / kThreads>;
    static int smem_set[2][64] = {};
    const int rc = hs_host::ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem,
                                                smem_set[one ? 0 : 1]);
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
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        cudaGetLastError();
        return HS_ERR_CUDA;
    }
    return HS_OK;
}
