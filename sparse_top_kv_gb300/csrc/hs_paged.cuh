// hs_paged.cuh -- attention of one new token per request over every cached
// token of a paged KV cache: arguments, work plan and helpers shared by the
// attention kernels (hs_paged_core.cuh, one translation unit per cache type)
// and the dispatcher with its finishing kernels (hs_paged.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "hs_common.cuh"

namespace hs_paged {

constexpr int kKey = 16;           // cached tokens per warp step
constexpr int kMaxHeads = 65536;
constexpr int kMaxRows = 4096;     // requests of one call (their plan sits in shared memory)
constexpr int kMaxCtas = 1024;     // most CTAs of the attention kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PagedArgs {
    const void* q;  // [rows, heads, D], rows q_stride elements apart
    const void* k;
    const void* v;
    int64_t q_stride, page_stride, row_stride, head_stride;  // elements
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* seq_lens;
    const float* k_scale;  // [kv_heads] or nullptr (E4M3)
    const float* v_scale;
    int32_t rows, heads, kv_heads, group, num_pages, page_size, max_len, window, sinks;
    int32_t page_shift;   // log2 of page_size, or -1
    int32_t q_is_half;  // E4M3 caches: the query is fp16 (else bf16)
    float scale_log2;   // scale * log2(e)
    void* out;          // [rows, heads, D]
    float* lse;         // [rows, heads] or nullptr
    float* score;       // [rows, score_stride] or nullptr
    int64_t score_stride;
    float decay;
    // The two ways to cut the call (below).
    int32_t hs[2], lth[2], chunks[2], gm, extra;
    int64_t wide_from, wide_to;  // places (way 0) between which way 0 is taken
    int32_t cl;  // > 0: a cluster of cl CTAs per unit (way 1) in place of the deal of tiles
    // Workspace.
    float* lse2;        // [rows, heads] log2 units (scored calls)
    float* part_ml;     // [2 * ctas][unit heads][2]
    float* part_o;      // [2 * ctas][unit heads][D]
    float* logits;      // [rows, heads, logit_stride] log2 units (scored calls)
    int64_t logit_stride;
    int32_t unit_heads_max;
    int32_t ctas;
    int32_t* status;
};

// How a call is cut into work.  A unit is one request x one chunk of its
// heads (hs KV heads, up to gm query heads of each); its tokens are cut into
// tiles of 2^lth.  The units' tiles, one after another, are dealt to the CTAs
// in equal contiguous runs, so ragged batches load every SM alike and one
// long context uses all of them.  Starting and ending a unit takes as long as
// a few tiles; each unit has that many places without work (`extra`) ahead of
// its tiles, so that a run of many short units holds fewer tiles (64 ragged
// E4M3 requests: the slowest CTA 85 us, 95 without).  There are two ways: units
// of as many heads as a tile holds (way 0: long DRAM pieces), or of one (way 1: small calls,
// fewer parts to merge); the kernels take one by the tiles that they find.
// Calls that are surely small are not dealt: each unit has a cluster of CTAs
// to itself, which join their parts through distributed shared memory.

// Token tiles of a request: those of the sinks, then those of the window,
// both on the grid of 2^lth tokens.  Attended are the first sc tokens and
// those from w0 on.
struct Tiling {
    int T, sc, w0, ns, tw0, n;
};
__device__ __forceinline__ Tiling tiling_of(const PagedArgs& a, int len, int lth) {
    Tiling v;
    v.T = min(max(len, 0), a.max_len);
    const int wc = a.window > 0 ? min(v.T, a.window) : v.T;
    v.w0 = v.T - wc;
    v.sc = a.window > 0 ? min(a.sinks, v.w0) : 0;
    v.tw0 = v.w0 >> lth;
    const int up = (1 << lth) - 1;
    v.ns = min((v.sc + up) >> lth, v.tw0);
    v.n = v.ns + ((v.T + up) >> lth) - v.tw0;  // 0: no token (the merge writes zeros)
    return v;
}

// Walks the tiles of a CTA's run; every role of the CTA walks alike.
struct Cursor {
    int row, chunk, tile, left;  // left: tiles of the run still to come, this one included
    bool first;                  // this tile starts a segment (a unit, or the run)
    Tiling v;
};
__device__ __forceinline__ bool last_of_segment(const Cursor& c) {
    return c.left == 1 || c.tile == c.v.n - 1;
}
__device__ __forceinline__ void advance(Cursor& c, const PagedArgs& a, int chunks, int lth) {
    c.first = false;
    --c.left;
    if (++c.tile < c.v.n || c.left == 0) return;
    c.tile = 0;
    c.first = true;
    if (++c.chunk < chunks) return;
    c.chunk = 0;
    do {  // the next request with a token; there is one, as left > 0
        ++c.row;
        c.v = tiling_of(a, a.seq_lens[c.row], lth);
    } while (c.v.n == 0 && c.row + 1 < a.rows);
}
// On to the run's next segment (left = 0: there is none).
__device__ __forceinline__ void next_segment(Cursor& c, const PagedArgs& a, int chunks, int lth) {
    const int n = min(c.left, c.v.n - c.tile);
    c.left -= n - 1;
    c.tile += n - 1;
    advance(c, a, chunks, lth);
}
__device__ __forceinline__ int tile_token(const Cursor& c, int lth) {
    return (c.tile < c.v.ns ? c.tile : c.tile - c.v.ns + c.v.tw0) << lth;
}
__device__ __forceinline__ bool visible(const Tiling& v, int t) {
    return t < v.T && (t < v.sc || t >= v.w0);
}
// Block of the page table that holds token t.
__device__ __forceinline__ int block_of(const PagedArgs& a, int t) {
    return a.page_shift >= 0 ? t >> a.page_shift : t / a.page_size;
}
// Place of an attended token among them.
__device__ __forceinline__ int visible_index(const Tiling& v, int t) {
    return t < v.sc ? t : t - v.w0 + v.sc;
}
// Whether any of the tokens [t, t + n) is attended to.
__device__ __forceinline__ bool any_visible(const Tiling& v, int t, int n) {
    return t < v.T && (t < v.sc || t + n > v.w0);
}

// floor(x / d) for 0 <= x < 2^23, by a float estimate and one correction (an
// integer division is a routine of many instructions).
__device__ __forceinline__ int div_small(int x, int d) {
    int q = __float2int_rz(__fdividef(float(x), float(d)));
    const int r = x - q * d;
    if (r < 0) --q;
    if (r >= d) ++q;
    return q;
}

// The runs of a call: places (tiles and extras) dealt to CTAs.
struct Plan {
    int tiles, n;   // places of the call, CTAs that share them
    int per, rest;  // tiles / n, tiles % n
};
// Places of one chunk of heads of a request with n tiles.
__device__ __forceinline__ int places(const PagedArgs& a, int n) { return n > 0 ? n + a.extra : 0; }
__device__ __forceinline__ Plan plan_of(const PagedArgs& a, int way, int total) {
    Plan p;
    p.tiles = total * a.chunks[way];
    p.n = max(1, min(a.ctas, p.tiles));
    p.per = p.tiles / p.n;
    p.rest = p.tiles - p.per * p.n;
    return p;
}
// floor(tiles c / n); rest, c <= n <= kMaxCtas
__device__ __forceinline__ int run_begin(const Plan& p, int c) {
    return p.per * c + div_small(p.rest * c, p.n);
}
__device__ __forceinline__ int run_of(const Plan& p, int tile) {
    int c = min(p.n - 1, __float2int_rz(float(tile) * __fdividef(float(p.n), float(p.tiles))));
    while (run_begin(p, c) > tile) --c;
    while (c + 1 < p.n && run_begin(p, c + 1) <= tile) ++c;
    return c;
}
__device__ __forceinline__ int way_of(const PagedArgs& a, int total0) {
    const int64_t n = int64_t(total0) * a.chunks[0];
    return n >= a.wide_from && n < a.wide_to ? 0 : 1;
}

// One CTA's run: `run` tiles from `tile` of chunk `chunk` of request `row` on.
struct Run {
    int way, chunks, run, row, chunk, tile;
    int len;  // of that request
};
// Every warp finds it for itself: a lane per request, a few dozen shuffles and
// no barrier, so each role starts as soon as the lengths have arrived.
__device__ __forceinline__ Run make_run(const PagedArgs& a, int cta) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    int len = 0, t0 = 0, t1 = 0;  // one request's length and tiles
    int n0 = 0, n1 = 0;           // places of this lane's
#pragma unroll 4
    for (int r = lane; r < a.rows; r += 32) {
        len = a.seq_lens[r];
        t0 = tiling_of(a, len, a.lth[0]).n;
        t1 = tiling_of(a, len, a.lth[1]).n;
        n0 += places(a, t0);
        n1 += places(a, t1);
    }
    n0 = __reduce_add_sync(kAll, n0);
    Run x;
    x.way = way_of(a, n0);
    const bool narrow = x.way != 0;
    x.chunks = a.chunks[x.way];
    const Plan pl = plan_of(a, x.way, narrow ? __reduce_add_sync(kAll, n1) : n0);
    const int v0 = cta < pl.n ? run_begin(pl, cta) : pl.tiles;
    const int v1 = cta < pl.n ? run_begin(pl, cta + 1) : pl.tiles;
    // The requests that places v0 and v1 lie in (the last whose first place is
    // at or before them; requests without tiles share theirs with the next),
    // and how many tiles come before each place.
    x.row = x.chunk = x.tile = x.len = 0;
    int before0 = 0, before1 = 0;
    for (int r0 = 0, tiles = 0, place = 0; r0 < a.rows; r0 += 32) {
        const int r = r0 + lane;
        int n = narrow ? t1 : t0;
        if (a.rows > 32) {
            len = r < a.rows ? a.seq_lens[r] : 0;
            n = tiling_of(a, len, a.lth[x.way]).n;
        } else if (r >= a.rows) {
            n = 0;
        }
        const int np = places(a, n);
        const int at = place + hs::warp_incl_scan(np) - np;      // places before request r
        const int tl = tiles + hs::warp_incl_scan(n) - n;        // tiles before it
        const bool in = r < a.rows;
        const uint32_t m0 = __ballot_sync(kAll, in && at * x.chunks <= v0);
        const uint32_t m1 = __ballot_sync(kAll, in && at * x.chunks <= v1);
        auto find = [&](uint32_t m, int v, int& chunk, int& tile) {
            const int last = 31 - __clz(m);
            const int f_at = __shfl_sync(kAll, at, last), f_tl = __shfl_sync(kAll, tl, last);
            const int f_n = __shfl_sync(kAll, n, last), f_p = __shfl_sync(kAll, np, last);
            const uint32_t rel = uint32_t(v - f_at * x.chunks);
            chunk = f_p > 0 ? min(int(rel / uint32_t(f_p)), x.chunks) : 0;
            tile = chunk < x.chunks ? max(0, int(rel) - chunk * f_p - a.extra) : 0;
            return f_tl * x.chunks + chunk * f_n + tile;
        };
        int c1, i1;
        if (m0 != 0) {
            before0 = find(m0, v0, x.chunk, x.tile);
            x.row = r0 + 31 - __clz(m0);
            x.len = __shfl_sync(kAll, len, 31 - __clz(m0));
        }
        if (m1 != 0) before1 = find(m1, v1, c1, i1);
        tiles = __shfl_sync(kAll, tl + n, 31);
        place = __shfl_sync(kAll, at + np, 31);
        if (place * x.chunks > v1) break;
    }
    x.run = before1 - before0;
    return x;
}
// The run of a CTA that shares its unit with the other CTAs of its cluster.
__device__ __forceinline__ Run unit_run(const PagedArgs& a, int unit, int rank) {
    Run x;
    x.way = 1;
    x.chunks = a.chunks[1];
    x.row = unit / x.chunks;
    x.chunk = unit - x.row * x.chunks;
    x.len = a.seq_lens[x.row];
    const int n = tiling_of(a, x.len, a.lth[1]).n;
    x.tile = n * rank / a.cl;
    x.run = n * (rank + 1) / a.cl - x.tile;
    return x;
}
// A length past max_len is reported once.
__device__ __forceinline__ void report_lengths(const PagedArgs& a) {
    for (int r = threadIdx.x; r < a.rows; r += blockDim.x)
        if (a.seq_lens[r] > a.max_len) hs::set_status(a.status, HS_ERR_BAD_INDEX);
}
__device__ __forceinline__ Cursor cursor_at(const PagedArgs& a, const Run& x) {
    Cursor c;
    c.row = x.row;
    c.v = tiling_of(a, x.len, a.lth[x.way]);
    c.chunk = x.chunk;
    c.tile = x.tile;
    c.left = x.run;
    c.first = true;
    return c;
}

// Host: the two ways of a kernel whose tiles have tile_rows cache rows and at
// most hs_max heads.
inline void set_ways(PagedArgs& a, int hs_max, int tile_rows, int gm, int tiles_for_wide,
                     int extra) {
    const int gch = (a.heads / a.kv_heads + gm - 1) / gm;
    int hs = 1;
    while (hs < hs_max && a.kv_heads % (2 * hs) == 0) hs *= 2;
    for (int way = 0; way < 2; ++way) {
        a.hs[way] = way == 0 ? hs : 1;
        a.lth[way] = 0;
        while ((a.hs[way] << (a.lth[way] + 1)) <= tile_rows) ++a.lth[way];
        a.chunks[way] = a.kv_heads / a.hs[way] * gch;
    }
    a.gm = gm;
    a.extra = extra;
    a.wide_from = int64_t(a.ctas) * tiles_for_wide;
    a.wide_to = INT64_MAX;
}

// Host: at most this many tiles of 2^lth tokens in one unit, by the bound on
// the lengths.
inline int64_t most_tiles(const PagedArgs& a, int lth) {
    const int64_t up = (int64_t(1) << lth) - 1;
    const int64_t all = (a.max_len + up) >> lth;
    if (a.window == 0) return all;
    return hs::min64(all, ((a.sinks + up) >> lth) + ((a.window + up) >> lth) + 1);
}

// Host: at most this many places in way `way`, by the bound on the lengths.
inline int64_t most_places(const PagedArgs& a, int way = 0) {
    const int64_t vis = a.window > 0 ? hs::min64(a.max_len, int64_t(a.window) + a.sinks) : a.max_len;
    return int64_t(a.rows) * a.chunks[way] * ((vis >> a.lth[way]) + 3 + a.extra);
}

int launch_bf16(PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_fp16(PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_e4m3(PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_bf16(PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_fp16(PagedArgs& a, int d, int group, hs_stream_t stream);
int launch_tc_e4m3(PagedArgs& a, int d, int group, hs_stream_t stream);

}  // namespace hs_paged
