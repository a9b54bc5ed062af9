// hs_plan.h -- integer arithmetic of how calls are cut into work.  Plain C++, so
// that it is checked on the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define HS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define HS_HOST_DEVICE inline
#endif

namespace hs_plan {

// Sums of lengths stop here: above anything that a call holds (2^30), and two of
// them still fit 32 bits without a sign.
constexpr int kSatMax = (1 << 30) + 1;

// a + b of [0, kSatMax], at most kSatMax.
HS_HOST_DEVICE int sat_add(int a, int b) {
    const uint32_t s = uint32_t(a) + uint32_t(b);
    return s < uint32_t(kSatMax) ? int(s) : kSatMax;
}

// Where a request's new tokens stand in a call of hs_paged_prefill, and its cached
// tokens.  Queries before position 0 attend to nothing and are no part of the work:
// n does not count them, and first stands behind them.
struct Request {
    int32_t first, n, T;
    int32_t blind;  // those queries, rows [first - blind, first)
};
HS_HOST_DEVICE int32_t within(int32_t x, int32_t most) { return x < 0 ? 0 : x < most ? x : most; }
// c0, c1: its entries of cu_new; held: its cached tokens as given.
HS_HOST_DEVICE Request request(int32_t c0, int32_t c1, int32_t held, int32_t tokens,
                               int32_t max_len) {
    Request x;
    x.first = within(c0, tokens);
    x.n = within(c1, tokens) - x.first;
    if (x.n < 0) x.n = 0;
    x.T = within(held, max_len);
    x.blind = x.n > x.T ? x.n - x.T : 0;
    x.first += x.blind;
    x.n -= x.blind;
    return x;
}

// Places of a request's blocks of tb new tokens: what they weigh when the work is
// dealt to the CTAs.  Block i sees up to position base + (i + 1) tb, with base = T -
// n, and, with a window, from base + i tb + 1 - window on (the grid of tiles, the
// sinks and a last block that is not full do not count); extra: its other work.
HS_HOST_DEVICE int places_of_block(const Request& x, int32_t tb, int32_t window, int32_t extra,
                                   int b) {
    const int base = x.T - x.n, from = base + b * tb + 1 - window;
    return extra + base + (b + 1) * tb - (window > 0 && from > 0 ? from : 0);
}
// Of the first b blocks, in closed form.
HS_HOST_DEVICE int64_t places_of_blocks(const Request& x, int32_t tb_, int32_t window,
                                        int32_t extra, int b) {
    const int64_t base = x.T - x.n, tb = tb_, n = b;
    int64_t sum = n * (extra + base) + tb * (n * (n + 1) / 2);
    if (window > 0) {
        const int64_t c0 = base + 1 - window;
        const int64_t i0 = c0 > 0 ? 0 : int(-c0) / tb_ + 1;  // the first block that starts behind 0
        if (n > i0) sum -= (n - i0) * c0 + tb * (n * (n - 1) / 2 - i0 * (i0 - 1) / 2);
    }
    return sum;
}

}  // namespace hs_plan
