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

}  // namespace hs_plan
