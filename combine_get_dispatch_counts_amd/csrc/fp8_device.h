// fp8_device.h -- e4m3 rows of fp32 values in the dispatch's format.
#pragma once

#include "dispatch_device.h"

namespace epx {

// Group scale of a largest magnitude: max(amax, 1e-4) / 448, both fp32.
__device__ __forceinline__ float group_scale(float amax) { return fmaxf(amax, 1e-4f) / 448.0f; }

// The larger of a running magnitude and |v|; a NaN never wins.
__device__ __forceinline__ float amax_of(float m, float v)
{
    const float a = fabsf(v);
    return a > m ? a : m;
}

// e4m3 code of v / s (the IEEE quotient, nearest even; NaN quotients 0x7F).
// |v / s| <= 448 up to one rounding for finite v, so no saturation is needed:
// the convert is exact up to 464. An infinite v has an infinite s, and their
// quotient is a NaN.
__device__ __forceinline__ uint32_t e4m3_of_quotient(float v, float s)
{
    const float q = v / s;
    return (q != q) ? 0x7Fu : ((uint32_t)cvt2_e4m3<false>(q, 0.0f, 0) & 0xFFu);
}

}  // namespace epx
