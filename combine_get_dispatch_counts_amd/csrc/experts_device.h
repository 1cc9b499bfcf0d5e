// experts_device.h -- device helpers shared by the experts' products (gfx950):
// which rows an expert has, matrix operands and the gated activation.
//
// Both products are computed as D = W X^T with 16 x 16 matrix instructions:
// the weights are the A operand, so a lane's four results are four
// consecutive output columns of ONE row (its lane % 16): a row's scale is one
// multiply per lane, and a store takes four columns at once. The channel
// order inside an operand is free as long as both sides use the same one.
#pragma once

#include "experts_internal.h"
#include "fp8_device.h"

namespace epx {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 128 channels of FP8 (32 bytes a lane).
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b, f32x4 c)
{
    // scale operands of constant 0 select the unscaled instruction
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// 32 channels of bf16 (16 bytes a lane).
__device__ __forceinline__ f32x4 mfma_bf16(i32x4 a, i32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32. exp as 2^(-g log2 e) and the
// reciprocal are the hardware's, each within an ulp; the argument of 2^x and
// the constant in it are rounded, which the exponential multiplies by g. Off
// by at most (8 + |g|) 2^-23 of the value: 5e-7 near zero, some 6e-6 for g =
// -80 (for g > 0 the exponential vanishes beside 1). Far below the bf16 or
// e4m3 rounding that follows, and as an error of the FP8 form's fp32 scales
// only where silu itself has gone to nothing. Below g = -87.3 the reciprocal,
// and below -88.7 the exponential's inverse, leave fp32's normal range: the
// quotient, 1e-36 at most, is zero.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// Rows of a region, kept inside it (bad: the count says otherwise).
__device__ __forceinline__ int region_rows(const GroupedArgs &a, int64_t region, bool &bad)
{
    const int c = a.counts[region];
    bad |= c > a.cap;
    return min(max(c, 0), a.cap);
}

// Rows of expert e where they lie together (expert-major, or one region):
// the first one and how many, kept inside the caller's buffer.
__device__ __forceinline__ int expert_rows(const GroupedArgs &a, int e, int64_t &first, bool &bad)
{
    if (a.off) {
        const int64_t lo = a.off[e], hi = a.off[e + 1];
        int64_t b = lo < 0 ? 0 : lo, t = hi;
        if (b > a.n_rows)
            b = a.n_rows;
        if (t > a.n_rows)
            t = a.n_rows;
        if (t < b)
            t = b;
        bad |= b != lo || t != hi;
        first = b;
        return (int)(t - b);
    }
    first = (int64_t)e * a.cap;
    return region_rows(a, e, bad);
}

// The rows of an expert spread over R_buf > 1 regions: lane s holds the rows
// of the regions up to s (R_buf <= 64). Every lane of a wave takes part.
struct Regions {
    int upto;
    __device__ __forceinline__ void load(const GroupedArgs &a, int e)
    {
        bool bad = false;
        const int s = lane_id();
        upto = wave_inclusive_sum(s < a.R_buf ? region_rows(a, (int64_t)e * a.R_buf + s, bad) : 0);
    }
    __device__ __forceinline__ int rows() const { return __builtin_amdgcn_readlane(upto, 63); }
    // row number i of the expert (0 <= i < rows()), counted from its first region
    __device__ __forceinline__ int row(const GroupedArgs &a, int i) const
    {
        int s = 0;
#pragma unroll
        for (int step = 32; step; step >>= 1)
            if (__shfl(upto, s + step - 1, kWave) <= i)
                s += step;
        const int before = __shfl(upto, max(s - 1, 0), kWave);
        return s * a.cap + i - (s ? before : 0);
    }
};

}  // namespace epx
