// gate_device.h -- device helpers of the norm, the choice of experts and the
// gradients (gfx950): reductions over a wave, the exponential, bf16 vectors.
#pragma once

#include "epx_device.h"
#include "gate_internal.h"

namespace epx {

// Reductions with data-parallel-primitive moves between lanes (no LDS). The
// order of a sum's additions is fixed.
#define EPX_DPP(v, ident, ctrl, rows) \
    __builtin_amdgcn_update_dpp((int)(ident), (int)(v), ctrl, rows, 0xF, false)

__device__ __forceinline__ float last_lane(float v)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Over the 64 lanes of a wave: 16 lanes by shifts within a row, the rows joined
// by two broadcasts; lane 63 ends with the whole, which every lane gets.
__device__ __forceinline__ float wave_sum(float v)
{
#define EPX_STEP(ctrl, rows) \
    v = v + __int_as_float(EPX_DPP(__float_as_int(v), 0, ctrl, rows))
    EPX_STEP(0x111, 0xF);  // row_shr:1
    EPX_STEP(0x112, 0xF);
    EPX_STEP(0x114, 0xF);
    EPX_STEP(0x118, 0xF);
    EPX_STEP(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
    EPX_STEP(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef EPX_STEP
    return last_lane(v);
}

// Over each 16 adjacent lanes (a row), the result in all 16 of them: rotations
// pair the same values in every lane, so a sum is the same in each.
#define EPX_ROW(v, ctrl) __builtin_amdgcn_mov_dpp((int)(v), ctrl, 0xF, 0xF, true)

__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, (uint32_t)EPX_ROW(v, 0x128));  // row_ror:8
    v = max(v, (uint32_t)EPX_ROW(v, 0x124));
    v = max(v, (uint32_t)EPX_ROW(v, 0x122));
    return max(v, (uint32_t)EPX_ROW(v, 0x121));
}

// (In assembly: the compiler spends four instructions a step on a maximum of
// numbers that may be NaN. The two wait states between a vector write and its
// use by another lane are in the block.)
__device__ __forceinline__ float row_max(float v)
{
    asm("s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_ror:4 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_ror:2 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 row_ror:1 row_mask:0xf bank_mask:0xf\n\t"
        "s_nop 1"
        : "+v"(v));
    return v;
}

__device__ __forceinline__ float row_sum(float v)
{
#define EPX_STEP(ctrl) v = v + __int_as_float(EPX_ROW(__float_as_int(v), ctrl))
    EPX_STEP(0x128);
    EPX_STEP(0x124);
    EPX_STEP(0x122);
    EPX_STEP(0x121);
#undef EPX_STEP
    return v;
}

// Over a wave's groups of LANES (16 or 32) adjacent lanes.
template <int LANES>
__device__ __forceinline__ float group_sum(float v)
{
    v = row_sum(v);
    if constexpr (LANES == 32)
        v += __shfl_xor(v, 16, kWave);
    return v;
}

// The row's 16 bits of a ballot.
__device__ __forceinline__ uint32_t row_ballot(bool b)
{
    const uint64_t m = __ballot(b);
    const int row = lane_id() >> 4;
    return (uint32_t)((row & 2 ? m >> 32 : m) >> (16 * (row & 1))) & 0xFFFFu;
}

// exp(x) in fp32 within two units of the last place for results in the normal
// range: the hardware's 2^t (one unit) at t = x log2 e, and the part of the
// product that its rounding drops -- up to |x| 2^-24 of the result -- put back
// as a factor. Below -200 the result is 0, as it is from -104 on.
__device__ __forceinline__ float exp_fp32(float x)
{
    x = fmaxf(x, -200.0f);
    const float t = x * 0x1.715476p+0f;
    const float r = __builtin_fmaf(x, 0x1.4ae0cp-26f, __builtin_fmaf(x, 0x1.715476p+0f, -t));
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, 0x1.62e43p-1f, 1.0f);
}

__device__ __forceinline__ void widen8(const u32x4 &p, float (&f)[8])
{
    const uint32_t e[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(e[i]);
        f[2 * i + 1] = bf16_hi(e[i]);
    }
}

// Two fp32 values rounded to bf16, nearest even, by gfx950's convert (a fifth of
// f32_to_bf16's instructions; a NaN stays one, not the canonical one).
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t,
                              __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

__device__ __forceinline__ u32x4 narrow8(const float (&f)[8])
{
    return u32x4{narrow2(f[0], f[1]), narrow2(f[2], f[3]), narrow2(f[4], f[5]),
                 narrow2(f[6], f[7])};
}

}  // namespace epx
