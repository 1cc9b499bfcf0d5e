// quantize.hip -- expert weights into the FP8 block format of the grouped
// products: one fp32 scale per 128 x 128 block of a row-major [N, K] matrix.
//
// s = max(amax, 1e-4) / 448 over the block, q = e4m3(w / s): the dispatch's
// formula with the block in the place of a row's 128 channels. Four waves
// have one block, 32 rows each: lane l holds channels 16 (l % 8) .. + 15 of
// rows l / 8 + 8 p in registers, so w is read once, and only the largest
// magnitudes meet, in LDS. HBM-bound (2 bytes read and 1 written per weight):
// 32 matrices of 4096 x 7168 in 515 us, 5.5 TB/s; 96 blocks, latency, 4.3 us
// (one wave a block: 2 us more, and 20% slower on large matrices whose rows are
// a power of two apart). The loads have no nontemporal hint: a lane's 32 bytes
// are two loads, and with it half a line came from memory twice (542 us).
#include "experts_internal.h"
#include "fp8_device.h"

namespace epx {
namespace {

constexpr int kShare = 4;                  // waves of a block
constexpr int kQuantPasses = 16 / kShare;  // of 8 rows

__device__ __forceinline__ uint32_t code4(const float (&f)[16], int j, float s, float rs)
{
    const int w = cvt2_e4m3<false>(quotient(f[4 * j], s, rs), quotient(f[4 * j + 1], s, rs), 0);
    return (uint32_t)cvt2_e4m3<true>(quotient(f[4 * j + 2], s, rs),
                                     quotient(f[4 * j + 3], s, rs), w);
}

__global__ __launch_bounds__(kWave *kShare) void quantize_kernel(QuantizeArgs a, int nb)
{
    const int kblocks = a.K >> 7;
    int64_t b = blockIdx.x;
    const int kb = (int)(b % kblocks);
    b /= kblocks;
    const int n_blk = (int)(b % nb);
    const int64_t e = b / nb;
    __shared__ uint32_t meet_bits[kShare];
    __shared__ float meet_max[kShare];
    const int share = (int)(threadIdx.x >> 6), lane = lane_id();
    const int n0 = n_blk * 128 + share * (128 / kShare), r = lane >> 3;
    const int c = kb * 128 + (lane & 7) * 16;
    const int rows = min(128 / kShare, a.N - n0);  // of this wave (may be none)
    const int64_t base = (e * a.N + n0) * (int64_t)a.K + c;
    u32x4 lo[kQuantPasses], hi[kQuantPasses];
#pragma unroll
    for (int p = 0; p < kQuantPasses; ++p) {
        lo[p] = hi[p] = u32x4{0u, 0u, 0u, 0u};
        if (p * 8 + r < rows) {
            const uint16_t *src = a.w + base + (int64_t)(p * 8 + r) * a.K;
            lo[p] = load16(src);
            hi[p] = load16(src + 8);
        }
    }
    uint32_t abits = 0;
#pragma unroll
    for (int p = 0; p < kQuantPasses; ++p) {
        const uint32_t v[8] = {lo[p].x, lo[p].y, lo[p].z, lo[p].w,
                               hi[p].x, hi[p].y, hi[p].z, hi[p].w};
        abits = max(abits, seg_abs_max_bits(v));
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1)
        abits = max(abits, (uint32_t)__shfl_xor((int)abits, d, kWave));
    if (lane == 0)
        meet_bits[share] = abits;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kShare; ++w)
        abits = max(abits, meet_bits[w]);
    // a block holding an Inf or NaN divides outright, its largest magnitude
    // taken over the values that compare (uniform over the block's waves)
    const bool finite = abits < 0x7F80u;
    float s = group_scale(__uint_as_float(abits << 16));
    if (!finite) {
        float m = 0.0f;
        for (int p = 0; p < kQuantPasses; ++p) {
            const uint32_t v[8] = {lo[p].x, lo[p].y, lo[p].z, lo[p].w,
                                   hi[p].x, hi[p].y, hi[p].z, hi[p].w};
            for (int i = 0; i < 8; ++i)
                m = amax_of(amax_of(m, bf16_lo(v[i])), bf16_hi(v[i]));
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1)
            m = amax_of(m, __shfl_xor(m, d, kWave));
        if (lane == 0)
            meet_max[share] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kShare; ++w)
            m = amax_of(m, meet_max[w]);
        s = group_scale(m);
    }
    const float rs = 1.0f / s;
#pragma unroll
    for (int p = 0; p < kQuantPasses; ++p) {
        const uint32_t v[8] = {lo[p].x, lo[p].y, lo[p].z, lo[p].w,
                               hi[p].x, hi[p].y, hi[p].z, hi[p].w};
        float f[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[2 * i] = bf16_lo(v[i]);
            f[2 * i + 1] = bf16_hi(v[i]);
        }
        uint32_t q[4];
        if (finite) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = code4(f, j, s, rs);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = e4m3_of_quotient(f[4 * j], s) | (e4m3_of_quotient(f[4 * j + 1], s) << 8) |
                       (e4m3_of_quotient(f[4 * j + 2], s) << 16) |
                       (e4m3_of_quotient(f[4 * j + 3], s) << 24);
        }
        if (p * 8 + r < rows)
            store16_stream(a.codes + base + (int64_t)(p * 8 + r) * a.K,
                           u32x4{q[0], q[1], q[2], q[3]});
    }
    if (share == 0 && lane == 0)
        a.scales[(e * nb + n_blk) * (int64_t)kblocks + kb] = s;
}

}  // namespace

hipError_t launch_quantize_weights(const QuantizeArgs &a, hipStream_t stream)
{
    const int nb = (a.N + 127) / 128;
    const int64_t blocks = (int64_t)a.E * nb * (a.K >> 7);
    if (blocks == 0)
        return hipSuccess;
    if (blocks > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(quantize_kernel, dim3((unsigned)blocks), dim3(kWave * kShare), 0, stream, a,
                       nb);
    return hipGetLastError();
}

}  // namespace epx
