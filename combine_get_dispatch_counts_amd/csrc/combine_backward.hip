// combine_backward.hip -- the combine's gradient: with out[t] = sum over k of
// w[t,k] y[pos[t,k]],
//   dy[pos[t,k]] = w[t,k] dout[t],   dw[t,k] = sum over channels dout[t] y[pos[t,k]].
//
// A block has one token and a wave one of its entries at a time: the wave
// holds the token's row in registers (its other waves find it in the cache),
// reads the entry's expert row once, stores the scaled row and sums the
// products over the wave. HBM-bound: per entry one row read and one written.
#include "gate_device.h"

namespace epx {
namespace {

template <int NV>
__global__ __launch_bounds__(kWave * 8) void combine_backward_kernel(CombineBwdArgs a)
{
    const int64_t t = blockIdx.x;
    const int waves = blockDim.x >> 6, nvec = a.h >> 3;
    const uint32_t bytes = (uint32_t)nvec * 16u;
    const int lane = lane_id();
    const __amdgpu_buffer_rsrc_t rd = row_rsrc(a.dout + (size_t)t * a.h, bytes);
    for (int k = threadIdx.x >> 6; k < a.K; k += waves) {
        const int64_t tk = t * a.K + k;
        const int p = __builtin_amdgcn_readfirstlane(a.pos[tk]);
        const float w = a.topk_w[tk];
        bool live = p >= 0;
        if (live && p >= a.n_rows) {
            if (lane == 0)
                flag_error(a.err, EPX_DEV_BAD_HANDLE);
            live = false;
        }
        float dot = 0.0f;
        if (live) {
            for (int v0 = 0; v0 < nvec; v0 += NV * kWave) {
                u32x4 dv[NV], yv[NV];
#pragma unroll
                for (int u = 0; u < NV; ++u)
                    dv[u] = __builtin_amdgcn_raw_buffer_load_b128(
                        rd, (int)((uint32_t)(v0 + u * kWave + lane) * 16u), 0, 0);
                if (a.dtopk_w) {
                    const __amdgpu_buffer_rsrc_t ry = row_rsrc(a.y + (size_t)p * a.h, bytes);
#pragma unroll
                    for (int u = 0; u < NV; ++u)
                        yv[u] = load16_row(ry, (uint32_t)(v0 + u * kWave + lane) * 16u);
                }
                if (a.dy) {
                    uint16_t *row = a.dy + (size_t)p * a.h;
#pragma unroll
                    for (int u = 0; u < NV; ++u) {
                        float d[8];
                        widen8(dv[u], d);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[i] *= w;
                        const int v = v0 + u * kWave + lane;
                        if (v < nvec)
                            store16_stream(row + (size_t)v * 8, narrow8(d));
                    }
                }
                if (a.dtopk_w) {
#pragma unroll
                    for (int u = 0; u < NV; ++u) {
                        float d[8], y[8];
                        widen8(dv[u], d);
                        widen8(yv[u], y);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dot = __builtin_fmaf(d[i], y[i], dot);
                    }
                }
            }
        }
        if (a.dtopk_w) {
            dot = wave_sum(dot);
            if (lane == 0)
                a.dtopk_w[tk] = dot;
        }
    }
}

template <int NV>
hipError_t launch(const CombineBwdArgs &a, hipStream_t stream)
{
    const int waves = a.K < 8 ? a.K : 8;
    hipLaunchKernelGGL((combine_backward_kernel<NV>), dim3((unsigned)a.T),
                       dim3((unsigned)waves * kWave), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_backward(const CombineBwdArgs &a, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (a.h <= 512)
        return launch<1>(a, stream);
    if (a.h <= 2048)
        return launch<4>(a, stream);
    if (a.h <= 4096)
        return launch<8>(a, stream);
    return launch<14>(a, stream);
}

}  // namespace epx
