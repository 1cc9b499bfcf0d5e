// combine_backward.hip -- the combine's gradient: with out[t] = sum over k of
// w[t,k] y[pos[t,k]],
//   dy[pos[t,k]] = w[t,k] dout[t],   dw[t,k] = sum over channels dout[t] y[pos[t,k]].
//
// A block has one token and a wave one of its entries at a time: the wave
// holds the token's row in registers (its other waves find it in the cache),
// reads the entry's expert row once, stores the scaled row and sums the
// products over the wave. HBM-bound: per entry one row read and one written
// (4096 tokens of top-8 x 7168, 1 GB: 172-177 us, 5.7 TB/s). Few tokens are
// bound by the wave that has an entry, its loads and then its stores, and by
// the compute units without a block: 16 tokens 6.2 us, 128 9.9, 512 22.5 (5.5
// TB/s).
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

// Rows of at most 8 LANES channels: LANES lanes have an entry, a vector each, so
// a wave has two or four. (32768 tokens of top-8 x 128: 26.1 us, 5.5 TB/s; a
// wave an entry 83.7.)
constexpr int kNarrowThreads = 256;

template <int LANES>
__global__ __launch_bounds__(kNarrowThreads) void combine_narrow_backward_kernel(CombineBwdArgs a)
{
    const int i = threadIdx.x % LANES, nvec = a.h >> 3;
    const int64_t tk = (int64_t)blockIdx.x * (kNarrowThreads / LANES) + threadIdx.x / LANES;
    const bool entry = tk < (int64_t)a.T * a.K;
    const int p = entry ? a.pos[tk] : -1;
    const float w = entry ? a.topk_w[tk] : 0.0f;
    if (p >= a.n_rows && i == 0)
        flag_error(a.err, EPX_DEV_BAD_HANDLE);
    const bool live = p >= 0 && p < a.n_rows && i < nvec;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const size_t at = (size_t)(live ? (int64_t)p * a.h + i * 8 : 0);
    const u32x4 dv = live ? load16(a.dout + (size_t)((uint32_t)tk / (uint32_t)a.K) * a.h + i * 8)
                          : zero;
    const u32x4 yv = live && a.dtopk_w ? load16_stream(a.y + at) : zero;
    float d[8], y[8], dot = 0.0f;
    widen8(dv, d);
    widen8(yv, y);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        dot = __builtin_fmaf(d[c], y[c], dot);
    if (a.dy && live) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            d[c] *= w;
        store16_stream(a.dy + at, narrow8(d));
    }
    if (a.dtopk_w) {
        dot = group_sum<LANES>(dot);
        if (entry && i == 0)
            a.dtopk_w[tk] = dot;
    }
}

template <int LANES>
hipError_t launch_narrow(const CombineBwdArgs &a, hipStream_t stream)
{
    constexpr int kRows = kNarrowThreads / LANES;
    const int64_t blocks = ((int64_t)a.T * a.K + kRows - 1) / kRows;
    hipLaunchKernelGGL((combine_narrow_backward_kernel<LANES>), dim3((unsigned)blocks),
                       dim3(kNarrowThreads), 0, stream, a);
    return hipGetLastError();
}

// With many rows the sums and the scaled rows take a launch each: the token's
// row is read twice, but memory reads alone and then writes alone. One against
// two launches, top-8, h = 7168: 256 tokens (28 MB of expert rows) 12.2 / 11.9
// us, 512 23.4 / 22.4, 1024 49 / 45, 4096 202 / 172-177, 8192 376 / 332; h =
// 2048, 4096 tokens 58 / 52.5; top-6 x 4096, 4096 tokens 85 / 79. Where the
// token's row is a larger part, or rows are short, one launch: 8192 tokens of
// top-2 x 4096 53-55 / 62, of top-4 x 2048 51-55 / 53, of top-8 x 1024 52-58 /
// 57-62. (Rows written in their own order by a second launch that finds each
// one's token, which is sequential for memory but reads the tokens' rows eight
// times past the L2: 221 us for 4096 tokens of top-8 x 7168.)
bool split(const CombineBwdArgs &a)
{
    return a.dy && a.dtopk_w && a.K >= 6 && a.h >= 2048 &&
           (int64_t)a.T * a.K * a.h * 2 > (48ll << 20);
}

template <int NV>
hipError_t launch(const CombineBwdArgs &a, hipStream_t stream)
{
    if (split(a)) {
        CombineBwdArgs sums = a, rows = a;
        sums.dy = nullptr;
        rows.dtopk_w = nullptr;
        const hipError_t e = launch<NV>(sums, stream);
        return e != hipSuccess ? e : launch<NV>(rows, stream);
    }
    const int waves = a.K < 8 ? a.K : 8;
    hipLaunchKernelGGL((combine_backward_kernel<NV>), dim3((unsigned)a.T),
                       dim3((unsigned)waves * kWave), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// A step takes 1, 4 or 8 vectors of a lane, the least that hold the row, or 8
// where none does. With 1 / 4 / 8 of them 4096 tokens of top-8 take at 512
// channels 15.2 / 22.2 / 33.5 us, 1024 26.6 / 28.6 / 41, 2048 54 / 51 / 60, 4096
// 100 / 97.5 / 97, 7168 171 / 172 / 171; 64 tokens at 512 channels 2.1 / 2.7 /
// 3.4, 2048 3.0 / 3.2 / 3.8, 4096 5.2 / 4.7 / 4.7, 7168 11.1 / 9.3 / 8.0. More
// vectors leave fewer waves a SIMD and longer rows a second step that is mostly
// empty: 14 against 8, 4096 tokens of 5120 channels 133 / 128.5, 7168 174 / 174,
// 8192 209 / 191; 128 tokens 7.5 / 8.3, 9.9 / 9.9 and 13.7 / 11.
static hipError_t launch_tokens(const CombineBwdArgs &a, hipStream_t stream)
{
    if (a.h <= 128)
        return launch_narrow<16>(a, stream);
    if (a.h <= 256)
        return launch_narrow<32>(a, stream);
    if (a.h <= 512)
        return launch<1>(a, stream);
    if (a.h <= 2048)
        return launch<4>(a, stream);
    return launch<8>(a, stream);
}

hipError_t launch_combine_backward(const CombineBwdArgs &args, hipStream_t stream)
{
    // a launch has at most 2^31 threads (8 waves a token, or 32 lanes an entry
    // of up to 32): more tokens go in several
    const int64_t most = 1ll << 21;
    CombineBwdArgs a = args;
    for (int64_t t = 0; t < args.T; t += most) {
        a.T = (int)(args.T - t < most ? args.T - t : most);
        const hipError_t e = launch_tokens(a, stream);
        if (e != hipSuccess)
            return e;
        a.dout += most * a.h;
        a.topk_w += most * a.K;
        a.pos += most * a.K;
        if (a.dtopk_w)
            a.dtopk_w += most * a.K;
    }
    return hipSuccess;
}

}  // namespace epx
