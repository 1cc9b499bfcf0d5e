// norm.hip -- root-mean-square norm of a residual stream's rows, with the
// residual's addition and the dispatch's FP8 rows, and its gradient.
//
// Forward, per row: v = x + residual (fp32), inv = 1 / sqrt(mean(v^2) + eps),
// y = v inv w. A block has one row, held in registers from its loads to its
// stores, so the row is read once whatever is written of it: the sum in bf16
// (the stream's next value), y in bf16, and y as e4m3 codes with a scale per
// 128 channels. Both forms of y are rounded once, from fp32.
//
// Backward, per row, with n = v inv and g = dout w:
//   dx = dres + inv (g - n mean(g n)),   dw = sum over rows of dout n.
// mean(g n) = inv mean(g v), so both row sums (v^2 and g v) come from one
// pass. A block walks rows b, b + blocks, ... with its share of dw in
// registers and leaves one row of partial sums, which a second launch adds in
// block order.
#include "fp8_device.h"
#include "gate_device.h"

namespace epx {
namespace {

constexpr int kMaxWaves = 16;

// The compiler forgets what it knows of a value (no instruction).
__device__ __forceinline__ void opaque(u32x4 &v) { asm volatile("" : "+v"(v)); }

template <bool WF32>
struct Weight8 {
    u32x4 lo, hi;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t v)
    {
        if constexpr (WF32) {
            lo = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(v * 32u), 0, 0);
            hi = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(v * 32u + 16u), 0, 0);
        } else {
            lo = __builtin_amdgcn_raw_buffer_load_b128(r, (int)(v * 16u), 0, 0);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if constexpr (WF32) {
            const uint32_t e[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __uint_as_float(e[i]);
        } else {
            widen8(lo, f);
        }
    }
};

// Codes of a lane's 8 channels; 16 adjacent lanes hold a group of 128, whose
// scale they all return.
__device__ __forceinline__ float codes8(const float (&y)[8], uint32_t &q0, uint32_t &q1)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    m = row_max(m);
    if (__builtin_expect(__ballot(m >= 0x7F800000u) == 0, 1)) {
        const float s = group_scale(__uint_as_float(m));
        const float rs = 1.0f / s;
        int w = cvt2_e4m3<false>(quotient(y[0], s, rs), quotient(y[1], s, rs), 0);
        q0 = (uint32_t)cvt2_e4m3<true>(quotient(y[2], s, rs), quotient(y[3], s, rs), w);
        w = cvt2_e4m3<false>(quotient(y[4], s, rs), quotient(y[5], s, rs), 0);
        q1 = (uint32_t)cvt2_e4m3<true>(quotient(y[6], s, rs), quotient(y[7], s, rs), w);
        return s;
    }
    // an Inf or NaN in one of the wave's groups: the largest magnitude that
    // compares, and quotients outright
    float f = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f = amax_of(f, y[i]);
    const float s = group_scale(__uint_as_float(row_max(__float_as_uint(f))));
    q0 = q1 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q0 |= e4m3_of_quotient(y[i], s) << (8 * i);
        q1 |= e4m3_of_quotient(y[4 + i], s) << (8 * i);
    }
    return s;
}

template <int NV, bool FP8, bool WF32>
__global__ __launch_bounds__(kWave *kMaxWaves) void norm_kernel(NormArgs a)
{
    __shared__ float sums[kMaxWaves];
    __shared__ float scales[FP8 ? kMaxWaves * NV * 4 : 1];
    const int tid = threadIdx.x, threads = blockDim.x;
    const int nvec = a.h >> 3;
    const size_t row = blockIdx.x;
    const __amdgpu_buffer_rsrc_t rx = row_rsrc(a.x + row * a.h, (uint32_t)nvec * 16u);
    const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.w, (uint32_t)nvec * (WF32 ? 32u : 16u));
    u32x4 xv[NV], rv[NV];
    Weight8<WF32> wv[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u)
        xv[u] = load16_row(rx, (uint32_t)(u * threads + tid) * 16u);
    if (a.residual) {
        const __amdgpu_buffer_rsrc_t rr = row_rsrc(a.residual + row * a.h, (uint32_t)nvec * 16u);
#pragma unroll
        for (int u = 0; u < NV; ++u)
            rv[u] = load16_row(rr, (uint32_t)(u * threads + tid) * 16u);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
        wv[u].load(rw, (uint32_t)(u * threads + tid));

    float v[NV][8], ss = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
        widen8(xv[u], v[u]);
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float r[8];
            widen8(rv[u], r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[u][i] += r[i];
            const int c = u * threads + tid;
            if (c < nvec)
                *reinterpret_cast<u32x4 *>(a.res_out + row * a.h + (size_t)c * 8) = narrow8(v[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = __builtin_fmaf(v[u][i], v[u][i], ss);
    ss = wave_sum(ss);
    const int waves = threads >> 6;
    if (waves > 1) {
        if (lane_id() == 0)
            sums[tid >> 6] = ss;
        __syncthreads();
        ss = 0.0f;
        for (int w = 0; w < waves; ++w)
            ss += sums[w];
    }
    const float inv = 1.0f / __builtin_sqrtf(ss / (float)a.h + a.eps);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float w[8], y[8];
        wv[u].get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = v[u][i] * inv * w[i];
        const int c = u * threads + tid;
        if (a.out && c < nvec)
            *reinterpret_cast<u32x4 *>(a.out + row * a.h + (size_t)c * 8) = narrow8(y);
        if constexpr (FP8) {
            uint32_t q0, q1;
            const float s = codes8(y, q0, q1);
            if (c < nvec) {
                *reinterpret_cast<uint2 *>(a.codes + row * a.h + (size_t)c * 8) = uint2{q0, q1};
                if ((tid & 15) == 0)
                    scales[c >> 4] = s;
            }
        }
    }
    if constexpr (FP8) {
        __syncthreads();
        const int stride = scale_stride(a.h), groups = a.h >> 7;
        for (int g = tid; g < stride; g += threads)
            a.scales[row * stride + g] = g < groups ? scales[g] : 0.0f;
    }
}

template <int NV, bool WF32>
__global__ __launch_bounds__(kWave *kMaxWaves) void norm_backward_kernel(NormBwdArgs a)
{
    // the next row's loads go out before this row's sums meet, where the
    // registers hold both rows
    constexpr bool kAhead = NV <= 2;
    __shared__ float2 sums[2][kMaxWaves];
    const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
    const int nvec = a.h >> 3;
    const uint32_t bytes = (uint32_t)nvec * 16u;
    const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.w, (uint32_t)nvec * (WF32 ? 32u : 16u));
    Weight8<WF32> wv[NV];
    float dw[NV][8];
    struct Row {
        u32x4 x[NV], d[NV], s[NV];
    } now, next;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        wv[u].load(rw, (uint32_t)(u * threads + tid));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dw[u][i] = 0.0f;
    }
    const auto load = [&](Row &r, size_t t) {
        const __amdgpu_buffer_rsrc_t rx = row_rsrc(a.x + t * a.h, bytes);
        const __amdgpu_buffer_rsrc_t rd = row_rsrc(a.dout + t * a.h, bytes);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            r.x[u] = load16_row(rx, (uint32_t)(u * threads + tid) * 16u);
            r.d[u] = load16_row(rd, (uint32_t)(u * threads + tid) * 16u);
        }
        if (a.dres) {
            const __amdgpu_buffer_rsrc_t rs = row_rsrc(a.dres + t * a.h, bytes);
#pragma unroll
            for (int u = 0; u < NV; ++u)
                r.s[u] = load16_row(rs, (uint32_t)(u * threads + tid) * 16u);
        }
    };
    int buf = 0;
    if (kAhead)
        load(next, blockIdx.x);
    for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x, buf ^= 1) {
        float ss = 0.0f, sg = 0.0f;
        if (kAhead)
            now = next;
        else
            load(now, t);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w[8], v[8], d[8];
            wv[u].get(w);
            widen8(now.x[u], v);
            widen8(now.d[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(v[i], v[i], ss);
                sg = __builtin_fmaf(d[i] * w[i], v[i], sg);
            }
        }
        if (kAhead && t + gridDim.x < (size_t)a.T)
            load(next, t + gridDim.x);
        ss = wave_sum(ss);
        sg = wave_sum(sg);
        if (waves > 1) {
            // two buffers: a wave that is a row ahead writes the other one
            if (lane_id() == 0)
                sums[buf][tid >> 6] = float2{ss, sg};
            __syncthreads();
            ss = sg = 0.0f;
            for (int w = 0; w < waves; ++w) {
                const float2 p = sums[buf][w];
                ss += p.x;
                sg += p.y;
            }
        }
        const float inv = 1.0f / __builtin_sqrtf(ss / (float)a.h + a.eps);
        const float c = inv * inv * (sg / (float)a.h);  // inv mean(g n)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            // widened again from the packed row: kept wide over the barrier it
            // would not fit the registers
            opaque(now.x[u]);
            opaque(now.d[u]);
            opaque(wv[u].lo);
            float w[8], v[8], d[8], o[8];
            wv[u].get(w);
            widen8(now.x[u], v);
            widen8(now.d[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = inv * __builtin_fmaf(-c, v[i], d[i] * w[i]);
                dw[u][i] = __builtin_fmaf(d[i], v[i] * inv, dw[u][i]);
            }
            if (a.dres) {
                float s[8];
                widen8(now.s[u], s);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] += s[i];
            }
            const int cc = u * threads + tid;
            if (cc < nvec)
                *reinterpret_cast<u32x4 *>(a.dx + t * a.h + (size_t)cc * 8) = narrow8(o);
        }
    }
    float *part = a.partial + (size_t)blockIdx.x * a.h;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = u * threads + tid;
        if (c < nvec) {
            float4 *p = reinterpret_cast<float4 *>(part + (size_t)c * 8);
            p[0] = float4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]};
            p[1] = float4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]};
        }
    }
}

// dw[c] = the sum of the partial rows, in a fixed order: 16 threads have four
// columns, each a sixteenth of the rows.
constexpr int kSumLanes = 16;

__global__ __launch_bounds__(256) void norm_weight_kernel(const float *partial, int rows, int h,
                                                          float *dw)
{
    __shared__ float4 meet[kSumLanes][256 / kSumLanes];
    const int col = threadIdx.x % (256 / kSumLanes), part = threadIdx.x / (256 / kSumLanes);
    const int c = (blockIdx.x * (256 / kSumLanes) + col) * 4;
    float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < h) {
#pragma unroll 8
        for (int r = part; r < rows; r += kSumLanes) {
            const float4 p = *reinterpret_cast<const float4 *>(partial + (size_t)r * h + c);
            s.x += p.x;
            s.y += p.y;
            s.z += p.z;
            s.w += p.w;
        }
    }
    meet[part][col] = s;
    __syncthreads();
    if (part == 0 && c < h) {
        for (int r = 1; r < kSumLanes; ++r) {
            const float4 p = meet[r][col];
            s.x += p.x;
            s.y += p.y;
            s.z += p.z;
            s.w += p.w;
        }
        *reinterpret_cast<float4 *>(dw + c) = s;
    }
}

// Vectors per thread and waves of a row's block: two vectors, four where
// sixteen waves of two do not hold the row (EPX_MAX_NORM_CHANNELS is 16 waves
// of four).
struct RowShape {
    int nv, waves;
};

RowShape row_shape(int h)
{
    const int nvec = h >> 3;
    const int nv = nvec > 2 * kWave * kMaxWaves ? 4 : 2;
    return {nv, (nvec + nv * kWave - 1) / (nv * kWave)};
}

template <int NV>
hipError_t launch_norm(const NormArgs &a, bool w_f32, int waves, hipStream_t stream)
{
    const dim3 grid((unsigned)a.T), block((unsigned)waves * kWave);
    if (a.codes) {
        if (w_f32)
            hipLaunchKernelGGL((norm_kernel<NV, true, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((norm_kernel<NV, true, false>), grid, block, 0, stream, a);
    } else if (w_f32) {
        hipLaunchKernelGGL((norm_kernel<NV, false, true>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((norm_kernel<NV, false, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

template <int NV>
hipError_t launch_norm_bwd(const NormBwdArgs &a, bool w_f32, int waves, int blocks,
                           hipStream_t stream)
{
    const dim3 grid((unsigned)blocks), block((unsigned)waves * kWave);
    if (w_f32)
        hipLaunchKernelGGL((norm_backward_kernel<NV, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_backward_kernel<NV, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, bool w_f32, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    const RowShape s = row_shape(a.h);
    return s.nv == 2 ? launch_norm<2>(a, w_f32, s.waves, stream)
                     : launch_norm<4>(a, w_f32, s.waves, stream);
}

int norm_bwd_blocks(int T, int h)
{
    (void)h;
    return T < 512 ? T : 512;
}

hipError_t launch_rms_norm_backward(const NormBwdArgs &a, bool w_f32, hipStream_t stream)
{
    const int blocks = norm_bwd_blocks(a.T, a.h);
    if (blocks > 0) {
        const RowShape s = row_shape(a.h);
        const hipError_t e = s.nv == 2 ? launch_norm_bwd<2>(a, w_f32, s.waves, blocks, stream)
                                       : launch_norm_bwd<4>(a, w_f32, s.waves, blocks, stream);
        if (e != hipSuccess)
            return e;
    }
    const int per = 256 / kSumLanes * 4;
    hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((a.h + per - 1) / per)), dim3(256), 0,
                       stream, a.partial, blocks, a.h, a.dw);
    return hipGetLastError();
}

}  // namespace epx
