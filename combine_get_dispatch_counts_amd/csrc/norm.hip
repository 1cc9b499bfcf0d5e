// norm.hip -- root-mean-square norm of a residual stream's rows, with the
// residual's addition and the dispatch's FP8 rows, and its gradient.
//
// Forward, per row: v = x + residual (fp32), inv = 1 / sqrt(mean(v^2) + eps),
// y = v inv w. A block has one row, held in registers from its loads to its
// stores, so the row is read once whatever is written of it: the sum in bf16
// (the stream's next value), y in bf16, and y as e4m3 codes with a scale per
// 128 channels. Both forms of y are rounded once, from fp32. Bound by memory:
// 4096 rows of 7168 with everything written (265 MB) 43 us, 6.2 TB/s; a single
// row 3.1 us, of which most is a launch and two waits, for the row and for the
// block's sums.
//
// Backward, per row, with n = v inv and g = dout w:
//   dx = dres + inv (g - n mean(g n)),   dw = sum over rows of dout n.
// mean(g n) = inv mean(g v), so both row sums (v^2 and g v) come from one
// pass. Groups of waves have a row each and walk the rows with their share of
// dw in registers; a block's groups add theirs in LDS and leave one row of
// partial sums, which a second launch adds in block order. Bound by memory too:
// 4096 rows of 7168 (235 MB) 47 us, 5.0 TB/s, of which the second launch 4.8;
// 1003 x 1416 8.3, two launches' latency. Above 16384 channels a thread has four
// vectors and spills some of them (2.8 TB/s).
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

template <int NV, bool FP8, bool WF32, bool STREAM>
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
                store16_stream(a.res_out + row * a.h + (size_t)c * 8, narrow8(v[u]));
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
        if (a.out && c < nvec) {
            uint16_t *to = a.out + row * a.h + (size_t)c * 8;
            if constexpr (STREAM)
                store16_stream(to, narrow8(y));
            else
                *reinterpret_cast<u32x4 *>(to) = narrow8(y);
        }
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

// Rows of at most 8 LANES channels: LANES lanes have a row, a vector each, so a
// wave has two or four and no block meets. (A wave a row: 32768 x 64 12.6 us,
// x 256 23.9; this 4.1 and 15.3.)
constexpr int kNarrowThreads = 256;

template <int LANES, bool FP8, bool WF32>
__global__ __launch_bounds__(kNarrowThreads) void norm_narrow_kernel(NormArgs a)
{
    const int i = threadIdx.x % LANES, nvec = a.h >> 3;
    const int64_t row = (int64_t)blockIdx.x * (kNarrowThreads / LANES) + threadIdx.x / LANES;
    const bool live = row < a.T && i < nvec;
    const size_t at = (size_t)(live ? row * a.h + i * 8 : 0);
    const u32x4 zero = {0u, 0u, 0u, 0u};
    Weight8<WF32> wv;
    wv.load(row_rsrc(a.w, (uint32_t)nvec * (WF32 ? 32u : 16u)), (uint32_t)i);
    float v[8], ss = 0.0f;
    widen8(live ? load16_stream(a.x + at) : zero, v);
    if (a.residual) {
        float r[8];
        widen8(live ? load16_stream(a.residual + at) : zero, r);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] += r[c];
        if (live)
            store16_stream(a.res_out + at, narrow8(v));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        ss = __builtin_fmaf(v[c], v[c], ss);
    ss = group_sum<LANES>(ss);
    const float inv = 1.0f / __builtin_sqrtf(ss / (float)a.h + a.eps);
    float w[8], y[8];
    wv.get(w);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        y[c] = v[c] * inv * w[c];
    if (a.out && live)
        *reinterpret_cast<u32x4 *>(a.out + at) = narrow8(y);
    if constexpr (FP8) {
        uint32_t q0, q1;
        const float s = codes8(y, q0, q1);
        if (live)
            *reinterpret_cast<uint2 *>(a.codes + at) = uint2{q0, q1};
        // 32 scales a row (128 or 256 channels have one or two groups)
        const float next = LANES == 32 ? __shfl(s, (lane_id() & 32) + 16, kWave) : 0.0f;
        if (row < a.T) {
            for (int g = i; g < 32; g += LANES)
                a.scales[row * 32 + g] = g == 0 ? s : g == 1 && a.h > 128 ? next : 0.0f;
        }
    }
}

template <int NV, bool WF32>
__global__ __launch_bounds__(kWave *kMaxWaves) void norm_backward_kernel(NormBwdArgs a, int waves)
{
    // the next row's loads go out before this row's sums meet, where the
    // registers hold both rows
    constexpr bool kAhead = NV <= 2;
    __shared__ float2 sums[2][kMaxWaves];
    extern __shared__ __align__(16) float meet[];  // [groups - 1, h]
    const int threads = waves * kWave, groups = blockDim.x / threads;
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / threads);  // (whole waves)
    const int tid = threadIdx.x - group * threads;
    const int nvec = a.h >> 3;
    const uint32_t bytes = (uint32_t)nvec * 16u;
    const __amdgpu_buffer_rsrc_t rw = row_rsrc(a.w, (uint32_t)nvec * (WF32 ? 32u : 16u));
    // held, where the registers allow; else read again where they are used
    constexpr bool kHold = NV <= 2;
    Weight8<WF32> wv[kHold ? NV : 1];
    const auto weight = [&](int u, float (&w)[8]) {
        if (kHold) {
            wv[kHold ? u : 0].get(w);
        } else {
            Weight8<WF32> v;
            v.load(rw, (uint32_t)(u * threads + tid));
            v.get(w);
        }
    };
    float dw[NV][8];
    struct Row {
        u32x4 x[NV], d[NV], s[NV];
    } now, next;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (kHold)
            wv[kHold ? u : 0].load(rw, (uint32_t)(u * threads + tid));
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
    const size_t step = (size_t)gridDim.x * groups, last = (size_t)a.T - 1;
    size_t t = (size_t)blockIdx.x * groups + group;
    int buf = 0;
    if (kAhead)
        load(next, min(t, last));
    // a block's groups make the same number of steps; behind the last row they
    // read that again and keep nothing
    for (size_t t0 = (size_t)blockIdx.x * groups; t0 < (size_t)a.T; t0 += step, t += step, buf ^= 1) {
        float ss = 0.0f, sg = 0.0f;
        const bool live = t <= last;
        if (kAhead)
            now = next;
        else
            load(now, min(t, last));
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float w[8], v[8], d[8];
            weight(u, w);
            widen8(now.x[u], v);
            widen8(now.d[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(v[i], v[i], ss);
                sg = __builtin_fmaf(d[i] * w[i], v[i], sg);
            }
            if (!kAhead)
                __builtin_amdgcn_sched_barrier(0);  // one vector's values at a time
        }
        if (kAhead && t0 + step < (size_t)a.T)
            load(next, min(t + step, last));
        ss = wave_sum(ss);
        sg = wave_sum(sg);
        if (waves > 1) {
            // two buffers: a wave that is a row ahead writes the other one
            if (lane_id() == 0)
                sums[buf][threadIdx.x >> 6] = float2{ss, sg};
            __syncthreads();
            ss = sg = 0.0f;
            for (int w = 0; w < waves; ++w) {
                const float2 p = sums[buf][group * waves + w];
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
            if (kHold)
                opaque(wv[kHold ? u : 0].lo);
            float w[8], v[8], d[8], o[8];
            weight(u, w);
            widen8(now.x[u], v);
            widen8(now.d[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = inv * __builtin_fmaf(-c, v[i], d[i] * w[i]);
                const float s = __builtin_fmaf(d[i], v[i] * inv, dw[u][i]);
                dw[u][i] = live ? s : dw[u][i];
            }
            if (a.dres) {
                float s[8];
                widen8(now.s[u], s);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] += s[i];
            }
            const int cc = u * threads + tid;
            if (live && cc < nvec)
                *reinterpret_cast<u32x4 *>(a.dx + t * a.h + (size_t)cc * 8) = narrow8(o);
            if (!kAhead)
                __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (groups > 1) {
        if (group > 0) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = u * threads + tid;
                if (c < nvec) {
                    float4 *p = reinterpret_cast<float4 *>(meet + (size_t)(group - 1) * a.h + c * 8);
                    p[0] = float4{dw[u][0], dw[u][1], dw[u][2], dw[u][3]};
                    p[1] = float4{dw[u][4], dw[u][5], dw[u][6], dw[u][7]};
                }
            }
        }
        __syncthreads();
        if (group > 0)
            return;
        for (int g = 0; g < groups - 1; ++g) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = u * threads + tid;
                if (c < nvec) {
                    const float *p = meet + (size_t)g * a.h + c * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dw[u][i] += p[i];
                }
            }
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

// Rows of at most 8 LANES channels, as the forward pass has them; a wave's
// groups of lanes walk the rows four steps at a time and meet once at the end.
constexpr int kNarrowSteps = 4;

template <int LANES, bool WF32>
__global__ __launch_bounds__(kNarrowThreads) void norm_narrow_backward_kernel(NormBwdArgs a)
{
    constexpr int kRows = kNarrowThreads / LANES;
    __shared__ float meet[kRows][LANES * 8];
    const int i = threadIdx.x % LANES, mine = threadIdx.x / LANES, nvec = a.h >> 3;
    const int64_t step = (int64_t)gridDim.x * kRows;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    Weight8<WF32> wv;
    wv.load(row_rsrc(a.w, (uint32_t)nvec * (WF32 ? 32u : 16u)), (uint32_t)i);
    float w[8], dw[8];
    wv.get(w);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        dw[c] = 0.0f;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows + mine; t0 - mine < a.T;
         t0 += kNarrowSteps * step) {
        u32x4 x[kNarrowSteps], d[kNarrowSteps], s[kNarrowSteps];
        bool live[kNarrowSteps];
        size_t at[kNarrowSteps];
#pragma unroll
        for (int q = 0; q < kNarrowSteps; ++q) {
            const int64_t t = t0 + q * step;
            live[q] = t < a.T && i < nvec;
            // (what a lane without a row or channels reads it does not use; in
            // place it may be another row's gradient already)
            at[q] = (size_t)(live[q] ? t * a.h + i * 8 : 0);
            x[q] = load16_stream(a.x + at[q]);
            d[q] = load16_stream(a.dout + at[q]);
            s[q] = a.dres ? load16_stream(a.dres + at[q]) : zero;
        }
#pragma unroll
        for (int q = 0; q < kNarrowSteps; ++q) {
            float v[8], g[8], r[8], ss = 0.0f, sg = 0.0f;
            widen8(live[q] ? x[q] : zero, v);
            widen8(live[q] ? d[q] : zero, g);
            widen8(s[q], r);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                ss = __builtin_fmaf(v[c], v[c], ss);
                sg = __builtin_fmaf(g[c] * w[c], v[c], sg);
            }
            ss = group_sum<LANES>(ss);
            sg = group_sum<LANES>(sg);
            const float inv = 1.0f / __builtin_sqrtf(ss / (float)a.h + a.eps);
            const float m = inv * inv * (sg / (float)a.h);
            float o[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                o[c] = inv * __builtin_fmaf(-m, v[c], g[c] * w[c]) + r[c];
                const float n = __builtin_fmaf(g[c], v[c] * inv, dw[c]);
                dw[c] = live[q] ? n : dw[c];  // (a row of zeros without eps is NaN)
            }
            if (live[q])
                *reinterpret_cast<u32x4 *>(a.dx + at[q]) = narrow8(o);
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        meet[mine][i * 8 + c] = dw[c];
    __syncthreads();
    for (int c = threadIdx.x; c < a.h; c += kNarrowThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            sum += meet[r][c];
        a.partial[(size_t)blockIdx.x * a.h + c] = sum;
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
        // eight rows' loads at a time, also of the last few (rows behind the
        // last are read as that and not added)
        for (int r0 = part; r0 < rows; r0 += 8 * kSumLanes) {
            float4 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = *reinterpret_cast<const float4 *>(
                    partial + (size_t)min(r0 + i * kSumLanes, rows - 1) * h + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = r0 + i * kSumLanes < rows;
                s.x += in ? p[i].x : 0.0f;
                s.y += in ? p[i].y : 0.0f;
                s.z += in ? p[i].z : 0.0f;
                s.w += in ? p[i].w : 0.0f;
            }
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

// The normed rows are read next, the sum with the residual only behind the
// whole layer: it is stored past the caches, and so are normed rows that would
// not stay in the memory-side cache until they are read. Measured at h = 7168
// with both and FP8 rows, alone / with a copy of the normed rows behind it, all
// cached, the sum streamed, both streamed: 1024 rows 14.9 / 20.7, 14.7 / 20.2,
// 14.7 / 22.4 us; 4096 rows 50.2 / 66.3, 44.3 / 62.2, 46.4 / 68.7; 8192 rows
// 94 / 145, 93 / 142, 85 / 132.
constexpr int64_t kStreamBytes = 96ll << 20;

template <int NV, bool FP8, bool WF32>
void launch_norm(const NormArgs &a, int waves, hipStream_t stream)
{
    const dim3 grid((unsigned)a.T), block((unsigned)waves * kWave);
    if ((int64_t)a.T * a.h * 2 > kStreamBytes)
        hipLaunchKernelGGL((norm_kernel<NV, FP8, WF32, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_kernel<NV, FP8, WF32, false>), grid, block, 0, stream, a);
}

// Widest rows that go to the narrow kernels' 16 and 32 lanes.
constexpr int kNarrow16 = 128, kNarrow32 = 256;

template <int LANES>
hipError_t launch_norm_narrow(const NormArgs &a, bool w_f32, hipStream_t stream)
{
    constexpr int kRows = kNarrowThreads / LANES;
    const dim3 grid((unsigned)(((int64_t)a.T + kRows - 1) / kRows)), block(kNarrowThreads);
    if (a.codes && w_f32)
        hipLaunchKernelGGL((norm_narrow_kernel<LANES, true, true>), grid, block, 0, stream, a);
    else if (a.codes)
        hipLaunchKernelGGL((norm_narrow_kernel<LANES, true, false>), grid, block, 0, stream, a);
    else if (w_f32)
        hipLaunchKernelGGL((norm_narrow_kernel<LANES, false, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_narrow_kernel<LANES, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <int NV>
hipError_t launch_norm(const NormArgs &a, bool w_f32, int waves, hipStream_t stream)
{
    if (a.codes && w_f32)
        launch_norm<NV, true, true>(a, waves, stream);
    else if (a.codes)
        launch_norm<NV, true, false>(a, waves, stream);
    else if (w_f32)
        launch_norm<NV, false, true>(a, waves, stream);
    else
        launch_norm<NV, false, false>(a, waves, stream);
    return hipGetLastError();
}

// Blocks and groups of waves of the backward pass. The registers hold 16 waves
// on a compute unit: two blocks, so that one loads while the other waits for
// its sums, of up to 8 waves (one block of 14 waves with two rows side by side
// took 46.5 us for 4096 x 7168 against 42.4, both without the second launch). Few narrow rows go side by side
// in as many blocks as there are compute units, which leaves fewer partial
// rows to write and add.
struct BwdShape {
    RowShape row;
    int groups, blocks;
};

constexpr int kBwdUnits = 256;

BwdShape bwd_shape(int T, int h)
{
    BwdShape s;
    s.row = row_shape(h);
    const int most = s.row.waves < 8 ? 8 / s.row.waves : 1;
    const int want = (int)(((int64_t)T + kBwdUnits - 1) / kBwdUnits);
    s.groups = want < 1 ? 1 : want < most ? want : most;
    const int64_t blocks = ((int64_t)T + s.groups - 1) / s.groups;
    const int places = kBwdUnits * (s.row.waves <= 8 ? 2 : 1);
    s.blocks = blocks < places ? (int)blocks : places;
    return s;
}

template <int NV>
hipError_t launch_norm_bwd(const NormBwdArgs &a, bool w_f32, const BwdShape &s, hipStream_t stream)
{
    const dim3 grid((unsigned)s.blocks), block((unsigned)(s.row.waves * s.groups) * kWave);
    const size_t lds = (size_t)(s.groups - 1) * a.h * sizeof(float);
    if (w_f32)
        hipLaunchKernelGGL((norm_backward_kernel<NV, true>), grid, block, lds, stream, a,
                           s.row.waves);
    else
        hipLaunchKernelGGL((norm_backward_kernel<NV, false>), grid, block, lds, stream, a,
                           s.row.waves);
    return hipGetLastError();
}

template <int LANES>
hipError_t launch_norm_narrow_bwd(const NormBwdArgs &a, bool w_f32, int blocks,
                                  hipStream_t stream)
{
    const dim3 grid((unsigned)blocks), block(kNarrowThreads);
    if (w_f32)
        hipLaunchKernelGGL((norm_narrow_backward_kernel<LANES, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((norm_narrow_backward_kernel<LANES, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &args, bool w_f32, hipStream_t stream)
{
    // a launch has at most 2^31 threads: more rows go in several
    const RowShape s = row_shape(args.h);
    const int per_row = args.h <= kNarrow16 ? 16 : args.h <= kNarrow32 ? 32 : s.waves * kWave;
    const int64_t most = (1ll << 31) / per_row;
    NormArgs a = args;
    for (int64_t row = 0; row < args.T; row += most) {
        a.T = (int)(args.T - row < most ? args.T - row : most);
        hipError_t e;
        if (a.h <= kNarrow32)
            e = a.h <= kNarrow16 ? launch_norm_narrow<16>(a, w_f32, stream)
                                 : launch_norm_narrow<32>(a, w_f32, stream);
        else
            e = s.nv == 2 ? launch_norm<2>(a, w_f32, s.waves, stream)
                          : launch_norm<4>(a, w_f32, s.waves, stream);
        if (e != hipSuccess)
            return e;
        const int64_t step = most * a.h;
        a.x += step;
        if (a.residual) {
            a.residual += step;
            a.res_out += step;
        }
        if (a.out)
            a.out += step;
        if (a.codes) {
            a.codes += step;
            a.scales += most * scale_stride(a.h);
        }
    }
    return hipSuccess;
}

int norm_bwd_blocks(int T, int h)
{
    if (h > kNarrow32)
        return bwd_shape(T, h).blocks;
    const int rows = kNarrowThreads / (h <= kNarrow16 ? 16 : 32);
    const int64_t blocks = ((int64_t)T + rows - 1) / rows;
    return blocks < 2 * kBwdUnits ? (int)blocks : 2 * kBwdUnits;
}

hipError_t launch_rms_norm_backward(const NormBwdArgs &a, bool w_f32, hipStream_t stream)
{
    const int blocks = norm_bwd_blocks(a.T, a.h);
    if (blocks > 0) {
        hipError_t e;
        if (a.h <= kNarrow32) {
            e = a.h <= kNarrow16 ? launch_norm_narrow_bwd<16>(a, w_f32, blocks, stream)
                                 : launch_norm_narrow_bwd<32>(a, w_f32, blocks, stream);
        } else {
            const BwdShape s = bwd_shape(a.T, a.h);
            e = s.row.nv == 2 ? launch_norm_bwd<2>(a, w_f32, s, stream)
                              : launch_norm_bwd<4>(a, w_f32, s, stream);
        }
        if (e != hipSuccess)
            return e;
    }
    const int per = 256 / kSumLanes * 4;
    hipLaunchKernelGGL(norm_weight_kernel, dim3((unsigned)((a.h + per - 1) / per)), dim3(256), 0,
                       stream, a.partial, blocks, a.h, a.dw);
    return hipGetLastError();
}

}  // namespace epx
