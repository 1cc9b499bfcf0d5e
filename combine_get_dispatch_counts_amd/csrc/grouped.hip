// grouped.hip -- products of the experts' rows with their weights, with the
// gated activation as an epilogue.
//
//   out[r, n] = sum_k x[r, k] w[e, n, k]                     (bf16)
//   out[r, n] = sum_b xs[r, b] ws[e, n/128, b] sum_{k in b} x[r, k] w[e, n, k]
//                                                            (FP8, b: 128 channels)
// summed in fp32. Gated: g and u are such products with the gate and the up
// rows of w, and out = g / (1 + exp(-g)) * u, in bf16 or again in FP8 with
// a scale per 128 columns.
#include "experts_device.h"

namespace epx {
namespace {

constexpr int kBM = 64, kBN = 128, kWaves = 4, kThreads = kWaves * kWave;

template <bool FP8, bool GATED>
__global__ __launch_bounds__(kThreads) void grouped_kernel(GroupedArgs a)
{
    constexpr int G = GATED ? 2 : 1, MT = kBM / 16, NF = kBN / kWaves / 16;
    __shared__ int tiles_before[EPX_MAX_EXPERTS + 1];
    __shared__ int wave_tiles[kWaves];
    __shared__ float row_amax[kWaves][kBM];
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
    const int g4 = lane >> 4, l16 = lane & 15;

    // row tiles of every expert, as running totals
    int carry = 0;
    for (int e0 = 0; e0 < a.L; e0 += kThreads) {
        const int e = e0 + tid;
        int n = 0;
        if (e < a.L) {
            int64_t first;
            bool bad;
            n = (expert_rows(a, e, first, bad) + kBM - 1) / kBM;
            if (bad && blockIdx.x == 0)
                flag_error(a.err, EPX_DEV_OVERFLOW);
        }
        const int incl = wave_inclusive_sum(n);
        if (lane == 63)
            wave_tiles[wave] = incl;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < wave; ++w)
            before += wave_tiles[w];
        if (e < a.L)
            tiles_before[e + 1] = before + incl;
        for (int w = 0; w < kWaves; ++w)
            carry += wave_tiles[w];
        __syncthreads();
    }
    if (tid == 0)
        tiles_before[0] = 0;
    __syncthreads();

    const int nt = (a.N + kBN - 1) / kBN;
    const int64_t total = (int64_t)carry * nt;
    const int wrows = GATED ? 2 * a.N : a.N;
    const int kb_n = a.K >> 7, nb_n = (wrows + 127) >> 7;
    const size_t esize = FP8 ? 1 : 2;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
        const int mt = (int)(t / nt), n0 = (int)(t - (int64_t)mt * nt) * kBN;
        int e = 0;
        for (int step = 512; step; step >>= 1)
            if (e + step < a.L && tiles_before[e + step] <= mt)
                e += step;
        int64_t first;
        bool bad;
        const int rows = expert_rows(a, e, first, bad);
        const int m0 = (mt - tiles_before[e]) * kBM;

        const char *xp[MT];
        const float *xsp[MT];
        int64_t row[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = min(m0 + i * 16 + l16, rows - 1);
            row[i] = first + expert_row(a, e, m);
            xp[i] = static_cast<const char *>(a.x) + (size_t)row[i] * a.K * esize;
            xsp[i] = FP8 ? a.xs + (size_t)row[i] * scale_stride(a.K) : nullptr;
        }
        const char *wp[G][NF];
        const float *wsp[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
            const int nw0 = n0 + wave * (NF * 16);
            for (int j = 0; j < NF; ++j) {
                const int n = min(nw0 + j * 16 + l16, a.N - 1) + q * a.N;
                wp[q][j] = static_cast<const char *>(a.w) + ((size_t)e * wrows + n) * a.K * esize;
            }
            wsp[q] = FP8 ? a.ws + ((size_t)e * nb_n + ((n0 + q * a.N) >> 7)) * kb_n : nullptr;
        }
        f32x4 acc[G][NF][MT];
#pragma unroll
        for (int q = 0; q < G; ++q)
            for (int j = 0; j < NF; ++j)
                for (int i = 0; i < MT; ++i)
                    acc[q][j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (FP8) {
            for (int kb = 0; kb < kb_n; ++kb) {
                const int off = kb * 128 + g4 * 32;
                i32x8 xv[MT];
                float sx[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const i32x4 *p = reinterpret_cast<const i32x4 *>(xp[i] + off);
                    xv[i] = join(p[0], p[1]);
                    sx[i] = xsp[i][kb];
                }
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    const float sw = wsp[q][kb];
#pragma unroll
                    for (int j = 0; j < NF; ++j) {
                        const i32x4 *p = reinterpret_cast<const i32x4 *>(wp[q][j] + off);
                        const i32x8 wv = join(p[0], p[1]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const f32x4 d = mfma_fp8(wv, xv[i], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                            const float s = sx[i] * sw;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                acc[q][j][i][c] = __builtin_fmaf(s, d[c], acc[q][j][i][c]);
                        }
                    }
                }
            }
        } else {
            for (int k0 = 0; k0 < a.K; k0 += 32) {
                const int k = k0 + g4 * 8;
                const bool in = k < a.K;  // K is a multiple of 8
                const i32x4 zero{0, 0, 0, 0};
                i32x4 xv[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    xv[i] = in ? *reinterpret_cast<const i32x4 *>(xp[i] + 2 * (size_t)k) : zero;
#pragma unroll
                for (int q = 0; q < G; ++q)
#pragma unroll
                    for (int j = 0; j < NF; ++j) {
                        const i32x4 wv =
                            in ? *reinterpret_cast<const i32x4 *>(wp[q][j] + 2 * (size_t)k) : zero;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
                            acc[q][j][i] = mfma_bf16(wv, xv[i], acc[q][j][i]);
                    }
            }
        }

        // lane l holds columns n0 + 32 wave + 16 j + 4 (l / 16) .. + 3 of rows m0 + 16 i + l % 16
        if constexpr (GATED) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
                for (int i = 0; i < MT; ++i)
                    for (int c = 0; c < 4; ++c)
                        acc[0][j][i][c] = silu_mul(acc[0][j][i][c], acc[1][j][i][c]);
        }
        if constexpr (GATED && FP8) {
            const int st = scale_stride(a.N);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float m = 0.0f;
                for (int j = 0; j < NF; ++j)
                    for (int c = 0; c < 4; ++c)
                        m = amax_of(m, acc[0][j][i][c]);
                m = amax_of(m, __shfl_xor(m, 16, kWave));
                m = amax_of(m, __shfl_xor(m, 32, kWave));
                if (g4 == 0)
                    row_amax[wave][i * 16 + l16] = m;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = i * 16 + l16;
                float am = row_amax[0][m];
                for (int w = 1; w < kWaves; ++w)
                    am = amax_of(am, row_amax[w][m]);
                const float s = group_scale(am);
                if (m0 + m >= rows)
                    continue;
                uint8_t *o = static_cast<uint8_t *>(a.out) + (size_t)row[i] * a.N;
                for (int j = 0; j < NF; ++j) {
                    uint32_t q = 0;
                    for (int c = 0; c < 4; ++c)
                        q |= e4m3_of_quotient(acc[0][j][i][c], s) << (8 * c);
                    *reinterpret_cast<uint32_t *>(o + n0 + wave * 32 + j * 16 + g4 * 4) = q;
                }
                float *os = a.out_s + (size_t)row[i] * st;
                if (wave == 0 && g4 == 0)
                    os[n0 >> 7] = s;
                if (n0 + kBN >= a.N)  // the last column tile also clears the padding
                    for (int p = (a.N >> 7) + wave * 4 + g4; p < st; p += 16)
                        os[p] = 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (m0 + i * 16 + l16 >= rows)
                    continue;
                uint16_t *o = static_cast<uint16_t *>(a.out) + (size_t)row[i] * a.N;
                for (int j = 0; j < NF; ++j) {
                    const int n = n0 + wave * (NF * 16) + j * 16 + g4 * 4;
                    if (n < a.N) {  // N is a multiple of 8
                        uint2 v;
                        v.x = f32_to_bf16(acc[0][j][i][0]) | (f32_to_bf16(acc[0][j][i][1]) << 16);
                        v.y = f32_to_bf16(acc[0][j][i][2]) | (f32_to_bf16(acc[0][j][i][3]) << 16);
                        *reinterpret_cast<uint2 *>(o + n) = v;
                    }
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, bool fp8, bool gated, hipStream_t stream)
{
    const int64_t nt = (a.N + kBN - 1) / kBN;
    const int64_t most = ((a.n_rows + kBM - 1) / kBM + a.L) * nt;  // tiles there can be
    const int64_t blocks = most < 4ll * a.cus ? most : 4ll * a.cus;
    if (a.n_rows == 0)
        return hipSuccess;
    const auto k = fp8 ? (gated ? grouped_kernel<true, true> : grouped_kernel<true, false>)
                       : (gated ? grouped_kernel<false, true> : grouped_kernel<false, false>);
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace epx
