// moe_decode.hip -- the whole expert layer for a few tokens in two launches:
//
//   a[t, k] = bf16( silu(Wg x_t) * (Wu x_t) )       Wg, Wu: the halves of w13[idx[t, k]]
//   out[t]  = bf16( sum_k topw[t, k] * (W2 a[t, k]) )
//
// With few tokens each expert's weights serve a handful of rows, so both
// launches are streams over the weights of the experts that were routed to:
// HBM-bound, every weight byte read once, and the matrix instructions only
// keep the arithmetic out of the way. FP8 weights are widened to bf16 in
// registers (exact) and their block scales applied to the fp32 sums of 128
// channels; the tokens stay in bf16.
//
// A wave owns 16 weight rows (the A operand of D = W X^T) and a share of the
// channels; its expert's tokens are the B operand, 16 at a time, up to all
// 64 held as accumulators at once, so a weight is loaded once whatever the
// number of tokens.
#include "experts_device.h"

namespace epx {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kMaxEntries = kDecodeMaxTokens * EPX_MAX_TOPK;

// Entries of the routing table grouped by expert, in LDS.
struct Groups {
    int start[EPX_MAX_EXPERTS + 1];   // first entry of each expert's list
    short active[EPX_MAX_EXPERTS];    // experts with entries, ascending
    short entry[kMaxEntries];         // t * K + k, expert by expert
    int n_active;
    int part[kWaves];
};

// Fills g. An entry whose token already has an earlier entry with the same
// expert is left out: its weight is added to the earlier one's where the
// weights are used. The order inside an expert's list is not fixed; nothing
// depends on it (each list position is a column of its own).
__device__ void group_entries(const DecodeArgs &a, Groups &g)
{
    const int tid = threadIdx.x, n = a.T * a.K;
    for (int e = tid; e <= EPX_MAX_EXPERTS; e += kThreads)
        g.start[e] = 0;
    __syncthreads();
    int mine[kMaxEntries / kThreads];  // expert << 16 | place in its list, or -1
#pragma unroll
    for (int i = 0; i < kMaxEntries / kThreads; ++i) {
        const int j = i * kThreads + tid;
        mine[i] = -1;
        if (j < n) {
            const int64_t e = a.idx[j];
            if (e >= 0 && e < a.E) {
                bool repeat = false;
                for (int p = j - j % a.K; p < j; ++p)
                    repeat |= a.idx[p] == e;
                if (!repeat)
                    mine[i] = (int)e << 16 | atomicAdd(&g.start[e + 1], 1);
            } else if (e != -1 && blockIdx.x == 0) {
                flag_error(a.err, EPX_DEV_BAD_ROUTE);
            }
        }
    }
    __syncthreads();
    // running totals of the counts, and the experts that have entries
    const int wave = tid >> 6, lane = lane_id();
    constexpr int kPer = EPX_MAX_EXPERTS / kThreads;
    int c[kPer], sum = 0, live = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        c[i] = g.start[tid * kPer + i + 1];
        sum += c[i];
        live += c[i] > 0;
    }
    const int packed = sum << 12 | live;  // sum <= 2048, live <= 512
    const int incl = wave_inclusive_sum(packed);
    if (lane == 63)
        g.part[wave] = incl;
    __syncthreads();
    int before = incl - packed;
    for (int w = 0; w < wave; ++w)
        before += g.part[w];
    int s = before >> 12, l = before & 0xFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        s += c[i];
        g.start[tid * kPer + i + 1] = s;
        if (c[i] > 0)
            g.active[l++] = (short)(tid * kPer + i);
    }
    if (tid == kThreads - 1)
        g.n_active = l;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxEntries / kThreads; ++i)
        if (mine[i] >= 0)
            g.entry[g.start[mine[i] >> 16] + (mine[i] & 0xFFFF)] = (short)(i * kThreads + tid);
    __syncthreads();
}

// A lane's 16 weights of a 64-channel step as two bf16 operands: channels
// 16 (lane / 16) + 0..7 and + 8..15.
__device__ __forceinline__ i32x4 widen(int lo, int hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return i32x4{__builtin_bit_cast(int, a), __builtin_bit_cast(int, b),
                 __builtin_bit_cast(int, c), __builtin_bit_cast(int, d)};
}

// acc[q][i] += W_q[16 rows] X^T over channels [k0, k1) for MT groups of 16
// tokens. wp[q]: the lane's weight row; xp[i]: the lane's token row (null:
// none, zeros); ws[q]: the weight rows' block scales over channels.
template <bool FP8, int G, int MT>
__device__ __forceinline__ void stream_products(const char *const (&wp)[G],
                                                const float *const (&ws)[G],
                                                const uint16_t *const (&xp)[MT], int k0, int k1,
                                                f32x4 (&acc)[G][MT])
{
    const int g4 = lane_id() >> 4;
    const i32x4 zero{0, 0, 0, 0};
    if constexpr (FP8) {
        for (int k = k0; k < k1; k += 128) {
            i32x4 wv[G][2];
#pragma unroll
            for (int q = 0; q < G; ++q)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    wv[q][u] = *reinterpret_cast<const i32x4 *>(wp[q] + k + u * 64 + g4 * 16);
            f32x4 p[G][MT];
#pragma unroll
            for (int q = 0; q < G; ++q)
                for (int i = 0; i < MT; ++i)
                    p[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                i32x4 xv[MT][2];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        xv[i][b] = xp[i] ? *reinterpret_cast<const i32x4 *>(xp[i] + k + u * 64 +
                                                                            g4 * 16 + b * 8)
                                         : zero;
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    const i32x4 w0 = widen(wv[q][u].x, wv[q][u].y);
                    const i32x4 w1 = widen(wv[q][u].z, wv[q][u].w);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        p[q][i] = mfma_bf16(w0, xv[i][0], p[q][i]);
                        p[q][i] = mfma_bf16(w1, xv[i][1], p[q][i]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < G; ++q) {
                const float s = ws[q][k >> 7];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[q][i][c] = __builtin_fmaf(s, p[q][i][c], acc[q][i][c]);
            }
        }
    } else {
        for (int k = k0; k < k1; k += 32) {
            const int kk = k + g4 * 8;
            const bool in = kk < k1;
            i32x4 wv[G];
#pragma unroll
            for (int q = 0; q < G; ++q)
                wv[q] = in ? *reinterpret_cast<const i32x4 *>(wp[q] + 2 * (size_t)kk) : zero;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const i32x4 xv =
                    in && xp[i] ? *reinterpret_cast<const i32x4 *>(xp[i] + kk) : zero;
#pragma unroll
                for (int q = 0; q < G; ++q)
                    acc[q][i] = mfma_bf16(wv[q], xv, acc[q][i]);
            }
        }
    }
}

// First launch: 16 columns of f, gate and up, for every token of one expert.
// The block's waves split the channels of h.
template <bool FP8, int MT>
__device__ void up_tile(const DecodeArgs &a, const Groups &g, int e, int n0,
                        float (&part)[kWaves][2][64][17])
{
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, l16 = lane & 15;
    const int first = g.start[e], rows = g.start[e + 1] - first;
    const size_t esize = FP8 ? 1 : 2;
    const int step = FP8 ? 128 : 32;
    const int units = (a.h + step - 1) / step;
    const int k0 = units * wave / kWaves * step, k1 = min(units * (wave + 1) / kWaves * step, a.h);
    const int n = min(n0 + l16, a.f - 1);
    const char *wp[2];
    const float *ws[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        wp[q] = static_cast<const char *>(a.w13) +
                ((size_t)e * 2 * a.f + (size_t)q * a.f + n) * a.h * esize;
        ws[q] = FP8 ? a.s13 + ((size_t)e * (2 * a.f >> 7) + ((q * a.f + n0) >> 7)) * (a.h >> 7)
                    : nullptr;
    }
    const uint16_t *xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = i * 16 + l16;
        xp[i] = m < rows ? a.x + (size_t)(g.entry[first + m] / a.K) * a.h : nullptr;
    }
    f32x4 acc[2][MT];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        for (int i = 0; i < MT; ++i)
            acc[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream_products<FP8, 2, MT>(wp, ws, xp, k0, k1, acc);
#pragma unroll
    for (int q = 0; q < 2; ++q)
        for (int i = 0; i < MT; ++i)
            for (int c = 0; c < 4; ++c)
                part[wave][q][i * 16 + l16][(lane >> 4) * 4 + c] = acc[q][i][c];
    __syncthreads();
    for (int v = tid; v < rows * 16; v += kThreads) {
        const int m = v >> 4, c = v & 15;
        float gate = 0.0f, up = 0.0f;
        for (int w = 0; w < kWaves; ++w) {
            gate += part[w][0][m][c];
            up += part[w][1][m][c];
        }
        if (n0 + c < a.f)
            a.act[(size_t)g.entry[first + m] * a.f + n0 + c] =
                (uint16_t)f32_to_bf16(silu_mul(gate, up));
    }
    __syncthreads();
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void decode_up_kernel(DecodeArgs a)
{
    __shared__ Groups g;
    __shared__ float part[kWaves][2][64][17];
    group_entries(a, g);
    const int nt = (a.f + 15) / 16;
    const int total = g.n_active * nt;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = g.active[t / nt], n0 = t % nt * 16;
        const int rows = g.start[e + 1] - g.start[e];
        if (rows <= 16)
            up_tile<FP8, 1>(a, g, e, n0, part);
        else
            up_tile<FP8, 4>(a, g, e, n0, part);
    }
}

// Second launch: 16 columns of h for all tokens. The block's waves take the
// active experts in turn, each with sums of its own, which are added in wave
// order at the end: the result does not depend on timing.
template <bool FP8, int MT>
__device__ void down_tile(const DecodeArgs &a, const Groups &g, int e, int n0,
                          float (&sum)[kDecodeMaxTokens][16])
{
    const int lane = lane_id(), l16 = lane & 15, g4 = lane >> 4;
    const int first = g.start[e], rows = g.start[e + 1] - first;
    const int n = min(n0 + l16, a.h - 1);
    const char *wp[1] = {static_cast<const char *>(a.w2) +
                         ((size_t)e * a.h + n) * a.f * (FP8 ? 1 : 2)};
    const float *ws[1] = {
        FP8 ? a.s2 + ((size_t)e * ((a.h + 127) >> 7) + (n0 >> 7)) * (a.f >> 7) : nullptr};
    const uint16_t *xp[MT];
    int token[MT];
    float weight[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = i * 16 + l16;
        xp[i] = nullptr;
        token[i] = -1;
        weight[i] = 0.0f;
        if (m < rows) {
            const int j = g.entry[first + m];
            token[i] = j / a.K;
            xp[i] = a.act + (size_t)j * a.f;
            for (int k = j; k < (token[i] + 1) * a.K; ++k)  // repeats of the expert included
                if (a.idx[k] == e)
                    weight[i] += a.topw[k];
        }
    }
    f32x4 acc[1][MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        acc[0][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream_products<FP8, 1, MT>(wp, ws, xp, 0, a.f, acc);
#pragma unroll
    for (int i = 0; i < MT; ++i)
        if (token[i] >= 0)
            for (int c = 0; c < 4; ++c) {
                float &s = sum[token[i]][g4 * 4 + c];
                s = __builtin_fmaf(weight[i], acc[0][i][c], s);
            }
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void decode_down_kernel(DecodeArgs a)
{
    __shared__ Groups g;
    __shared__ float sum[kWaves][kDecodeMaxTokens][16];
    const int tid = threadIdx.x, wave = tid >> 6;
    group_entries(a, g);
    for (int v = tid; v < kWaves * kDecodeMaxTokens * 16; v += kThreads)
        (&sum[0][0][0])[v] = 0.0f;
    __syncthreads();
    const int n0 = blockIdx.x * 16;
    for (int i = wave; i < g.n_active; i += kWaves) {
        const int e = g.active[i];
        if (g.start[e + 1] - g.start[e] <= 16)
            down_tile<FP8, 1>(a, g, e, n0, sum[wave]);
        else
            down_tile<FP8, 4>(a, g, e, n0, sum[wave]);
    }
    __syncthreads();
    for (int v = tid; v < a.T * 16; v += kThreads) {
        const int t = v >> 4, c = v & 15;
        float s = 0.0f;
        for (int w = 0; w < kWaves; ++w)
            s += sum[w][t][c];
        if (n0 + c < a.h)
            a.out[(size_t)t * a.h + n0 + c] = (uint16_t)f32_to_bf16(s);
    }
}

}  // namespace

hipError_t launch_moe_decode(const DecodeArgs &a, bool fp8, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    const int64_t items = (int64_t)(a.E < a.T * a.K ? a.E : a.T * a.K) * ((a.f + 15) / 16);
    const unsigned up = (unsigned)(items < 4ll * a.cus ? items : 4ll * a.cus);
    const unsigned down = (unsigned)((a.h + 15) / 16);
    if (fp8) {
        hipLaunchKernelGGL(decode_up_kernel<true>, dim3(up), dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL(decode_down_kernel<true>, dim3(down), dim3(kThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL(decode_up_kernel<false>, dim3(up), dim3(kThreads), 0, stream, a);
        hipLaunchKernelGGL(decode_down_kernel<false>, dim3(down), dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace epx
