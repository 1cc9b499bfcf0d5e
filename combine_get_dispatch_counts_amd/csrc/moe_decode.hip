// moe_decode.hip -- the whole expert layer for a few tokens in two launches:
//
//   a[t, k] = bf16( silu(Wg x_t) * (Wu x_t) )       Wg, Wu: the halves of w13[idx[t, k]]
//   out[t]  = bf16( sum_k topw[t, k] * (W2 a[t, k]) )
//
// With few tokens each expert's weights serve a handful of rows, so both
// launches are streams over the weights of the experts that were routed to: a
// weight is read once for every 32 tokens of its expert, and the matrix
// instructions only keep the arithmetic out of the way. FP8 weights are widened
// to bf16 in registers (exact) and their block scales applied to the fp32 sums
// of 128 channels; the tokens stay in bf16, and so do the activations between
// the launches: what grouped_swiglu writes for bf16 rows, and the operand of
// the second product either way (the result is off by 0.0023 of its norm in
// place of 0.0017 with fp32 activations).
//
// Measured per call, back to back: FP8, h 7168, f 2048, top-8: 1 token 80 us,
// 48 tokens over 128 experts 1130 us, 4.8 TB/s; bf16, h 4096, f 1536, 8 tokens
// of top-6 over 64 experts 229 to 250 us. First and second launch in a kernel
// trace, which lengthens them by some percent: 49 + 35, 731 + 445 (4.9 and 4.0
// TB/s), 162 + 89. The second launch's grid is one block per 16 columns of h
// and knows nothing of the device: 448 blocks for h = 7168, but 64 for h = 1024,
// whose experts then stream through 64 of 256 compute units (32 tokens of
// top-8, 256 experts, f 4096: 858 us a call, 2.5 TB/s).
//
// A wave owns 16 weight rows (the A operand of D = W X^T) and a share of the
// channels; its expert's tokens are the B operand, up to 32 at a time: a
// weight is loaded once for 32 tokens of its expert.
#include "experts_device.h"

namespace epx {
namespace {

constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kMaxEntries = kDecodeMaxTokens * EPX_MAX_TOPK;

// Entries of the routing table grouped by expert, in LDS.
struct Groups {
    int start[EPX_MAX_EXPERTS + 1];   // first entry of each expert's list
    short active[EPX_MAX_EXPERTS];    // experts with entries, ascending
    short entry[kMaxEntries];         // t * K + k, expert by expert
    int n_active;
    int part[kDownWaves];
};

// Fills g. An entry whose token already has an earlier entry with the same
// expert is left out: its weight is added to the earlier one's where the
// weights are used. The order inside an expert's list is not fixed; nothing
// depends on it (each list position is a column of its own).
template <int kWaves>
__device__ __forceinline__ void group_entries(const DecodeArgs &a, Groups &g)
{
    constexpr int kThreads = kWaves * kWave;
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

// Eight e4m3 codes as one bf16 operand.
__device__ __forceinline__ i32x4 widen8(int lo, int hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return i32x4{__builtin_bit_cast(int, a), __builtin_bit_cast(int, b),
                 __builtin_bit_cast(int, c), __builtin_bit_cast(int, d)};
}

// No nontemporal hint: a fragment's rows are read in two halves of a 128-byte
// line, and with the hint the second half came from memory again (first
// launch, 48 tokens: 837 us against 696 when it was tried).
__device__ __forceinline__ i32x4 load_weights(const char *p)
{
    return *reinterpret_cast<const i32x4 *>(p);
}

// What a wave needs for 128 bytes of every weight row: G fragments of 16
// weight rows and MT of 16 tokens.
template <bool FP8, int G, int MT>
struct Step {
    static constexpr int kX = FP8 ? 4 : 2;  // 16-byte pieces of a token per lane
    i32x4 w[G][2], x[MT][kX];
    float s[G];
    // wp, xp: the lane's rows; s: the step
    __device__ __forceinline__ void load(const char *const (&wp)[G], const float *const (&ws)[G],
                                         const char *const (&xp)[MT], int s_)
    {
        const int g4 = lane_id() >> 4;
#pragma unroll
        for (int q = 0; q < G; ++q) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                w[q][u] = load_weights(wp[q] + (size_t)s_ * 128 + u * 64 + g4 * 16);
            if (FP8)
                s[q] = ws[q][s_];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < kX; ++v)
                x[i][v] = *reinterpret_cast<const i32x4 *>(
                    xp[i] + (FP8 ? (size_t)s_ * 256 + (v >> 1) * 128 + g4 * 32 + (v & 1) * 16
                                 : (size_t)s_ * 128 + v * 64 + g4 * 16));
    }
    // the last, partial step of bf16 rows: zeros past their end
    __device__ __forceinline__ void load_tail(const char *const (&wp)[G],
                                              const char *const (&xp)[MT], int s_, int bytes)
    {
        const int g4 = lane_id() >> 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at = u * 64 + g4 * 16;
            const bool in = at < bytes;
#pragma unroll
            for (int q = 0; q < G; ++q)
                w[q][u] = in ? load_weights(wp[q] + (size_t)s_ * 128 + at) : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MT; ++i)
                x[i][u] = in ? *reinterpret_cast<const i32x4 *>(xp[i] + (size_t)s_ * 128 + at)
                             : i32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void multiply(f32x4 (&acc)[G][MT]) const
    {
        if constexpr (FP8) {
            f32x4 p[G][MT];
#pragma unroll
            for (int q = 0; q < G; ++q)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    p[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    const i32x4 r = w[q][v >> 1];
                    const i32x4 wv = v & 1 ? widen8(r.z, r.w) : widen8(r.x, r.y);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        p[q][i] = mfma_bf16(wv, x[i][v], p[q][i]);
                }
#pragma unroll
            for (int q = 0; q < G; ++q)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[q][i][c] = __builtin_fmaf(s[q], p[q][i][c], acc[q][i][c]);
        } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int q = 0; q < G; ++q)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        acc[q][i] = mfma_bf16(w[q][u], x[i][u], acc[q][i]);
        }
    }
};

// acc[q][i] = W_q X_i^T over the steps [s0, s1) of rows of `bytes` bytes, the
// loads of D steps under way at a time.
template <bool FP8, int G, int MT, int D>
__device__ __forceinline__ void stream_products(const char *const (&wp)[G],
                                                const float *const (&ws)[G],
                                                const char *const (&xp)[MT], int s0, int s1,
                                                int64_t bytes, f32x4 (&acc)[G][MT])
{
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int full = min(s1, (int)(bytes >> 7));
    if (s0 < full) {
        Step<FP8, G, MT> buf[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            buf[d].load(wp, ws, xp, min(s0 + d, full - 1));
        for (int s = s0; s < full; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d < full)
                    buf[d].multiply(acc);
                buf[d].load(wp, ws, xp, min(s + d + D, full - 1));
            }
        }
    }
    if (!FP8 && full < s1) {
        Step<FP8, G, MT> t;
        t.load_tail(wp, xp, full, (int)(bytes & 127));
        t.multiply(acc);
    }
}

// First launch: 16 columns of f, gate and up, for every token of one expert.
// The block's waves split the channels of h; their sums meet in LDS, part
// [wave][gate, up][token][17].
template <bool FP8, int MT, int D>
__device__ __forceinline__ void up_tile(const DecodeArgs &a, const Groups &g, int e, int n0,
                                        int m0, float *part)
{
    constexpr int kThreads = kUpWaves * kWave;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, l16 = lane & 15;
    const int first = g.start[e] + m0, rows = min(g.start[e + 1] - first, 16 * MT);
    const int64_t bytes = (int64_t)a.h * (FP8 ? 1 : 2);
    const int steps = (int)((bytes + 127) >> 7);
    const int s0 = steps * wave / kUpWaves, s1 = steps * (wave + 1) / kUpWaves;
    const int n = min(n0 + l16, a.f - 1);
    const char *wp[2];
    const float *ws[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        wp[q] = static_cast<const char *>(a.w13) +
                ((int64_t)e * 2 * a.f + (int64_t)q * a.f + n) * bytes;
        ws[q] = FP8 ? a.s13 + ((int64_t)e * (2 * a.f >> 7) + ((q * a.f + n0) >> 7)) * (a.h >> 7)
                    : nullptr;
    }
    // a fragment's rows past the expert's last repeat it: their results are
    // columns of their own, not used
    const char *xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xp[i] = reinterpret_cast<const char *>(
            a.x + (size_t)(g.entry[first + min(i * 16 + l16, rows - 1)] / a.K) * a.h);
    f32x4 acc[2][MT];
    stream_products<FP8, 2, MT, D>(wp, ws, xp, s0, s1, bytes, acc);
    const int T = a.T;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (i * 16 + l16 < rows)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    part[((wave * 2 + q) * T + i * 16 + l16) * 17 + (lane >> 4) * 4 + c] =
                        acc[q][i][c];
    __syncthreads();
    for (int v = tid; v < rows * 16; v += kThreads) {
        const int m = v >> 4, c = v & 15;
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
            gate += part[((w * 2) * T + m) * 17 + c];
            up += part[((w * 2 + 1) * T + m) * 17 + c];
        }
        if (n0 + c < a.f)
            a.act[(size_t)g.entry[first + m] * a.f + n0 + c] =
                (uint16_t)f32_to_bf16(silu_mul(gate, up));
    }
    __syncthreads();
}

template <bool FP8>
__global__ __launch_bounds__(kUpWaves *kWave, 4) void decode_up_kernel(DecodeArgs a)
{
    __shared__ Groups g;
    extern __shared__ float part[];
    group_entries<kUpWaves>(a, g);
    const int nt = (a.f + 15) / 16;
    const int total = g.n_active * nt;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(g.active[t / nt]), n0 = t % nt * 16;
        const int rows = __builtin_amdgcn_readfirstlane(g.start[e + 1] - g.start[e]);
        for (int m0 = 0; m0 < rows; m0 += 32)
            if (rows - m0 <= 16)
                up_tile<FP8, 1, 1>(a, g, e, n0, m0, part);
            else
                up_tile<FP8, 2, 1>(a, g, e, n0, m0, part);
    }
}

// Second launch: 16 columns of h for all tokens. The block's waves take the
// active experts in turn (few experts: shares of their channels), each with
// sums of its own [wave][token][16], which are added in wave order at the
// end: the result does not depend on timing.
template <bool FP8, int MT, int D>
__device__ __forceinline__ void down_tile(const DecodeArgs &a, const Groups &g, int e, int n0,
                                          int m0, int s0, int s1, float *sum)
{
    const int lane = lane_id(), l16 = lane & 15, g4 = lane >> 4;
    const int first = g.start[e] + m0, rows = min(g.start[e + 1] - first, 16 * MT);
    const int64_t bytes = (int64_t)a.f * (FP8 ? 1 : 2);
    const int n = min(n0 + l16, a.h - 1);
    const char *wp[1] = {static_cast<const char *>(a.w2) + ((int64_t)e * a.h + n) * bytes};
    const float *ws[1] = {
        FP8 ? a.s2 + ((int64_t)e * ((a.h + 127) >> 7) + (n0 >> 7)) * (a.f >> 7) : nullptr};
    const char *xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xp[i] = reinterpret_cast<const char *>(
            a.act + (size_t)g.entry[first + min(i * 16 + l16, rows - 1)] * a.f);
    f32x4 acc[1][MT];
    stream_products<FP8, 1, MT, D>(wp, ws, xp, s0, s1, bytes, acc);
#pragma unroll
    for (int i = 0; i < MT; ++i)
        if (i * 16 + l16 < rows) {
            const int j = g.entry[first + i * 16 + l16], t = j / a.K;
            float weight = 0.0f;
            for (int k = j; k < (t + 1) * a.K; ++k)  // repeats of the expert included
                if (a.idx[k] == e)
                    weight += a.topw[k];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float &s = sum[t * 16 + g4 * 4 + c];
                s = __builtin_fmaf(weight, acc[0][i][c], s);
            }
        }
}

template <bool FP8>
__global__ __launch_bounds__(kDownWaves *kWave, 4) void decode_down_kernel(DecodeArgs a)
{
    constexpr int kThreads = kDownWaves * kWave;
    __shared__ Groups g;
    extern __shared__ float sum[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int v = tid; v < kDownWaves * a.T * 16; v += kThreads)
        sum[v] = 0.0f;
    group_entries<kDownWaves>(a, g);
    const int n0 = blockIdx.x * 16;
    const int steps = (int)(((int64_t)a.f * (FP8 ? 1 : 2) + 127) >> 7);
    const int n_active = __builtin_amdgcn_readfirstlane(g.n_active);
    // parts of the channels, so that there is one for every wave
    const int parts = n_active >= kDownWaves ? 1
                                             : min((kDownWaves + n_active - 1) / max(n_active, 1),
                                                   steps);
    for (int i = wave; i < n_active * parts; i += kDownWaves) {
        const int e = __builtin_amdgcn_readfirstlane(g.active[i / parts]), p = i % parts;
        const int s0 = steps * p / parts, s1 = steps * (p + 1) / parts;
        const int rows = __builtin_amdgcn_readfirstlane(g.start[e + 1] - g.start[e]);
        float *const own = sum + wave * a.T * 16;
        for (int m0 = 0; m0 < rows; m0 += 32)
            if (rows - m0 <= 16)
                down_tile<FP8, 1, FP8 ? 1 : 4>(a, g, e, n0, m0, s0, s1, own);
            else
                down_tile<FP8, 2, FP8 ? 1 : 2>(a, g, e, n0, m0, s0, s1, own);
    }
    __syncthreads();
    for (int v = tid; v < a.T * 16; v += kThreads) {
        const int t = v >> 4, c = v & 15;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w)
            s += sum[w * a.T * 16 + v];
        if (n0 + c < a.h)
            a.out[(size_t)t * a.h + n0 + c] = (uint16_t)f32_to_bf16(s);
    }
}

template <bool FP8>
void launch(const DecodeArgs &a, hipStream_t stream)
{
    const int64_t items = (int64_t)(a.E < a.T * a.K ? a.E : a.T * a.K) * ((a.f + 15) / 16);
    const int64_t up = items < 4ll * a.cus ? items : 4ll * a.cus;
    hipLaunchKernelGGL(decode_up_kernel<FP8>, dim3((unsigned)up), dim3(kUpWaves * kWave),
                       kUpWaves * 2 * a.T * 17 * sizeof(float), stream, a);
    hipLaunchKernelGGL(decode_down_kernel<FP8>, dim3((unsigned)((a.h + 15) / 16)),
                       dim3(kDownWaves * kWave), kDownWaves * a.T * 16 * sizeof(float), stream, a);
}

}  // namespace

hipError_t launch_moe_decode(const DecodeArgs &a, bool fp8, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (fp8)
        launch<true>(a, stream);
    else
        launch<false>(a, stream);
    return hipGetLastError();
}

}  // namespace epx
