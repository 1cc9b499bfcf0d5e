// route.hip -- the router's choice of experts, the balance loss with its
// per-expert counts, and the gradient of both with respect to the logits.
//
// Scores of a token's logits l (an expert is live unless its logit is -inf):
//   softmax  s_e = exp(l_e) / sum exp(l),   sigmoid  s_e = 1 / (1 + exp(-l_e)),
// and their shares of one p_e = s_e / sum s (softmax: p = s).
//
// A wave has four tokens, 16 lanes (a row of the data-parallel moves) each:
// sums and maxima over a token's experts take four moves, and instructions
// that concern a token as a whole serve four. Lane i of a token holds the N
// logits of experts 4 (i + 16 q) .. + 3, q < N / 4, which are 16-byte pieces
// of one row, adjacent over the lanes.
#include "gate_device.h"

namespace epx {
namespace {

constexpr float kInf = __builtin_inff();
constexpr int kRow = 16;                  // lanes of a token
constexpr int kTokens = kWave / kRow;     // tokens of a wave

__device__ __forceinline__ int row_lane() { return threadIdx.x & (kRow - 1); }

// The expert of a lane's j-th logit.
__device__ __forceinline__ int expert(int j) { return 4 * (row_lane() + kRow * (j >> 2)) + (j & 3); }

// A lane's N of a row's E values (0 where it has no expert). No load is
// guarded: a lane without an expert reads another of the row's, so the loads
// go out together. wide: E % 4 == 0 and rows of whole 16-byte pieces.
template <int N, typename V4, typename V>
__device__ __forceinline__ void load_row(const V *row, int E, bool wide, V (&v)[N])
{
    if (wide) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const V4 q = *reinterpret_cast<const V4 *>(row + min(expert(j), E - 4));
            v[j] = q.x;
            v[j + 1] = q.y;
            v[j + 2] = q.z;
            v[j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = row[min(expert(j), E - 1)];
    }
}

// A token's logits as loaded: -inf where the lane has no expert or the token is
// not live, and for a NaN or +inf, which sets bad.
template <int N>
__device__ __forceinline__ void clean_logits(int E, bool live, float (&l)[N], bool &bad)
{
    const int end = live ? E : 0;
    if (__ballot(end != kRow * N)) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            l[j] = expert(j) < end ? l[j] : -kInf;
    }
    bool odd = false;
#pragma unroll
    for (int j = 0; j < N; ++j)
        odd |= !(l[j] < kInf);
    if (__ballot(odd)) {
        bad |= odd;
#pragma unroll
        for (int j = 0; j < N; ++j)
            l[j] = l[j] < kInf ? l[j] : -kInf;
    }
}

template <int N>
__device__ __forceinline__ float largest(const float (&l)[N])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < N; ++j)
        m = fmaxf(m, l[j]);
    return row_max(m);
}

// Unnormalised scores with a common factor that keeps the largest near one:
// softmax exp(l - ref), ref the largest logit; sigmoid s / exp(ref), ref the
// largest logit or 0 if that is positive. 0 where not live.
template <bool SIGMOID>
__device__ __forceinline__ float raw_score(float l, float ref)
{
    if (!(l > -kInf))
        return 0.0f;
    if constexpr (SIGMOID) {
        const float t = exp_fp32(-fabsf(l));
        return (l >= 0.0f ? 1.0f : exp_fp32(l - ref)) / (1.0f + t);
    } else {
        return exp_fp32(l - ref);
    }
}

// The logit below which a sigmoid may leave fp32's normal range (it does at
// -87.3): such a token's scores are taken relative to its largest.
constexpr float kLowLogit = -80.0f;

// The reference of a token's entries (-inf where there is none): the largest
// logit; for sigmoids 0, their scores being their own, unless one is low.
template <bool SIGMOID, int M>
__device__ __forceinline__ float entry_ref(const float (&l)[M])
{
    if constexpr (SIGMOID) {
        bool low = false;
#pragma unroll
        for (int m = 0; m < M; ++m)
            low |= l[m] < kLowLogit && l[m] > -kInf;
        if (!__ballot(low))
            return 0.0f;
        const float top = largest(l);
        return row_ballot(low) ? fminf(top, 0.0f) : 0.0f;
    }
    return largest(l);
}

// A score and its slope (softmax: no factor of its gradient, 1; sigmoid
// 1 - s) of an entry, unnormalised as raw_score; ref is the token's.
template <bool SIGMOID>
__device__ __forceinline__ float entry_score(float l, float ref, float &slope)
{
    if constexpr (SIGMOID) {
        const float t = exp_fp32(-fabsf(l));  // 0 for -inf
        const float r = 1.0f / (1.0f + t), u = t * r;
        slope = l >= 0.0f ? u : r;
        return ref < 0.0f ? raw_score<true>(l, ref) : l >= 0.0f ? r : u;
    } else {
        slope = 1.0f;
        return l > -kInf ? exp_fp32(l - ref) : 0.0f;
    }
}

// A token's shares p of one, and with `slopes` the factor of their gradient
// (softmax 1; sigmoid 1 - s). An expert that is not live has p = 0.
template <int N, bool SIGMOID>
__device__ __forceinline__ void shares_of(const float (&l)[N], float (&p)[N], float *slopes)
{
    float sum = 0.0f;
    if constexpr (SIGMOID) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float t = exp_fp32(-fabsf(l[j]));  // 0 for -inf
            const float r = __builtin_amdgcn_rcpf(1.0f + t), u = t * r;
            p[j] = l[j] >= 0.0f ? r : u;
            if (slopes)
                slopes[j] = l[j] >= 0.0f ? u : r;
            sum += p[j];
        }
        sum = row_sum(sum);
        // a share is in fp32's normal range and its score may not be: relative
        // to the largest, the token's alone, so that none depends on the others
        // of its wave (above a sum of 1/2 the shares leave the range too)
        if (__ballot(sum < 0.5f)) {
            bool low = false;
#pragma unroll
            for (int j = 0; j < N; ++j)
                low |= l[j] < kLowLogit && l[j] > -kInf;
            low = row_ballot(low) != 0 && sum < 0.5f;
            if (__ballot(low)) {
                const float ref = fminf(largest(l), 0.0f);
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float q = raw_score<true>(l[j], ref);
                    p[j] = low ? q : p[j];
                    s += q;
                }
                s = row_sum(s);
                sum = low ? s : sum;
            }
        }
    } else {
        const float top = largest(l);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p[j] = exp_fp32(l[j] - top);  // 0 for -inf (and -inf less itself, a NaN)
            sum += p[j];
        }
        sum = row_sum(sum);
    }
    const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
        p[j] *= r;
}

// ------------------------------------------------------------------- choice
//
// The choice is that of the scores in 64 bits (without a bias that of the
// logits). It is made on whole numbers that rise with the keys (score + bias; without a bias the logits themselves): a
// key's distance from the token's largest in fixed point, with the expert's
// number below it, so that one unsigned maximum or minimum moves both and
// equal keys order by their experts. Each lane sorts its experts in such
// words, lists of the L best are merged over the 16 lanes, and a token whose
// outcome falls between keys that are nearer than their error (or than the
// fixed point tells), unless these are of equal logits and biases, is done
// again in 64 bits.
//
// Bound by vector instructions, not by memory: 16384 tokens of 256 experts, top-8
// of the best 4 of 8 groups, sigmoid with a bias (18 MB, 2.6 us at a read's
// rate) 14.4 us at 1060 instructions a wave, four waves a SIMD. Without the
// second look it would be 12.4: some ten tokens take it, which the others do not
// hide (it is part of the kernel, since as a function it took its arguments
// from memory, 0.5 us more; compared through LDS its candidates took another
// 0.5). Softmax without groups or bias 8.0 us. 128 tokens 3.0: one wave's chain
// of a load, the merges and the weights.

// Fixed point: B bits for a window below the token's largest key. Keys below
// the window all have 0, as does what is not live (and what the conversion
// gets as a NaN or less than nothing): a token that takes such a key is done
// again.
template <int N>
struct Word {
    static constexpr int kId = N == 4 ? 6 : N == 8 ? 7 : N == 16 ? 8 : 9;
    static constexpr uint32_t kIdMask = (1u << kId) - 1u;
    static constexpr int kBits = N <= 16 ? 24 : 23;  // what fp32 counts exactly
    static constexpr float kMost = (float)((1u << kBits) - 1u);
    static __device__ __forceinline__ uint32_t make(float key, float top, float per_unit, int e)
    {
        uint32_t f;  // as the instruction does: 0 below nothing and for a NaN
        asm("v_cvt_u32_f32 %0, %1" : "=v"(f) : "v"(__builtin_fmaf(key - top, per_unit, kMost)));
        return (f << kId) | (kIdMask - (uint32_t)e);
    }
    static __device__ __forceinline__ int id(uint32_t w) { return (int)(kIdMask - (w & kIdMask)); }
    static __device__ __forceinline__ int key(uint32_t w) { return (int)(w >> kId); }
};

// Width of the window: logits, and keys that are scores with a bias.
constexpr float kLogitWindow = 32.0f, kKeyWindow = 2.0f;

__device__ __forceinline__ void descend(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// Any order -> descending: odd-even merges (19 exchanges of 8 words, 63 of 16).
template <int M>
__device__ __forceinline__ void sort_words(uint32_t (&w)[M])
{
#pragma unroll
    for (int p = 1; p < M; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = 0; j < M; ++j) {
                // j is the upper of a pair of its merge
                const int r = j - k % p;
                if (r >= 0 && (r / k) % 2 == 0 && j + k < M && j / (2 * p) == (j + k) / (2 * p))
                    descend(w[j], w[j + k]);
            }
}

// One that falls and then rises (or the reverse) -> descending.
template <int M>
__device__ __forceinline__ void sort_bitonic(uint32_t (&w)[M])
{
#pragma unroll
    for (int j = M / 2; j > 0; j /= 2)
#pragma unroll
        for (int i = 0; i < M; ++i)
            if ((i ^ j) > i)
                descend(w[i], w[i ^ j]);
}

// The L best of a lane's N words, descending.
template <int N, int L>
__device__ __forceinline__ void best_of_lane(const uint32_t (&w)[N], uint32_t (&best)[L])
{
    if constexpr (N <= L) {
        uint32_t s[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            s[j] = w[j];
        sort_words<N>(s);
#pragma unroll
        for (int j = 0; j < L; ++j)
            best[j] = j < N ? s[j < N ? j : 0] : 0u;
    } else {
#pragma unroll
        for (int p = 0; p < N; p += L) {
            uint32_t s[L];
#pragma unroll
            for (int j = 0; j < L; ++j)
                s[j] = w[p + j];
            sort_words<L>(s);
            if (p == 0) {
#pragma unroll
                for (int j = 0; j < L; ++j)
                    best[j] = s[j];
            } else {
                // of two descending lists the larger of i-th and (L-1-i)-th
                // are the L best
#pragma unroll
                for (int j = 0; j < L; ++j)
                    best[j] = max(best[j], s[L - 1 - j]);
                sort_bitonic<L>(best);
            }
        }
    }
}

template <int L, int CTRL>
__device__ __forceinline__ void merge_lanes(uint32_t (&best)[L])
{
    uint32_t o[L];
#pragma unroll
    for (int j = 0; j < L; ++j)
        o[j] = (uint32_t)EPX_ROW(best[j], CTRL);
#pragma unroll
    for (int j = 0; j < L; ++j)
        best[j] = max(best[j], o[L - 1 - j]);
    sort_bitonic<L>(best);
}

// How near two keys may be and yet stand the other way round when exact: twice
// a key's error. Without a bias the words rise with the logits themselves and
// only equal ones tell nothing. With one, a key is off by
//   the sigmoid's error, below 3e-7: its exponential is within
//     (1.25 |l| + 2) 2^-24 of itself, which s (1 - s) |l| < 0.224 and s (1 - s)
//     <= 1/4 scale down, then an addition's rounding and a reciprocal's unit;
//   the softmax's, below 4e-6 of the token's largest score for a pair (the sum
//     of 512 terms, each within (2.25 |x| + 2) 2^-24, is common to both);
//   the bias's addition, 2^-24 of the key.
template <bool SIGMOID>
__device__ __forceinline__ float pair_tol(float largest_score, float largest_key)
{
    return (SIGMOID ? 0x1p-20f : 0x1p-17f * largest_score) + 0x1p-22f * largest_key;
}

// LDS of a wave's four tokens.
template <int N, int L>
struct RouteLds {
    // a unit of a group is one expert's key, or where groups are made of fours
    // the two best of these; spread so that lanes which walk different groups
    // meet different banks
    float unit[kTokens][kRow * N + kRow * N / 8 + 4];
    float score[kTokens][64];
    uint32_t chosen[kTokens][L];
    double key64[kRow * N];
    uint16_t candidate[kRow * N];
    static __device__ __forceinline__ int at(int u) { return u + (u >> 3); }
};

// What a wave wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The two largest of x, y and of another's.
__device__ __forceinline__ void best_two(float &x, float &y, float ox, float oy)
{
    y = fmaxf(fmaxf(y, oy), fminf(x, ox));
    x = fmaxf(x, ox);
}

// Bits of the groups that stay, at (group << shift); near: half of a kept and
// of a dropped group's scores are within tol of each other (halves, because
// two keys of the type's largest or lowest value have no sum in fp32).
// 2^shift lanes of a token walk a group (one with more than 16 groups, when a
// lane has several).
template <int N, int L>
__device__ __forceinline__ uint64_t best_groups(const RouteArgs &a, RouteLds<N, L> &lds, int shift,
                                                bool fours, float tol, bool &near)
{
    const int row = lane_id() / kRow, i = row_lane(), P = 1 << shift, part = i & (P - 1);
    const float *unit = lds.unit[row];
    float *score = lds.score[row];
    for (int g0 = 0; g0 < a.G; g0 += kRow >> shift) {
        const int g = min(g0 + (i >> shift), a.G - 1);
        float x = -kInf, y = -kInf;
        if (fours) {
            const int units = a.group_size >> 2;
            for (int m = part; m < units; m += P) {
                const float2 k = *reinterpret_cast<const float2 *>(
                    &unit[2 * RouteLds<N, L>::at(g * units + m)]);
                best_two(x, y, k.x, k.y);
            }
        } else {
            for (int m = part; m < a.group_size; m += P)
                best_two(x, y, unit[RouteLds<N, L>::at(g * a.group_size + m)], -kInf);
        }
        for (int d = 1; d < P; d <<= 1)
            best_two(x, y, __shfl_xor(x, d, kWave), __shfl_xor(y, d, kWave));
        if (part == 0)
            score[g] = y > -kInf ? 0.5f * x + 0.5f * y : 0.5f * x;
    }
    wave_lds();
    uint64_t bits = 0;
    float lo = kInf, hi = -kInf;
    for (int g0 = 0; g0 < a.G; g0 += kRow >> shift) {
        const int g = g0 + (i >> shift);
        const float mine = g < a.G ? score[g] : -kInf;
        int rank = 0;
        for (int o = 0; o < a.G; ++o) {
            const float s = score[o];
            rank += s > mine || (s == mine && o < g);
        }
        const bool kept = g < a.G && rank < a.top_groups && mine > -kInf;
        bits |= (uint64_t)row_ballot(kept && part == 0) << (g0 << shift);
        lo = kept ? fminf(lo, mine) : lo;
        hi = kept ? hi : fmaxf(hi, mine);
    }
    lo = -row_max(-lo);
    hi = row_max(hi);
    near = lo < kInf && hi > -kInf && lo - hi <= tol;
    return bits;
}

// Scores in 64 bits, one token's by the whole wave.
template <bool SIGMOID>
struct Exact {
    const RouteArgs &a;
    const float *row;
    double top, sum;
    // scores: keys are scores (else nothing is made of them)
    __device__ __forceinline__ Exact(const RouteArgs &args, int64_t t, bool scores)
        : a(args), row(args.logits + (size_t)t * args.E), top(0.0), sum(0.0)
    {
        if (!SIGMOID && scores) {
            float m = -kInf;
            for (int e = lane_id(); e < a.E; e += kWave)
                m = fmaxf(m, logit(e));
            for (int d = 1; d < kWave; d <<= 1)
                m = fmaxf(m, __shfl_xor(m, d, kWave));
            top = (double)m;
            for (int e = lane_id(); e < a.E; e += kWave) {
                const float l = logit(e);
                sum += l > -kInf ? exp((double)l - top) : 0.0;
            }
            for (int d = 1; d < kWave; d <<= 1)
                sum += __shfl_xor(sum, d, kWave);
        }
    }
    __device__ __forceinline__ float logit(int e) const { return row[e] < kInf ? row[e] : -kInf; }
    // score and bias of a logit, -inf if it can not be chosen
    __device__ __forceinline__ double key(float l, float b) const
    {
        const double v = (double)l;
        const double s = SIGMOID ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum;
        return l > -kInf && l < kInf && b < kInf ? s + (double)b : -(double)kInf;
    }
};

// One token's groups in 64 bits by the whole wave: bit g for a group that stays.
template <int N, int L, bool SIGMOID>
__device__ __forceinline__ uint64_t groups64(const RouteArgs &a, int64_t t, RouteLds<N, L> &lds)
{
    const Exact<SIGMOID> exact(a, t, true);
    const int lane = lane_id();
    for (int e = lane; e < a.E; e += kWave)
        lds.key64[e] = exact.key(exact.row[e], a.bias ? a.bias[e] : 0.0f);
    wave_lds();
    int P = 1;  // lanes of a group
    while (2 * P * a.G <= kWave)
        P *= 2;
    const int g = lane / P;
    double x = -(double)kInf, y = x;
    if (g < a.G)
        for (int m = lane % P; m < a.group_size; m += P) {
            const double k = lds.key64[g * a.group_size + m];
            y = k > x ? x : k > y ? k : y;
            x = k > x ? k : x;
        }
    for (int d = 1; d < P; d <<= 1) {
        const double ox = __shfl_xor(x, d, kWave), oy = __shfl_xor(y, d, kWave);
        y = ox > x ? (x > oy ? x : oy) : (ox > y ? ox : y);
        x = ox > x ? ox : x;
    }
    const double mine = y > -(double)kInf ? x + y : x;
    int rank = 0;
    for (int o = 0; o < a.G; ++o) {
        const double s = __shfl(mine, o * P, kWave);
        rank += s > mine || (s == mine && o < g);
    }
    uint64_t todo = uniform64(__ballot(g < a.G && lane % P == 0 && rank < a.top_groups &&
                                       mine > -(double)kInf));
    uint64_t bits = 0;
    for (; todo; todo &= todo - 1)
        bits |= 1ull << (__builtin_ctzll(todo) / P);
    return bits;
}

// One token's choice in 64 bits by the whole wave, among n candidates: chosen[r]
// is the r-th expert's number, or ~0.
template <int N, int L, bool SIGMOID>
__device__ __forceinline__ void choose64(const RouteArgs &a, int64_t t, int n, RouteLds<N, L> &lds,
                                         uint32_t *chosen)
{
    const int lane = lane_id();
    const Exact<SIGMOID> exact(a, t, a.bias != nullptr);
    // a candidate's place in the order (without a bias that of the logits), -inf
    // if it can not be chosen
    const auto key = [&](int e) {
        const float l = exact.row[e];
        return a.bias ? exact.key(l, a.bias[e]) : l < kInf ? (double)l : -(double)kInf;
    };
    if (lane < L)
        chosen[lane] = ~0u;
    wave_lds();
    if (n <= kWave) {  // one each, compared from lane to lane
        const int e = lane < n ? lds.candidate[lane] : 0;
        const double k = key(e);
        const int lo = __double2loint(k), hi = __double2hiint(k);
        int rank = 0;
        for (int o = 0; o < n; ++o) {
            const double ok = __hiloint2double(__builtin_amdgcn_readlane(hi, o),
                                               __builtin_amdgcn_readlane(lo, o));
            rank += ok > k || (ok == k && __builtin_amdgcn_readlane(e, o) < e);
        }
        if (lane < n && k > -(double)kInf && rank < a.K)
            chosen[rank] = (uint32_t)e;
    } else {
        for (int c = lane; c < n; c += kWave)
            lds.key64[c] = key(lds.candidate[c]);
        wave_lds();
        for (int c = lane; c < n; c += kWave) {
            const int e = lds.candidate[c];
            const double k = lds.key64[c];
            if (!(k > -(double)kInf))
                continue;
            int rank = 0;
#pragma unroll 4
            for (int o = 0; o < n; ++o) {
                const double ok = lds.key64[o];
                rank += ok > k || (ok == k && lds.candidate[o] < e);
            }
            if (rank < a.K)
                chosen[rank] = (uint32_t)e;
        }
    }
    wave_lds();
}

template <int N, int L, bool SIGMOID>
__global__ __launch_bounds__(kWave, N <= 16 ? 4 : 2) void route_kernel(RouteArgs a, bool wide, bool wide_bias,
                                                      int shift, bool normalize)
{
    typedef Word<N> W;
    __shared__ RouteLds<N, L> lds;
    const int row = lane_id() / kRow, i = row_lane();
    const int64_t t = (int64_t)blockIdx.x * kTokens + row;
    const int64_t tc = min(t, (int64_t)a.T - 1);  // what is read in place of a token behind the last
    const bool live = t < a.T && (!a.mask || a.mask[tc]);
    const float *logits = a.logits + (size_t)tc * a.E;
    float l[N], b[N];
    bool bad = false;
    load_row<N, float4, float>(logits, a.E, wide, l);
    if (a.bias)
        load_row<N, float4, float>(a.bias, a.E, wide_bias, b);
    clean_logits<N>(a.E, live, l, bad);
    const float top_l = largest(l);
    float sum_l = 1.0f;  // of the softmax, where the weights need it
    if (!SIGMOID && !normalize) {
        sum_l = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            sum_l += exp_fp32(l[j] - top_l);  // 0 for -inf
        sum_l = row_sum(sum_l);
    }

    // order values: the logits, or scores with their bias
    float order[N];
    float per_unit = (W::kMost + 1.0f) / kLogitWindow, top = top_l;
    int tol = 0;
    bool near = false;
    uint64_t kept = 0;  // groups that stay
    const auto stays = [&](int e) {
        return kept >> (div_by_magic(e, a.size_mul) << shift & 63) & 1;
    };
#pragma unroll
    for (int j = 0; j < N; ++j)
        order[j] = l[j];
    if (a.bias || a.G > 1) {
        float best = 0.0f, key[N], most = 0.0f;  // most: largest magnitude of a key
        if constexpr (SIGMOID) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                key[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[j] * -0x1.715476p+0f));
            most = 1.0f;
        } else {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                key[j] = __builtin_amdgcn_exp2f((l[j] - top_l) * 0x1.715476p+0f);
                sum += l[j] > -kInf ? key[j] : 0.0f;
            }
            best = most = __builtin_amdgcn_rcpf(row_sum(sum));  // of the largest logit
#pragma unroll
            for (int j = 0; j < N; ++j)
                key[j] *= best;
        }
        if (a.bias) {
            bool odd = false;
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                key[j] += b[j];
                odd |= !(fabsf(b[j]) < kInf);
                m = fmaxf(m, fabsf(b[j]));
            }
            if (__ballot(odd)) {  // -inf: not chosen; NaN, +inf: nor those
                m = 0.0f;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const bool can = fabsf(b[j]) < kInf;
                    bad |= live && !(b[j] < kInf);
                    key[j] = can ? key[j] : -kInf;
                    m = fmaxf(m, can ? fabsf(b[j]) : 0.0f);
                }
            }
            most += row_max(m);
        }
        float least = l[0];
#pragma unroll
        for (int j = 1; j < N; ++j)
            least = fminf(least, l[j]);
        if (__ballot(!(least > -kInf))) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                key[j] = l[j] > -kInf ? key[j] : -kInf;
        }
        const float pair = pair_tol<SIGMOID>(best, most);
        const bool fours = a.group_size % 4 == 0;
        if (a.G > 1) {
            float *unit = lds.unit[row];
            if (fours) {
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    float x = fmaxf(key[j], key[j + 1]), y = fminf(key[j], key[j + 1]);
                    best_two(x, y, fmaxf(key[j + 2], key[j + 3]), fminf(key[j + 2], key[j + 3]));
                    *reinterpret_cast<float2 *>(
                        &unit[2 * RouteLds<N, L>::at(expert(j) >> 2)]) = float2{x, y};
                }
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    unit[RouteLds<N, L>::at(expert(j))] = key[j];
            }
            wave_lds();
            // half a score is two halves of a key and a rounding
            kept = best_groups<N, L>(a, lds, shift, fours, 1.5f * pair, near);
            const uint64_t unsure = uniform64(__ballot(near && live));
#pragma unroll 1
            for (int q = 0; unsure && q < kTokens; ++q) {
                if (!(unsure >> (q * kRow) & 0xFFFF))
                    continue;
                uint64_t bits = groups64<N, L, SIGMOID>(
                    a, (int64_t)blockIdx.x * kTokens + q, lds);
                if (row == q) {
                    kept = 0;
                    for (; bits; bits &= bits - 1)
                        kept |= 1ull << (__builtin_ctzll(bits) << shift);
                }
            }
        }
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                order[j] = key[j];
        }
        if (a.G > 1) {
            if (fours) {
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    const bool s = stays(expert(j));
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        order[j + r] = s ? order[j + r] : -kInf;
                }
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    order[j] = stays(expert(j)) ? order[j] : -kInf;
            }
        }
        top = largest(order);
        if (a.bias) {
            per_unit = (W::kMost + 1.0f) / kKeyWindow;
            tol = (int)fminf(pair * per_unit, W::kMost) + 2;
        }
    }
    uint32_t w[N], best[L];
#pragma unroll
    for (int j = 0; j < N; ++j)
        w[j] = W::make(order[j], top, per_unit, expert(j));
    best_of_lane<N, L>(w, best);
    merge_lanes<L, 0x128>(best);  // row_ror: 8, 4, 2, 1
    merge_lanes<L, 0x124>(best);
    merge_lanes<L, 0x122>(best);
    merge_lanes<L, 0x121>(best);
    if (i == 0) {
#pragma unroll
        for (int j = 0; j < L; ++j)
            lds.chosen[row][j] = best[j];
    }
    wave_lds();
    // the K-th, and whether one that is left out is as near
    const uint32_t last = lds.chosen[row][a.K - 1];
    const uint32_t from = W::key(last) > tol ? (uint32_t)(W::key(last) - tol) << W::kId : 0u;
    bool beside = false;
#pragma unroll
    for (int j = 0; j < N; ++j)
        beside |= w[j] - from < last - from;
    // (all experts again where the K-th is below the window or not live)
    const bool blind = live && W::key(last) <= tol;
    near = blind;
    if (__ballot(beside && live && !blind)) {
        const int le = W::id(last);
        const bool look = beside && live && !blind;
        const float ll = look ? logits[le] : 0.0f;
        const float lb = look && a.bias ? a.bias[le] : 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (look && w[j] - from < last - from)
                near |= logits[expert(j)] != ll || (a.bias && a.bias[expert(j)] != lb);
    }
    constexpr int kPer = (L + kRow - 1) / kRow;  // entries of a lane: i, i + 16
    int e[kPer];
    float lk[kPer];
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        const int r = i + m * kRow;
        const bool have = live && !blind && r < a.K;
        const uint32_t mine = have ? lds.chosen[row][r] : 0u;
        e[m] = have ? W::id(mine) : -1;
        lk[m] = have ? logits[e[m]] : -kInf;
        const uint32_t next = have && r + 1 < a.K ? lds.chosen[row][r + 1] : 0u;
        if (next && W::key(mine) - W::key(next) <= tol) {
            const int ne = W::id(next);
            near |= lk[m] != logits[ne] || (a.bias && a.bias[e[m]] != a.bias[ne]);
        }
    }
    const uint64_t again = uniform64(__ballot(near));
    if (again) {
        // (the compiler is kept from holding what this rare path needs in
        // registers from before)
        int experts = a.E;
        asm volatile("" : "+v"(kept), "+v"(experts));
#pragma unroll 1
        for (int q = 0; q < kTokens; ++q) {
            if (!(again >> (q * kRow) & 0xFFFF))
                continue;
            // the experts that are not clearly below the K-th
            int n = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool can = row == q && expert(j) < experts &&
                                 (blind ? a.G == 1 || stays(expert(j)) : w[j] >= from);
                const uint64_t m = uniform64(__ballot(can));
                if (!m)
                    continue;
                if (can)
                    lds.candidate[n + __builtin_popcountll(m & lanes_below(lane_id()))] =
                        (uint16_t)expert(j);
                n += __builtin_popcountll(m);
            }
            wave_lds();
            choose64<N, L, SIGMOID>(a, (int64_t)blockIdx.x * kTokens + q, n, lds, lds.chosen[q]);
        }
        if (again >> (row * kRow) & 0xFFFF) {
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
                const int r = i + m * kRow;
                e[m] = r < a.K ? (int)lds.chosen[row][r] : -1;
                lk[m] = e[m] >= 0 ? logits[e[m]] : -kInf;
            }
        }
    }
    // weights
    float v[kPer], total = 1.0f;
    if (normalize) {
        float sum = 0.0f;
        const float ref = entry_ref<SIGMOID>(lk);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            float slope;
            v[q] = entry_score<SIGMOID>(lk[q], ref, slope);
            sum += v[q];
        }
        total = row_sum(sum);
    } else if constexpr (SIGMOID) {
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            v[q] = raw_score<true>(lk[q], 0.0f);
    } else {
        total = sum_l;
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            v[q] = raw_score<false>(lk[q], top_l);
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int r = i + q * kRow;
        if (t < a.T && r < a.K) {
            a.topk_idx[t * a.K + r] = e[q];
            a.topk_w[t * a.K + r] = e[q] >= 0 ? a.scale * (v[q] / total) : 0.0f;
        }
    }
    if (bad)
        flag_error(a.err, EPX_DEV_BAD_LOGIT);
}

// -------------------------------------------------------------- balance loss
//
// Per sequence s of n tokens that have a route (an entry >= 0), with c_e
// entries for expert e and P_e the mean share of e over those tokens:
//   loss_s = E / (K n) sum_e c_e P_e,  loss = mean of loss_s over the
// sequences with n > 0 (0 without any).
//
// First launch: a block has a run of consecutive tokens, one for each 16
// lanes, and leaves a row of sums for each sequence that meets the run, at row
// (run + sequence): a place of its own, because runs and sequences ascend
// together. Second launch: a block has 64 experts of one sequence and adds
// their rows; the last block to end adds the losses. A batch of one run needs
// the first launch alone. Bound by the chain of the two launches' latencies:
// 16384 tokens of 256 experts in 24 sequences (17 MB, 2.4 us at a read's rate)
// 14 us, of which the first launch 9.3; 64 tokens of 8 experts 4.2 us.

template <int N, int TOKENS>
struct Run {
    static constexpr int kTokensOfRun = TOKENS;
    static constexpr int kWaves = kTokensOfRun / kTokens;
    static constexpr int kColumns = kRow * N;
    static constexpr int kThreads = kWaves * kWave;
    // threads of a column share the run's tokens
    static constexpr int kShares = kThreads / kColumns < kTokensOfRun ? kThreads / kColumns
                                                                      : kTokensOfRun;
    static constexpr int kShare = kTokensOfRun / kShares;
};

constexpr int kFinalColumns = 64, kFinalThreads = 1024;

inline size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Tokens of a run: 64, or with more than 128 experts 32, so that two blocks
// share a compute unit (65536 tokens of 256 experts 29.6 us against 38.5, 1024
// 9.9 against 11.9) -- but 64 still where that spares the second launch (64
// tokens 6.6 against 9.2; above 256 experts the LDS does not hold them).
__host__ __device__ inline int run_shift(int T, int E)
{
    return E <= 128 || (E <= 256 && T <= 64) ? 6 : 5;
}

inline int run_tokens(int T, int E) { return 1 << run_shift(T, E); }

inline int64_t balance_rows(int T, int E, int S)
{
    return ((int64_t)T + run_tokens(T, E) - 1) / run_tokens(T, E) + (int64_t)S;
}

// The parts of a workspace that begins at p; returns its bytes.
size_t balance_ws(char *p, int T, int E, int S, BalanceWs &w)
{
    const size_t rows = (size_t)balance_rows(T, E, S);
    const size_t parts = (E + kFinalColumns - 1) / kFinalColumns;
    char *const p0 = p;
    w.done = reinterpret_cast<unsigned int *>(p);
    p += 16;
    w.dot = reinterpret_cast<float *>(p);
    p += up16((size_t)S * parts * 4);
    w.seen = reinterpret_cast<int *>(p);
    p += up16(rows * 4);
    w.counts = reinterpret_cast<int *>(p);
    p += up16(rows * E * 4);
    w.probs = reinterpret_cast<float *>(p);
    p += up16(rows * E * 4);
    return (size_t)(p - p0);
}

// Sequence s's tokens, kept inside [0, T).
__device__ __forceinline__ void sequence(const int32_t *off, int s, int T, int &lo, int &hi,
                                         bool &bad)
{
    if (!off) {
        lo = 0;
        hi = T;
        return;
    }
    const int a = off[s], b = off[s + 1];
    lo = min(max(a, 0), T);
    hi = min(max(b, lo), T);
    bad |= a != lo || b != hi;
}

// The sequence that a token is in: the offsets that are not above t are the
// first ones, and the last of them begins it. The token's 16 lanes look at 64
// offsets at a time, so that up to 63 sequences take one load's latency; that
// load is apart, to go out before the token's own.
struct SequenceSearch {
    int o[4];
    static __device__ __forceinline__ int step(int n) { return (n + 63) >> 6; }
    static __device__ __forceinline__ int at(int m, int n)
    {
        return (m * kRow + row_lane() + 1) * step(n) - 1;
    }
    __device__ __forceinline__ void load(const int32_t *off, int S, int lo, int n)
    {
#pragma unroll
        for (int m = 0; m < 4; ++m)
            o[m] = off[min(lo + at(m, n), S)];
    }
    __device__ __forceinline__ void begin(const int32_t *off, int S)
    {
        if (off)
            load(off, S, 0, S + 1);
    }
    // the number, or -1
    __device__ __forceinline__ int find(const int32_t *off, int S, int t)
    {
        if (!off)
            return 0;
        int lo = 0, n = S + 1;  // offsets [lo, lo + n) are not decided
        for (;;) {
            int c = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                c += __builtin_popcount(row_ballot(n > 0 && at(m, n) < n && o[m] <= t));
            lo += c * step(n);
            n = n > 0 ? min(n - c * step(n), step(n) - 1) : 0;
            if (!__ballot(n > 0))
                return lo <= S ? lo - 1 : -1;
            load(off, S, lo, n);
        }
    }
};

template <int N, int TOKENS, bool SIGMOID>
__global__ __launch_bounds__((Run<N, TOKENS>::kThreads)) void balance_kernel(BalanceArgs a, bool wide)
{
    typedef Run<N, TOKENS> R;
    __shared__ __align__(16) float share[R::kTokensOfRun][R::kColumns];
    __shared__ __align__(16) uint32_t cnt[R::kTokensOfRun][R::kColumns / 2];  // two experts a word
    __shared__ int seq[R::kTokensOfRun];
    __shared__ int has_route[R::kTokensOfRun];
    __shared__ float seq_loss[R::kTokensOfRun];
    const int tid = threadIdx.x, wave = tid / kWave, lane = lane_id();
    const int mine = tid / kRow, i = row_lane();  // this token of the run
    const BalanceWs &ws = a.ws;
    const bool whole = gridDim.x == 1;
    const int64_t t = (int64_t)blockIdx.x * R::kTokensOfRun + mine;
    bool bad_off = false, bad_logit = false, bad_route = false;

    // what is read of the token, before its sequence is known
    SequenceSearch search;
    search.begin(a.seq_off, a.S);
    constexpr int kPer = 2;  // entries of a lane: i, i + 16
    int64_t e[kPer];
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        const int k = i + m * kRow;
        e[m] = t < a.T && k < a.K ? a.topk_idx[t * a.K + k] : -1;
    }
    float l[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
        l[j] = -kInf;
    if (a.T > 0)
        load_row<N, float4, float>(a.logits + (size_t)min(t, (int64_t)a.T - 1) * a.E, a.E, wide, l);
    for (int c = tid; c < R::kTokensOfRun * R::kColumns / 8; c += R::kThreads)
        reinterpret_cast<uint4 *>(&cnt[0][0])[c] = uint4{0u, 0u, 0u, 0u};
    int s = search.find(a.seq_off, a.S, (int)min(t, (int64_t)a.T));
    s = t < a.T ? s : -1;
    bool named[kPer];
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        named[m] = s >= 0 && e[m] >= 0 && e[m] < a.E;
        bad_route |= s >= 0 && (e[m] < -1 || e[m] >= a.E);
    }
    const bool seen = row_ballot(named[0] || named[1]) != 0;
    clean_logits<N>(a.E, t < a.T, l, bad_logit);
    bad_logit = bad_logit && seen;
    if (i == 0) {
        seq[mine] = s;
        has_route[mine] = seen;
    }
    if (blockIdx.x == 0) {
        if (tid == 0 && !whole)
            *ws.done = 0;
        for (int q = tid; q < a.S; q += R::kThreads) {
            int lo, hi;
            sequence(a.seq_off, q, a.T, lo, hi, bad_off);
            if (whole && lo == hi) {  // without tokens
                a.num_tokens[q] = 0;
                for (int c = 0; c < a.E; ++c) {
                    a.counts[(size_t)q * a.E + c] = 0;
                    a.probs[(size_t)q * a.E + c] = 0.0f;
                }
            }
        }
    }
    {
        float p[N];
        shares_of<N, SIGMOID>(l, p, nullptr);
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(&share[mine][expert(j)]) =
                seen ? float4{p[j], p[j + 1], p[j + 2], p[j + 3]}
                     : float4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();
    // the run's sequences: bit b of starts is set where token b's is another
    // than the one's before it
    const int sq = lane < R::kTokensOfRun ? seq[lane] : -2;
    const int before = lane == 0 ? -2 : seq[lane < R::kTokensOfRun ? lane - 1 : 0];
    const uint64_t starts =
        uniform64(__ballot(lane < R::kTokensOfRun && (lane == 0 || sq != before)));
    const uint64_t routed = uniform64(__ballot(lane < R::kTokensOfRun && has_route[lane]));
    const int segments = __builtin_popcountll(starts);
    const int segment = __builtin_popcountll(starts & lanes_below(mine + 1)) - 1;
#pragma unroll
    for (int m = 0; m < kPer; ++m)
        if (named[m])
            atomicAdd(&cnt[segment][(int)e[m] >> 1], (e[m] & 1) ? 0x10000u : 1u);
    // sums over the tokens of a sequence, a part of the run each; a sum is left
    // in the place of its first token
    const int col = tid % R::kColumns;
    const int part = __builtin_amdgcn_readfirstlane(tid / R::kColumns);  // (whole waves)
    if (part < R::kShares) {
        float q = 0.0f;
        int first = part * R::kShare;
#pragma unroll
        for (int b = 0; b < R::kShare; ++b) {
            const int at = part * R::kShare + b;
            const float v = share[at][col];
            if (b > 0 && (starts >> at & 1)) {
                share[first][col] = q;
                first = at;
                q = 0.0f;
            }
            q += v;
        }
        share[first][col] = q;
    }
    __syncthreads();
    for (int g = wave; g < segments; g += R::kWaves) {
        // tokens [b0, b1) of the run
        uint64_t rest = starts;
        for (int d = 0; d < g; ++d)
            rest &= rest - 1;
        const int b0 = __builtin_ctzll(rest);
        rest &= rest - 1;
        const int b1 = rest ? __builtin_ctzll(rest) : R::kTokensOfRun;
        const int sg = seq[b0];
        if (sg < 0) {
            if (lane == 0)
                seq_loss[g] = -1.0f;
            continue;
        }
        const int n = __builtin_popcountll(routed >> b0 << b0 & (b1 == 64 ? ~0ull : ~(~0ull << b1)));
        const size_t out = (size_t)(whole ? sg : blockIdx.x + sg) * a.E;
        float dot = 0.0f;
        for (int c = lane; c < a.E; c += kWave) {
            float q = share[b0][c];
            for (int b = (b0 / R::kShare + 1) * R::kShare; b < b1; b += R::kShare)
                q += share[b][c];
            const int k = cnt[g][c >> 1] >> ((c & 1) * 16) & 0xFFFF;
            if (whole) {
                q = n ? q / (float)n : 0.0f;
                a.counts[out + c] = k;
                a.probs[out + c] = q;
                dot = __builtin_fmaf((float)k, q, dot);
            } else {
                ws.counts[out + c] = k;
                ws.probs[out + c] = q;
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) {
            seq_loss[g] = n ? dot * ((float)a.E / ((float)a.K * (float)n)) : -1.0f;
            if (whole)
                a.num_tokens[sg] = n;
            else
                ws.seen[blockIdx.x + sg] = n;
        }
    }
    if (whole) {
        __syncthreads();
        if (tid == 0) {
            float total = 0.0f;
            int some = 0;
            for (int g = 0; g < segments; ++g)
                if (seq_loss[g] >= 0.0f) {  // of a sequence with tokens
                    total += seq_loss[g];
                    ++some;
                }
            a.num_tokens[a.S] = some;
            a.loss[0] = some ? total / (float)some : 0.0f;
        }
    }
    if (bad_logit || bad_off || bad_route)
        flag_error(a.err, (bad_logit ? EPX_DEV_BAD_LOGIT : 0) | (bad_off ? EPX_DEV_OVERFLOW : 0) |
                              (bad_route ? EPX_DEV_BAD_ROUTE : 0));
}

// Tokens of sequence s that count: the sum of its rows' numbers.
__device__ __forceinline__ int tokens_seen(const BalanceWs &ws, int s, int r0, int r1)
{
    int n = 0;
    for (int r = r0 + lane_id(); r < r1; r += kWave)
        n += ws.seen[r + s];
    return __builtin_amdgcn_readlane(wave_inclusive_sum(n), 63);
}

__global__ __launch_bounds__(kFinalThreads) void balance_final_kernel(BalanceArgs a, int parts)
{
    constexpr int kShares = kFinalThreads / kFinalColumns;  // of the rows
    constexpr int kWaves = kFinalThreads / kWave;
    __shared__ float sum_p[kShares][kFinalColumns];
    __shared__ int sum_c[kShares][kFinalColumns];
    __shared__ float total_w[kWaves];
    __shared__ int some_w[kWaves];
    __shared__ bool last;
    const int tid = threadIdx.x, wave = tid / kWave, lane = lane_id();
    const int col = tid % kFinalColumns, share = tid / kFinalColumns;
    const int shift = run_shift(a.T, a.E);
    const BalanceWs &ws = a.ws;
    // 64 experts of a sequence, and with more sequences than blocks others behind
    for (uint32_t item = blockIdx.x; item < (uint32_t)(a.S * parts); item += gridDim.x) {
        const int s = (int)(item / (uint32_t)parts), part = (int)item - s * parts;
        const int e = part * kFinalColumns + col;
        int lo, hi;
        bool bad = false;
        sequence(a.seq_off, s, a.T, lo, hi, bad);
        const int r0 = hi > lo ? lo >> shift : 0, r1 = hi > lo ? ((hi - 1) >> shift) + 1 : 0;
        float q = 0.0f;
        int c = 0;
        if (e < a.E) {
            // eight rows' loads at a time (rows behind the last are read as that
            // and not added)
            for (int r = r0 + share; r < r1; r += 8 * kShares) {
                float p[8];
                int n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const size_t at = (size_t)(min(r + i * kShares, r1 - 1) + s) * a.E + e;
                    p[i] = ws.probs[at];
                    n[i] = ws.counts[at];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = r + i * kShares < r1;
                    q += in ? p[i] : 0.0f;
                    c += in ? n[i] : 0;
                }
            }
        }
        sum_p[share][col] = q;
        sum_c[share][col] = c;
        const int n = wave == 0 ? tokens_seen(ws, s, r0, r1) : 0;
        __syncthreads();
        if (wave == 0) {
            q = 0.0f;
            c = 0;
            if (lane < kFinalColumns) {
#pragma unroll
                for (int i = 0; i < kShares; ++i) {
                    q += sum_p[i][lane];
                    c += sum_c[i][lane];
                }
                q = n ? q / (float)n : 0.0f;
                if (e < a.E) {
                    a.counts[(size_t)s * a.E + e] = c;
                    a.probs[(size_t)s * a.E + e] = q;
                }
            }
            const float dot = wave_sum((float)c * q);
            if (lane == 0) {
                if (part == 0)
                    a.num_tokens[s] = n;
                // -1 marks a sequence without tokens (the sums are not negative)
                __hip_atomic_store(&ws.dot[item],
                                   n ? dot * ((float)a.E / ((float)a.K * (float)n)) : -1.0f,
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        // the sums have left this XCD's L2 (device-coherent stores, waited for)
        // before the block counts itself; nothing else is handed over, so the
        // L2 need not be written back
        __builtin_amdgcn_s_waitcnt(0);
        last = __hip_atomic_fetch_add(ws.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               gridDim.x - 1;
    }
    __syncthreads();
    if (!last)
        return;
    float total = 0.0f;
    int some = 0;
    for (int q = tid; q < a.S; q += kFinalThreads) {
        float v = 0.0f;
        for (int p = 0; p < parts; ++p)
            v += __hip_atomic_load(&ws.dot[(size_t)q * parts + p], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        total += v >= 0.0f ? v : 0.0f;
        some += v >= 0.0f;
    }
    total = wave_sum(total);
    some = __builtin_amdgcn_readlane(wave_inclusive_sum(some), 63);
    if (lane == 0) {
        total_w[wave] = total;
        some_w[wave] = some;
    }
    __syncthreads();
    if (tid == 0) {
        total = 0.0f;
        some = 0;
        for (int w = 0; w < kWaves; ++w) {
            total += total_w[w];
            some += some_w[w];
        }
        a.num_tokens[a.S] = some;
        a.loss[0] = some ? total / (float)some : 0.0f;
    }
}

// ----------------------------------------------------------- gradient
//
// With c the weights' scale, d the gradient of topk_w, q the chosen scores'
// shares of their sum, and a_e = dloss E c_e / (K n^2 S') (S' sequences with
// tokens) the loss's gradient with respect to p_e:
//   normalised weights  dl_k += c q_k g_k (d_k - sum q d),
//   else                softmax dl_e += p_e (D_e - sum p D), D = c d at the
//                       chosen; sigmoid dl_k += c d_k s_k (1 - s_k),
//   loss                dl_e += p_e g_e (a_e - sum p a),
// where g is 1 for softmax and 1 - s for sigmoid. The entries' values reach
// their experts' lanes through LDS. One pass: 16384 tokens of 256 experts with
// both gradients (34 MB, 6.6 us at a copy's rate) 11.5 us at 800 vector
// instructions a wave behind two dependent loads (the offsets, then the
// sequence's counts); 8192 tokens of 64 experts 3.4 us.

// kPer: entries of a lane, i and (with more than 16 of them) i + 16.
template <int N, int kPer, bool SIGMOID>
__global__ __launch_bounds__(kWave) void route_backward_kernel(RouteBwdArgs a, bool wide,
                                                               bool wide_counts, bool wide_out,
                                                               bool normalize)
{
    __shared__ __align__(16) float at_expert[kTokens][kRow * N];
    const int row = lane_id() / kRow, i = row_lane();
    const int64_t t = (int64_t)blockIdx.x * kTokens + row;
    const bool live = t < a.T;
    const int64_t tc = min(t, (int64_t)a.T - 1);  // what is read in place of a token behind the last
    bool bad = false, bad_route = false;
    // loads in the order of their use: loads end in the order of their issue
    SequenceSearch search;
    if (a.counts)
        search.begin(a.seq_off, a.S);
    int64_t v[kPer];
    float d[kPer], l[N];
#pragma unroll
    for (int m = 0; m < kPer; ++m)
        v[m] = a.topk_idx[tc * a.K + min(i + m * kRow, a.K - 1)];
#pragma unroll
    for (int m = 0; m < kPer; ++m)
        d[m] = a.dtopk_w ? a.dtopk_w[tc * a.K + min(i + m * kRow, a.K - 1)] : 0.0f;
    load_row<N, float4, float>(a.logits + (size_t)tc * a.E, a.E, wide, l);
    const int s = a.counts ? search.find(a.seq_off, a.S, (int)min(t, (int64_t)a.T)) : -1;
    int cnt[N];  // (of experts that there are; the others have no share)
    float tokens = 0.0f, sequences = 1.0f, dloss = 0.0f;
    if (a.counts) {
        load_row<N, int4, int>(a.counts + (size_t)max(s, 0) * a.E, a.E, wide_counts, cnt);
        tokens = (float)a.num_tokens[max(s, 0)];
        sequences = (float)a.num_tokens[a.S];
        dloss = a.dloss[0];
    }
    int e[kPer];
    float lk[kPer];
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        v[m] = live && i + m * kRow < a.K ? v[m] : -1;
        bad_route |= v[m] < -1 || v[m] >= a.E;
        e[m] = v[m] >= 0 && v[m] < a.E ? (int)v[m] : -1;
        lk[m] = a.dtopk_w ? a.logits[(size_t)tc * a.E + max(e[m], 0)] : 0.0f;
    }
    clean_logits<N>(a.E, live, l, bad);
    const bool routed = row_ballot(e[0] >= 0 || (kPer > 1 && e[kPer - 1] >= 0)) != 0;
    bad = bad && routed;
    // the gradients with respect to shares (D) and logits (dl)
    float D[N], dl[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
        D[j] = dl[j] = 0.0f;
    bool shares = a.dtopk_w && !normalize && !SIGMOID;
    if (a.counts) {
        if (s >= 0 && routed) {
            const float c = tokens > 0.0f ? dloss * ((float)a.E / (float)a.K) /
                                                fmaxf(sequences, 1.0f) / (tokens * tokens)
                                          : 0.0f;
            // what all shares' gradients have in common is none of the logits',
            // as the shares sum to one: counts relative to an even spread, so
            // that nearly equal ones do not cancel in fp32
            const float even = tokens * (float)a.K / (float)a.E;
#pragma unroll
            for (int j = 0; j < N; ++j)
                D[j] = c * ((float)cnt[j] - even);
        }
        shares = true;
    }
    if (a.dtopk_w) {
        float g[kPer];
#pragma unroll
        for (int m = 0; m < kPer; ++m) {
            lk[m] = e[m] >= 0 && lk[m] < kInf ? lk[m] : -kInf;
            d[m] = e[m] >= 0 ? d[m] * a.scale : 0.0f;
        }
        if (normalize) {
            float n[kPer], slopes[kPer], sum = 0.0f, mean = 0.0f;
            const float ref = entry_ref<SIGMOID>(lk);
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
                n[m] = entry_score<SIGMOID>(lk[m], ref, slopes[m]);
                sum += n[m];
            }
            sum = row_sum(sum);
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
                n[m] = sum > 0.0f ? n[m] / sum : 0.0f;
                mean = __builtin_fmaf(n[m], d[m], mean);
            }
            mean = row_sum(mean);
#pragma unroll
            for (int m = 0; m < kPer; ++m)
                g[m] = n[m] * (d[m] - mean) * slopes[m];
        } else {
#pragma unroll
            for (int m = 0; m < kPer; ++m) {
                g[m] = d[m];
                if constexpr (SIGMOID) {
                    float slope;
                    g[m] *= entry_score<true>(lk[m], 0.0f, slope);
                    g[m] *= slope;
                }
            }
        }
        float *cell = at_expert[row];
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(&cell[expert(j)]) = float4{0.0f, 0.0f, 0.0f, 0.0f};
        wave_lds();
        // an expert named twice: one of the two finds the other's mark
#pragma unroll
        for (int m = 0; m < kPer; ++m)
            if (e[m] >= 0)
                cell[e[m]] = (float)(i + m * kRow);
        wave_lds();
        bool twice = false;
#pragma unroll
        for (int m = 0; m < kPer; ++m)
            twice |= e[m] >= 0 && cell[e[m]] != (float)(i + m * kRow);
        wave_lds();
        const bool any = __ballot(twice) != 0;
#pragma unroll
        for (int m = 0; m < kPer; ++m)
            if (e[m] >= 0)
                cell[e[m]] = any ? 0.0f : g[m];
        wave_lds();
        if (any) {  // one entry after the other
            for (int k = 0; k < a.K; ++k) {
                if (i == k % kRow) {
                    const int ek = k < kRow ? e[0] : e[kPer - 1];
                    if (ek >= 0)
                        cell[ek] += k < kRow ? g[0] : g[kPer - 1];
                }
                wave_lds();
            }
        }
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(&cell[expert(j)]);
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (!SIGMOID && !normalize)
                    D[j + q] += f[q];
                else
                    dl[j + q] += f[q];
            }
        }
    }
    if (shares) {
        float p[N], slopes[N], dot = 0.0f;
        shares_of<N, SIGMOID>(l, p, slopes);
#pragma unroll
        for (int j = 0; j < N; ++j)
            dot = __builtin_fmaf(p[j], D[j], dot);
        dot = row_sum(dot);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (SIGMOID)
                p[j] *= slopes[j];
            dl[j] = __builtin_fmaf(p[j], D[j] - dot, dl[j]);
        }
    }
    if (live) {
        float *out = a.dlogits + (size_t)t * a.E;
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const int c = expert(j);
            if (wide_out) {
                if (c < a.E)
                    *reinterpret_cast<float4 *>(out + c) =
                        float4{dl[j], dl[j + 1], dl[j + 2], dl[j + 3]};
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < a.E)
                        out[c + q] = dl[j + q];
            }
        }
    }
    if (bad || bad_route)
        flag_error(a.err, (bad ? EPX_DEV_BAD_LOGIT : 0) | (bad_route ? EPX_DEV_BAD_ROUTE : 0));
}

// Rows of E values that lanes take 16 bytes at a time.
bool wide_rows(const void *p, int E)
{
    return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

dim3 token_blocks(int T) { return dim3((unsigned)(((int64_t)T + kTokens - 1) / kTokens)); }

template <int N, int L>
hipError_t route_for(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    int shift = 0;  // lanes of a group
    while ((2 << shift) * a.G <= kRow)
        ++shift;
    const bool wide = wide_rows(a.logits, a.E), wide_bias = wide_rows(a.bias, a.E);
    if (sigmoid)
        hipLaunchKernelGGL((route_kernel<N, L, true>), token_blocks(a.T), dim3(kWave), 0, stream,
                           a, wide, wide_bias, shift, normalize);
    else
        hipLaunchKernelGGL((route_kernel<N, L, false>), token_blocks(a.T), dim3(kWave), 0, stream,
                           a, wide, wide_bias, shift, normalize);
    return hipGetLastError();
}

// Lists of 8 experts a lane, or of all the K there may be.
template <int N>
hipError_t route_for(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    return a.K <= 8 ? route_for<N, 8>(a, sigmoid, normalize, stream)
                    : route_for<N, EPX_MAX_TOPK>(a, sigmoid, normalize, stream);
}

template <int N, int TOKENS>
hipError_t balance_for(const BalanceArgs &a, bool sigmoid, hipStream_t stream)
{
    typedef Run<N, TOKENS> R;
    const int runs = a.T > 0 ? (int)(((int64_t)a.T + R::kTokensOfRun - 1) / R::kTokensOfRun) : 1;
    const dim3 grid((unsigned)runs), block(R::kThreads);
    const bool wide = wide_rows(a.logits, a.E);
    if (sigmoid)
        hipLaunchKernelGGL((balance_kernel<N, TOKENS, true>), grid, block, 0, stream, a, wide);
    else
        hipLaunchKernelGGL((balance_kernel<N, TOKENS, false>), grid, block, 0, stream, a, wide);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || runs == 1)
        return e;
    const int parts = (a.E + kFinalColumns - 1) / kFinalColumns;
    const int64_t items = (int64_t)a.S * parts, blocks = items < (1 << 16) ? items : 1 << 16;
    hipLaunchKernelGGL(balance_final_kernel, dim3((unsigned)blocks), dim3(kFinalThreads), 0,
                       stream, a, parts);
    return hipGetLastError();
}

template <int N, int kPer>
hipError_t backward_for(const RouteBwdArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    const bool wide = wide_rows(a.logits, a.E), wide_out = wide_rows(a.dlogits, a.E);
    const bool wide_counts = wide_rows(a.counts, a.E);
    if (sigmoid)
        hipLaunchKernelGGL((route_backward_kernel<N, kPer, true>), token_blocks(a.T), dim3(kWave),
                           0, stream, a, wide, wide_counts, wide_out, normalize);
    else
        hipLaunchKernelGGL((route_backward_kernel<N, kPer, false>), token_blocks(a.T), dim3(kWave),
                           0, stream, a, wide, wide_counts, wide_out, normalize);
    return hipGetLastError();
}

template <int N>
hipError_t backward_for(const RouteBwdArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    return a.K <= kRow ? backward_for<N, 1>(a, sigmoid, normalize, stream)
                       : backward_for<N, 2>(a, sigmoid, normalize, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (a.E <= 64)
        return route_for<4>(a, sigmoid, normalize, stream);
    if (a.E <= 128)
        return route_for<8>(a, sigmoid, normalize, stream);
    if (a.E <= 256)
        return route_for<16>(a, sigmoid, normalize, stream);
    return route_for<32>(a, sigmoid, normalize, stream);
}

size_t balance_workspace_bytes(int T, int E, int S)
{
    if (T <= run_tokens(T, E))  // one run: the first launch alone
        return 0;
    BalanceWs w;
    return balance_ws(nullptr, T, E, S, w);
}

hipError_t launch_balance(const BalanceArgs &args, bool sigmoid, hipStream_t stream)
{
    BalanceArgs a = args;
    balance_ws(static_cast<char *>(a.ws_base), a.T, a.E, a.S, a.ws);
    if (a.E <= 64)
        return balance_for<4, 64>(a, sigmoid, stream);
    if (a.E <= 128)
        return balance_for<8, 64>(a, sigmoid, stream);
    if (a.E <= 256)
        return run_tokens(a.T, a.E) == 64 ? balance_for<16, 64>(a, sigmoid, stream)
                                          : balance_for<16, 32>(a, sigmoid, stream);
    return balance_for<32, 32>(a, sigmoid, stream);
}

hipError_t launch_route_backward(const RouteBwdArgs &a, bool sigmoid, bool normalize,
                                 hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (a.E <= 64)
        return backward_for<4>(a, sigmoid, normalize, stream);
    if (a.E <= 128)
        return backward_for<8>(a, sigmoid, normalize, stream);
    if (a.E <= 256)
        return backward_for<16>(a, sigmoid, normalize, stream);
    return backward_for<32>(a, sigmoid, normalize, stream);
}

}  // namespace epx
