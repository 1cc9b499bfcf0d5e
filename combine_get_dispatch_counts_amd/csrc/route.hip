// route.hip -- the router's choice of experts, the balance loss with its
// per-expert counts, and the gradient of both with respect to the logits.
//
// Scores of a token's logits l (an expert is live unless its logit is -inf):
//   softmax  s_e = exp(l_e) / sum exp(l),   sigmoid  s_e = 1 / (1 + exp(-l_e)),
// and their shares of one p_e = s_e / sum s (softmax: p = s). A wave has one
// token; lane i holds the logits of experts V i .. V i + V - 1, so lanes
// ascend with the experts and the lowest lane that has a value also has the
// lowest expert that has it.
//
// The choice is that of the exact scores: fp32 scores decide wherever they
// are further apart than their error, and a token whose decision falls
// between nearer ones is done again in 64 bits.
#include "gate_device.h"

namespace epx {
namespace {

constexpr float kInf = __builtin_inff();

// A token's logits: -inf where the lane has no expert, and for a NaN or +inf,
// which sets bad.
template <int V>
__device__ __forceinline__ void load_logits(const float *row, int E, bool wide, float (&l)[V],
                                            bool &bad)
{
    const int e0 = lane_id() * V;
    if constexpr (V >= 4) {
        if (wide && e0 < E) {  // E % 4 == 0 and rows of whole 16-byte pieces
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float4 q = {-kInf, -kInf, -kInf, -kInf};
                if (e0 + j < E)
                    q = *reinterpret_cast<const float4 *>(row + e0 + j);
                l[j] = q.x;
                l[j + 1] = q.y;
                l[j + 2] = q.z;
                l[j + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                l[j] = e0 + j < E ? row[e0 + j] : -kInf;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            l[j] = e0 + j < E ? row[e0 + j] : -kInf;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (!(l[j] < kInf)) {
            bad = true;
            l[j] = -kInf;
        }
        l[j] += 0.0f;  // -0 orders as 0
    }
}

__device__ __forceinline__ float wave_max_float(float v) { return unordered(wave_max(ordered(v))); }

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

template <bool SIGMOID>
__device__ __forceinline__ float score_ref(float largest)
{
    return SIGMOID ? fminf(largest, 0.0f) : largest;
}

template <int V, bool SIGMOID>
__device__ __forceinline__ float raw_scores(const float (&l)[V], float (&s)[V])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j)
        m = fmaxf(m, l[j]);
    m = score_ref<SIGMOID>(wave_max_float(m));
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s[j] = raw_score<SIGMOID>(l[j], m);
        sum += s[j];
    }
    return wave_sum(sum);
}

// The two largest of a group's keys, by lanes that each look at every P-th of
// the group's experts; -inf keys do not count. Every lane of group g (lanes
// g P .. g P + P - 1) gets the sum; -inf for a group without experts.
template <typename F>
__device__ __forceinline__ F group_score(const F *key, int g, int size, int P, int G)
{
    F a = (F)-kInf, b = (F)-kInf;
    if (g < G)
        for (int i = lane_id() % P; i < size; i += P) {
            const F k = key[g * size + i];
            b = k > a ? a : k > b ? k : b;
            a = k > a ? k : a;
        }
    for (int d = 1; d < P; d <<= 1) {
        const F oa = __shfl_xor(a, d, kWave), ob = __shfl_xor(b, d, kWave);
        b = oa > a ? (a > ob ? a : ob) : (oa > b ? oa : b);
        a = oa > a ? oa : a;
    }
    return b > (F)-kInf ? a + b : a;
}

// Bit g of the result: group g is one of the `top` best (ties to the lower
// group). near: a kept and a dropped group's scores lie within tol of each
// other. 64 / P >= G; score is the same in the P lanes of a group.
template <typename F>
__device__ __forceinline__ uint64_t best_groups(F score, int P, int G, int top, F tol, bool &near)
{
    const int g = lane_id() / P;
    int rank = 0;
    for (int o = 0; o < G; ++o) {
        const F s = __shfl(score, o * P, kWave);
        rank += s > score || (s == score && o < g);
    }
    const bool kept = g < G && rank < top && score > (F)-kInf;
    uint64_t bits = 0, todo = uniform64(__ballot(kept && lane_id() % P == 0));
    while (todo) {
        bits |= 1ull << (__builtin_ctzll(todo) / P);
        todo &= todo - 1;
    }
    // the least kept and the best dropped score
    F lo = kept ? score : (F)kInf, hi = kept || g >= G ? (F)-kInf : score;
    for (int d = 1; d < kWave; d <<= 1) {
        const F ol = __shfl_xor(lo, d, kWave), oh = __shfl_xor(hi, d, kWave);
        lo = ol < lo ? ol : lo;
        hi = oh > hi ? oh : hi;
    }
    near = lo < (F)kInf && hi > (F)-kInf && lo - hi <= tol;
    return bits;
}

// The choice in 64 bits, one expert a round: lane r of the result has the
// r-th expert, or -1.
template <int V, bool SIGMOID>
__device__ __noinline__ int choose64(const RouteArgs &a, const float (&l)[V], double *lds, int P)
{
    const int lane = lane_id(), e0 = lane * V;
    double key[V];
    if constexpr (SIGMOID) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = l[j] > -kInf ? 1.0 / (1.0 + exp(-(double)l[j])) : -(double)kInf;
    } else {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j)
            m = fmaxf(m, l[j]);
        const double ref = (double)wave_max_float(m);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            key[j] = l[j] > -kInf ? exp((double)l[j] - ref) : 0.0;
            sum += key[j];
        }
        for (int d = 1; d < kWave; d <<= 1)
            sum += __shfl_xor(sum, d, kWave);
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = l[j] > -kInf ? key[j] / sum : -(double)kInf;
    }
    double order[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (a.bias && e0 + j < a.E) {
            const float b = a.bias[e0 + j];
            key[j] = b < kInf ? key[j] + (double)b : -(double)kInf;
        }
        // without a bias the logits are in the scores' order
        order[j] = a.bias ? key[j] : (double)l[j];
    }
    if (a.G > 1) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E)
                lds[e0 + j] = key[j];
        __builtin_amdgcn_wave_barrier();
        const double s = group_score<double>(lds, lane / P, a.group_size, P, a.G);
        bool near;
        const uint64_t kept = best_groups<double>(s, P, a.G, a.top_groups, 0.0, near);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E && !(kept >> div_by_magic(e0 + j, a.size_mul) & 1))
                order[j] = -(double)kInf;
    }
    int mine = -1;
    for (int r = 0; r < a.K; ++r) {
        double best = order[0];
        int e = e0;
#pragma unroll
        for (int j = 1; j < V; ++j)
            if (order[j] > best) {
                best = order[j];
                e = e0 + j;
            }
        for (int d = 1; d < kWave; d <<= 1) {
            const double ob = __shfl_xor(best, d, kWave);
            const int oe = __shfl_xor(e, d, kWave);
            if (ob > best || (ob == best && oe < e)) {
                best = ob;
                e = oe;
            }
        }
        if (!(best > -(double)kInf))
            break;
        if (lane == r)
            mine = e;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j == e)
                order[j] = -(double)kInf;
    }
    return mine;
}

constexpr int kTokens = 4;  // tokens (waves) of a block

// How far an fp32 key k may be from the exact one, for both of a pair: twice
// the error of the score -- sigmoid below 3e-7 (exp within 2^-22 of itself
// wherever s (1 - s) |l| matters), softmax below 2.3e-6 (the same, and the
// rounding of a sum over 512 experts) -- and of the bias's addition, 2^-24 of
// the key.
template <bool SIGMOID>
__device__ __forceinline__ float key_tol(float k)
{
    return (SIGMOID ? 0x1p-20f : 0x1p-17f) * (1.0f + fabsf(k));
}

template <int V, bool SIGMOID, bool NORM>
__global__ __launch_bounds__(kWave *kTokens) void route_kernel(RouteArgs a, bool wide, int P)
{
    __shared__ double lds_all[kTokens][V * kWave];
    __shared__ float key_all[kTokens][V * kWave];
    const int wave = threadIdx.x >> 6, lane = lane_id(), e0 = lane * V;
    const int64_t t = (int64_t)blockIdx.x * kTokens + wave;
    if (t >= a.T)
        return;
    double *lds = lds_all[wave];
    if (a.mask && !a.mask[t]) {
        if (lane < a.K) {
            a.topk_idx[t * a.K + lane] = -1;
            a.topk_w[t * a.K + lane] = 0.0f;
        }
        return;
    }
    float l[V];
    bool bad = false;
    load_logits<V>(a.logits + (size_t)t * a.E, a.E, wide, l, bad);
    // scores are needed whole by a bias, by groups and by weights that are
    // not normalised
    float s[V], sum = 1.0f;
    const bool scored = a.bias || a.G > 1 || (!NORM && !SIGMOID);
    if (scored) {
        if constexpr (SIGMOID) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                s[j] = raw_score<true>(l[j], 0.0f);
        } else {
            sum = raw_scores<V, false>(l, s);
#pragma unroll
            for (int j = 0; j < V; ++j)
                s[j] /= sum;
        }
    }
    float order[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        order[j] = l[j];
    if (a.bias) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (e0 + j < a.E) {
                const float b = a.bias[e0 + j];
                if (!(b < kInf))
                    bad = true;
                order[j] = l[j] > -kInf && b < kInf ? s[j] + b : -kInf;
            }
        }
    }
    if (__ballot(bad) && lane == 0)
        flag_error(a.err, EPX_DEV_BAD_LOGIT);
    bool near = false;
    if (a.G > 1) {
        float *key = key_all[wave];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E) {
                const float k = a.bias ? order[j] : l[j] > -kInf ? s[j] : -kInf;
                key[e0 + j] = k;
                top = fmaxf(top, k > -kInf ? fabsf(k) : 0.0f);
            }
        __builtin_amdgcn_wave_barrier();
        const float score = group_score<float>(key, lane / P, a.group_size, P, a.G);
        // a score is two keys, and rounded once more
        const float tol = 2.5f * key_tol<SIGMOID>(wave_max_float(top));
        const uint64_t kept = best_groups<float>(score, P, a.G, a.top_groups, tol, near);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E && !(kept >> div_by_magic(e0 + j, a.size_mul) & 1))
                order[j] = -kInf;
    }
    // each lane's experts in descending order (neighbours exchanged only where
    // strictly out of order, so equal values keep the experts' order)
    uint32_t k[V];
    int id[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        k[j] = order[j] > -kInf ? ordered(order[j]) : 0u;
        id[j] = e0 + j;
    }
#pragma unroll
    for (int p = 0; p < V; ++p)
#pragma unroll
        for (int j = p & 1; j + 1 < V; j += 2) {
            const bool swap = k[j + 1] > k[j];
            const uint32_t ka = swap ? k[j + 1] : k[j], kb = swap ? k[j] : k[j + 1];
            const int ia = swap ? id[j + 1] : id[j], ib = swap ? id[j] : id[j + 1];
            k[j] = ka; k[j + 1] = kb;
            id[j] = ia; id[j + 1] = ib;
        }
    // one expert a round, the best of the lanes' firsts; lane r keeps the r-th
    // (and, to see how near the first one left out is, the K-th)
    int mine = -1;
    uint32_t mine_key = 0;
    const int rounds = a.bias ? a.K + 1 : a.K;
    for (int r = 0; r < rounds; ++r) {
        const uint32_t best = wave_max(k[0]);
        if (best == 0)
            break;
        const int from = __builtin_ctzll(__ballot(k[0] == best));
        const int e = __builtin_amdgcn_readlane(id[0], from);
        if (lane == r) {
            mine = e;
            mine_key = best;
        }
        if (lane == from) {
#pragma unroll
            for (int j = 0; j + 1 < V; ++j) {
                k[j] = k[j + 1];
                id[j] = id[j + 1];
            }
            k[V - 1] = 0;
        }
    }
    // the chosen logits (lane e / V holds expert e)
    const auto pick = [&](int e) {
        float v = -kInf;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float o = __shfl(l[j], e / V, kWave);
            if (e % V == j)
                v = o;
        }
        return v;
    };
    float lk = pick(mine < 0 ? 0 : mine);
    if (a.bias) {
        // a neighbour in the order that is nearer than the keys' errors,
        // unless the two are alike in logit and bias
        const int oe = __shfl_down(mine, 1, kWave);
        const float ok = unordered((uint32_t)__shfl_down((int)mine_key, 1, kWave));
        const float ol = __shfl_down(lk, 1, kWave);
        if (lane < a.K && mine >= 0 && oe >= 0) {
            const float mk = unordered(mine_key);
            near |= mk - ok <= key_tol<SIGMOID>(mk) &&
                    !(lk == ol && a.bias[mine] == a.bias[oe]);
        }
    }
    if (__ballot(near)) {
        mine = choose64<V, SIGMOID>(a, l, lds, P);
        lk = pick(mine < 0 ? 0 : mine);
    }
    const bool have = lane < a.K && mine >= 0;
    lk = have ? lk : -kInf;
    float w;
    if constexpr (NORM) {
        const float ref = score_ref<SIGMOID>(wave_max_float(lk));
        const float n = raw_score<SIGMOID>(lk, ref);
        const float total = wave_sum(n);
        w = n / total;
    } else if constexpr (SIGMOID) {
        w = raw_score<true>(lk, 0.0f);
    } else {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j)
            m = fmaxf(m, l[j]);
        w = raw_score<false>(lk, wave_max_float(m)) / sum;
    }
    if (lane < a.K) {
        a.topk_idx[t * a.K + lane] = have ? mine : -1;
        a.topk_w[t * a.K + lane] = have ? a.scale * w : 0.0f;
    }
}

// -------------------------------------------------------------- balance loss
//
// Per sequence s of n tokens that have a route (an entry >= 0), with c_e
// entries for expert e and P_e the mean share of e over those tokens:
//   loss_s = E / (K n) sum_e c_e P_e,  loss = mean of loss_s over the
// sequences with n > 0 (0 without any).
//
// First launch: a block has a run of tokens and leaves one row of sums per
// sequence that meets the run, at row (run + sequence), which is a place of
// its own because the runs' and sequences' numbers ascend together. Second
// launch: a block per sequence adds its rows in order; the last block to end
// adds the losses. A batch of one run needs the first launch alone.

constexpr int kRun = 64;       // tokens of a run
constexpr int kRunWaves = 16;  // waves that share it
constexpr int kFinalThreads = 1024;

struct BalanceWs {
    unsigned int *done;  // blocks of the second launch that have ended
    float *seq_loss;     // [S]
    int *seen;           // [rows]
    int *counts;         // [rows, E]
    float *probs;        // [rows, E]
};

__host__ __device__ inline size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

__host__ __device__ inline int64_t balance_rows(int T, int S)
{
    return (T + kRun - 1) / kRun + (int64_t)S;
}

__host__ __device__ inline BalanceWs balance_ws(void *ws, int T, int E, int S)
{
    const int64_t rows = balance_rows(T, S);
    char *p = static_cast<char *>(ws);
    BalanceWs w;
    w.done = reinterpret_cast<unsigned int *>(p);
    p += 16;
    w.seq_loss = reinterpret_cast<float *>(p);
    p += up16((size_t)S * 4);
    w.seen = reinterpret_cast<int *>(p);
    p += up16((size_t)rows * 4);
    w.counts = reinterpret_cast<int *>(p);
    p += up16((size_t)rows * E * 4);
    w.probs = reinterpret_cast<float *>(p);
    return w;
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

// The first sequence that ends behind token t (S if none does).
__device__ __forceinline__ int first_sequence(const int32_t *off, int S, int t)
{
    if (!off)
        return 0;
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid + 1] > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ float block_sum(float v, float *meet)
{
    v = wave_sum(v);
    __syncthreads();
    if (lane_id() == 0)
        meet[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < (int)blockDim.x >> 6; ++w)
        v += meet[w];
    return v;
}

template <int V, bool SIGMOID>
__global__ __launch_bounds__(kWave *kRunWaves) void balance_kernel(BalanceArgs a, bool wide)
{
    __shared__ int cnt[V * kWave];
    __shared__ float part[kRunWaves][V * kWave];
    __shared__ int n_seen[kRunWaves];
    __shared__ float meet[kRunWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = lane_id(), e0 = lane * V;
    const BalanceWs ws = balance_ws(a.ws, a.T, a.E, a.S);
    const bool whole = gridDim.x == 1;  // the one run of the batch: outputs at once
    const int c0 = blockIdx.x * kRun, c1 = min(c0 + kRun, a.T);
    bool bad_logit = false, bad_off = false, bad_route = false;
    if (blockIdx.x == 0) {
        if (tid == 0)
            *ws.done = 0;
        // every sequence's offsets are looked at once
        for (int s = tid; s < a.S; s += blockDim.x) {
            int lo, hi;
            sequence(a.seq_off, s, a.T, lo, hi, bad_off);
        }
    }
    float total = 0.0f;
    int some = 0;
    for (int s = whole ? 0 : first_sequence(a.seq_off, a.S, c0); s < a.S; ++s) {
        int lo, hi;
        sequence(a.seq_off, s, a.T, lo, hi, bad_off);
        if (!whole && lo >= c1)
            break;
        lo = max(lo, c0);
        hi = min(hi, c1);
        for (int e = tid; e < V * kWave; e += blockDim.x)
            cnt[e] = 0;
        __syncthreads();
        float p[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            p[j] = 0.0f;
        int seen = 0;
        for (int t = lo + wave; t < hi; t += kRunWaves) {
            const int64_t e = lane < a.K ? a.topk_idx[(int64_t)t * a.K + lane] : -1;
            bad_route |= e < -1 || e >= a.E;
            const bool named = e >= 0 && e < a.E;
            if (named)
                atomicAdd(&cnt[(int)e], 1);
            if (!__ballot(named))
                continue;
            ++seen;
            float l[V], sc[V];
            load_logits<V>(a.logits + (size_t)t * a.E, a.E, wide, l, bad_logit);
            const float sum = raw_scores<V, SIGMOID>(l, sc);
            const float r = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                p[j] = __builtin_fmaf(sc[j], r, p[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            part[wave][e0 + j] = p[j];
        if (lane == 0)
            n_seen[wave] = seen;
        __syncthreads();
        int n = 0;
        for (int w = 0; w < kRunWaves; ++w)
            n += n_seen[w];
        float dot = 0.0f;
        for (int e = tid; e < a.E; e += blockDim.x) {
            float q = 0.0f;
            for (int w = 0; w < kRunWaves; ++w)
                q += part[w][e];
            if (whole) {
                q = n ? q / (float)n : 0.0f;
                a.counts[(size_t)s * a.E + e] = cnt[e];
                a.probs[(size_t)s * a.E + e] = q;
                dot = __builtin_fmaf((float)cnt[e], q, dot);
            } else {
                const size_t row = (size_t)(blockIdx.x + s) * a.E + e;
                ws.counts[row] = cnt[e];
                ws.probs[row] = q;
            }
        }
        if (whole) {
            dot = block_sum(dot, meet);
            if (n) {
                total += dot * ((float)a.E / ((float)a.K * (float)n));
                ++some;
            }
            if (tid == 0)
                a.num_tokens[s] = n;
        } else if (tid == 0) {
            ws.seen[blockIdx.x + s] = n;
        }
        __syncthreads();
    }
    if (whole && tid == 0) {
        a.num_tokens[a.S] = some;
        a.loss[0] = some ? total / (float)some : 0.0f;
    }
    if (bad_logit || bad_off || bad_route)
        flag_error(a.err, (bad_logit ? EPX_DEV_BAD_LOGIT : 0) | (bad_off ? EPX_DEV_OVERFLOW : 0) |
                              (bad_route ? EPX_DEV_BAD_ROUTE : 0));
}

__global__ __launch_bounds__(kFinalThreads) void balance_final_kernel(BalanceArgs a, int lanes)
{
    __shared__ float meet[kFinalThreads / kWave];
    __shared__ float part[kFinalThreads];
    __shared__ int part_n[kFinalThreads];
    __shared__ int n_shared;
    __shared__ bool last;
    const int s = blockIdx.x, tid = threadIdx.x;
    const BalanceWs ws = balance_ws(a.ws, a.T, a.E, a.S);
    int lo, hi;
    bool bad = false;
    sequence(a.seq_off, s, a.T, lo, hi, bad);
    const int r0 = hi > lo ? lo / kRun : 0, r1 = hi > lo ? (hi - 1) / kRun + 1 : 0;
    if (tid < kWave) {
        int n = 0;
        for (int r = r0 + tid; r < r1; r += kWave)
            n += ws.seen[r + s];
        n = __builtin_amdgcn_readlane(wave_inclusive_sum(n), 63);
        if (tid == 0)
            n_shared = n;
    }
    // `lanes` threads per share of the runs, an expert each
    const int share = tid / lanes, shares = kFinalThreads / lanes, e = tid % lanes;
    float q = 0.0f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int r = r0 + share; r < r1; r += shares) {
            q += ws.probs[(size_t)(r + s) * a.E + e];
            c += ws.counts[(size_t)(r + s) * a.E + e];
        }
    }
    part[tid] = q;
    part_n[tid] = c;
    __syncthreads();
    const int n = n_shared;
    float dot = 0.0f;
    if (share == 0 && e < a.E) {
        for (int i = 1; i < shares; ++i) {
            q += part[i * lanes + e];
            c += part_n[i * lanes + e];
        }
        q = n ? q / (float)n : 0.0f;
        a.counts[(size_t)s * a.E + e] = c;
        a.probs[(size_t)s * a.E + e] = q;
        dot = (float)c * q;
    }
    dot = block_sum(dot, meet);
    if (tid == 0) {
        a.num_tokens[s] = n;
        const float loss = n ? dot * ((float)a.E / ((float)a.K * (float)n)) : 0.0f;
        __hip_atomic_store(&ws.seq_loss[s], n ? loss : -1.0f, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(ws.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               gridDim.x - 1;
    }
    __syncthreads();
    if (!last)
        return;
    // losses are sums of products that are not negative: -1 marks an empty sequence
    float sum = 0.0f, some = 0.0f;
    for (int i = tid; i < a.S; i += kFinalThreads) {
        const float v = __hip_atomic_load(&ws.seq_loss[i], __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
        sum += v >= 0.0f ? v : 0.0f;
        some += v >= 0.0f ? 1.0f : 0.0f;
    }
    sum = block_sum(sum, meet);
    some = block_sum(some, meet);
    if (tid == 0) {
        a.num_tokens[a.S] = (int)some;
        a.loss[0] = some > 0.0f ? sum / some : 0.0f;
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
// where g is 1 for softmax and 1 - s for sigmoid.

template <bool SIGMOID>
__device__ __forceinline__ float slope(float l)
{
    if constexpr (!SIGMOID)
        return 1.0f;
    const float t = exp_fp32(-fabsf(l));
    return (l >= 0.0f ? t : 1.0f) / (1.0f + t);
}

template <int V, bool SIGMOID, bool NORM>
__global__ __launch_bounds__(kWave *kTokens) void route_backward_kernel(RouteBwdArgs a, bool wide)
{
    const int lane = lane_id(), e0 = lane * V;
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
    if (t >= a.T)
        return;
    bool bad = false;
    float l[V], dl[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
        dl[j] = 0.0f;
    int64_t e64 = lane < a.K ? a.topk_idx[t * a.K + lane] : -1;
    float d = lane < a.K && a.dtopk_w ? a.dtopk_w[t * a.K + lane] : 0.0f;
    const bool bad_route = e64 < -1 || e64 >= a.E;
    const int e = bad_route ? -1 : (int)e64;
    const uint64_t named = uniform64(__ballot(e >= 0));
    if (named) {
        load_logits<V>(a.logits + (size_t)t * a.E, a.E, wide, l, bad);
        int s = 0;
        bool inside = a.counts != nullptr;
        if (a.counts && a.seq_off) {
            s = first_sequence(a.seq_off, a.S, (int)t);
            inside = s < a.S && a.seq_off[s] <= t;
        }
        // the gradient with respect to the shares, where they are needed
        const bool shares = inside || (a.dtopk_w && !NORM && !SIGMOID);
        float D[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            D[j] = 0.0f;
        if (inside) {
            const float n = (float)a.num_tokens[s];
            const float c = n > 0.0f ? a.dloss[0] * ((float)a.E / (float)a.K) /
                                           (float)max(a.num_tokens[a.S], 1) / (n * n)
                                     : 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e0 + j < a.E)
                    D[j] = c * (float)a.counts[(size_t)s * a.E + e0 + j];
        }
        float g = 0.0f;  // of this lane's entry, added to its expert below
        if (a.dtopk_w) {
            float lk = -kInf;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float o = __shfl(l[j], (e < 0 ? 0 : e) / V, kWave);
                if (e >= 0 && e % V == j)
                    lk = o;
            }
            d = e >= 0 ? d * a.scale : 0.0f;
            if constexpr (NORM) {
                const float n = raw_score<SIGMOID>(lk, score_ref<SIGMOID>(wave_max_float(lk)));
                const float sum = wave_sum(n);
                const float q = sum > 0.0f ? n / sum : 0.0f;
                g = q * (d - wave_sum(q * d));
                if (SIGMOID && lk > -kInf)
                    g *= slope<true>(lk);
            } else if constexpr (SIGMOID) {
                g = lk > -kInf ? d * raw_score<true>(lk, 0.0f) * slope<true>(lk) : 0.0f;
            } else {
                g = d;
            }
            for (uint64_t todo = named; todo; todo &= todo - 1) {
                const int k = __builtin_ctzll(todo);
                const int ek = __builtin_amdgcn_readlane(e, k);
                const float gk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), k));
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (ek == e0 + j) {
                        if constexpr (!NORM && !SIGMOID)
                            D[j] += gk;
                        else
                            dl[j] += gk;
                    }
            }
        }
        if (shares) {
            float p[V], dot = 0.0f;
            const float sum = raw_scores<V, SIGMOID>(l, p);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                p[j] = sum > 0.0f ? p[j] / sum : 0.0f;
                dot = __builtin_fmaf(p[j], D[j], dot);
            }
            dot = wave_sum(dot);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = p[j] * (D[j] - dot);
                if (SIGMOID && l[j] > -kInf)
                    v *= slope<true>(l[j]);
                dl[j] += v;
            }
        }
    }
    float *out = a.dlogits + (size_t)t * a.E;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (e0 + j < a.E)
            out[e0 + j] = dl[j];
    if (bad || bad_route)
        flag_error(a.err, (bad ? EPX_DEV_BAD_LOGIT : 0) | (bad_route ? EPX_DEV_BAD_ROUTE : 0));
}

// Rows of logits that lanes read 16 bytes at a time.
bool wide_rows(const float *p, int E)
{
    return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <int V>
hipError_t route_for(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    int P = 1;  // lanes per group
    while (2 * P * a.G <= kWave)
        P *= 2;
    const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kWave * kTokens);
    const bool wide = wide_rows(a.logits, a.E);
    if (sigmoid && normalize)
        hipLaunchKernelGGL((route_kernel<V, true, true>), grid, block, 0, stream, a, wide, P);
    else if (sigmoid)
        hipLaunchKernelGGL((route_kernel<V, true, false>), grid, block, 0, stream, a, wide, P);
    else if (normalize)
        hipLaunchKernelGGL((route_kernel<V, false, true>), grid, block, 0, stream, a, wide, P);
    else
        hipLaunchKernelGGL((route_kernel<V, false, false>), grid, block, 0, stream, a, wide, P);
    return hipGetLastError();
}

template <int V>
hipError_t balance_for(const BalanceArgs &a, bool sigmoid, hipStream_t stream)
{
    const int runs = a.T > 0 ? (a.T + kRun - 1) / kRun : 1;
    const dim3 grid((unsigned)runs), block(kWave * kRunWaves);
    const bool wide = wide_rows(a.logits, a.E);
    if (sigmoid)
        hipLaunchKernelGGL((balance_kernel<V, true>), grid, block, 0, stream, a, wide);
    else
        hipLaunchKernelGGL((balance_kernel<V, false>), grid, block, 0, stream, a, wide);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || runs == 1)
        return e;
    hipLaunchKernelGGL(balance_final_kernel, dim3((unsigned)a.S), dim3(kFinalThreads), 0, stream,
                       a, V * kWave);
    return hipGetLastError();
}

template <int V>
hipError_t backward_for(const RouteBwdArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(kWave * kTokens);
    const bool wide = wide_rows(a.logits, a.E);
    if (sigmoid && normalize)
        hipLaunchKernelGGL((route_backward_kernel<V, true, true>), grid, block, 0, stream, a, wide);
    else if (sigmoid)
        hipLaunchKernelGGL((route_backward_kernel<V, true, false>), grid, block, 0, stream, a, wide);
    else if (normalize)
        hipLaunchKernelGGL((route_backward_kernel<V, false, true>), grid, block, 0, stream, a, wide);
    else
        hipLaunchKernelGGL((route_backward_kernel<V, false, false>), grid, block, 0, stream, a,
                           wide);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (a.E <= 64)
        return route_for<1>(a, sigmoid, normalize, stream);
    if (a.E <= 128)
        return route_for<2>(a, sigmoid, normalize, stream);
    if (a.E <= 256)
        return route_for<4>(a, sigmoid, normalize, stream);
    return route_for<8>(a, sigmoid, normalize, stream);
}

size_t balance_workspace_bytes(int T, int E, int S)
{
    const size_t rows = (size_t)balance_rows(T, S);
    return 16 + up16((size_t)S * 4) + up16(rows * 4) + 2 * up16(rows * E * 4);
}

hipError_t launch_balance(const BalanceArgs &a, bool sigmoid, hipStream_t stream)
{
    if (a.E <= 64)
        return balance_for<1>(a, sigmoid, stream);
    if (a.E <= 128)
        return balance_for<2>(a, sigmoid, stream);
    if (a.E <= 256)
        return balance_for<4>(a, sigmoid, stream);
    return balance_for<8>(a, sigmoid, stream);
}

hipError_t launch_route_backward(const RouteBwdArgs &a, bool sigmoid, bool normalize,
                                 hipStream_t stream)
{
    if (a.T == 0)
        return hipSuccess;
    if (a.E <= 64)
        return backward_for<1>(a, sigmoid, normalize, stream);
    if (a.E <= 128)
        return backward_for<2>(a, sigmoid, normalize, stream);
    if (a.E <= 256)
        return backward_for<4>(a, sigmoid, normalize, stream);
    return backward_for<8>(a, sigmoid, normalize, stream);
}

}  // namespace epx
