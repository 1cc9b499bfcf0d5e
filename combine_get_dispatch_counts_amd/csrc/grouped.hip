// grouped.hip -- products of the experts' rows with their weights, with the
// gated activation as an epilogue.
//
//   out[r, n] = sum_k x[r, k] w[e, n, k]                     (bf16)
//   out[r, n] = sum_b xs[r, b] ws[e, n/128, b] sum_{k in b} x[r, k] w[e, n, k]
//                                                            (FP8, b: 128 channels)
// summed in fp32. Gated: g and u are such products with the gate and the up
// rows of w, and out = g / (1 + exp(-g)) * u, in bf16 or again in FP8 with
// a scale per 128 columns.
//
// One persistent block of eight waves per compute unit walks over output
// tiles of BM rows x 256 weight rows (gated: 128 gate and the 128 up rows of
// the same columns), 128 bytes of every row per step. Both operands go from
// memory straight into LDS (buffer loads with the LDS as destination), STAGES
// steps deep, and the loads run ahead across tile boundaries, so the next
// tile's first steps arrive while this tile's epilogue runs. One barrier per
// step: it publishes the step's data and tells that the buffer to be loaded
// next has been read by every wave.
#include "experts_device.h"

namespace epx {
namespace {

// How a step's 128 bytes are multiplied.
//  kBf16: 64 channels, two 16x16x32 bf16 instructions per pair of operands.
//  kFp8:  128 channels, one 16x16x128 instruction; its sum of 8 products each
//         is aligned to the largest of them with about 16 bits (measured:
//         1.5e-5 of the result's spread), below the bf16 rounding of the result.
//  kWide: FP8 codes widened to bf16 (exact) in registers, four bf16
//         instructions, whose sums are full fp32: for the gated FP8 form,
//         whose scales are fp32 results.
enum Mode { kBf16, kFp8, kWide };

constexpr int kBN = 256;   // weight rows of a tile
constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kWM = 2, kWN = 4;          // wave grid: rows x weight rows
constexpr int kRow = 128;                // bytes of a row in LDS
constexpr uint32_t kNowhere = 0xFFFFFF00u;  // a buffer offset past every range: reads as zero

template <Mode MODE, bool GATED, int BM, int STAGES>
struct Shape {
    static constexpr bool kFp8Rows = MODE != kBf16;
    static constexpr int kEsize = kFp8Rows ? 1 : 2;
    static constexpr int kMF = BM / 16 / kWM;      // row fragments of a wave
    static constexpr int kALoads = BM / 8 / kWaves;  // 8-row loads of a wave and step
    static constexpr int kWLoads = kBN / 8 / kWaves;
    static constexpr int kLoads = kALoads + kWLoads;
    static constexpr int kStage = (BM + kBN) * kRow;
    static constexpr int kScale = kFp8Rows ? (BM + kWave) * 16 : 0;  // 4 steps of scales
    static constexpr int kAmax = GATED && kFp8Rows ? kWN * BM * 4 : 0;
    static constexpr int kTiles = 2064;            // running row tiles of the experts
    static constexpr int kRing = STAGES + 1;       // tiles loaded and not yet finished
    static constexpr int kLds = STAGES * (kStage + kScale) + kAmax + kTiles + 64 + kRing * 32;
};

// 64 lanes x 16 bytes from a buffer into LDS at lds (wave-uniform), lane l's
// bytes at lds + 16 l. Not tracked by the compiler: wait with wait_loads.
__device__ __forceinline__ void load_lds(uint32_t lds, i32x4 rsrc, uint32_t voff, uint32_t soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                     lds),
                 "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}

// Wait until at most N of the wave's memory operations are under way, and
// all its LDS reads have returned; then meet the other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void meet()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ i32x4 buffer_of(const void *p, int64_t bytes)
{
    const uint64_t b = uniform64((uint64_t)p);
    const int64_t n = bytes < (int64_t)kNowhere ? bytes : (int64_t)kNowhere;
    return i32x4{(int)(uint32_t)b, (int)((uint32_t)(b >> 32) & 0xFFFFu),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)n), 0x00020000};
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sixteen e4m3 codes as two bf16 operands of eight.
__device__ __forceinline__ void widen16(i32x4 c, i32x4 (&o)[2])
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
        o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(int, a);
        o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(int, b);
    }
}

template <int V>
struct Const {
    static constexpr int value = V;
};

// An output tile.
struct Tile {
    int64_t first;  // the expert's first row
    int e, m0, rows, n0;  // rows: of this tile
};

// A wave fragment of one step as it lies in LDS: 2 x 16 bytes per lane.
struct Raw {
    i32x4 lo, hi;
    static __device__ __forceinline__ Raw read(const char *row, int pos)
    {
        return Raw{*reinterpret_cast<const i32x4 *>(row + pos),
                   *reinterpret_cast<const i32x4 *>(row + (pos ^ 64))};
    }
};

// The same in the form the instructions take.
template <Mode MODE>
struct Frag {
    i32x4 v[MODE == kWide ? 4 : 2];
    Frag() = default;
    __device__ __forceinline__ explicit Frag(const Raw &r)
    {
        if constexpr (MODE == kWide) {
            i32x4 t[2];
            widen16(r.lo, t);
            v[0] = t[0], v[1] = t[1];
            widen16(r.hi, t);
            v[2] = t[0], v[3] = t[1];
        } else {
            v[0] = r.lo, v[1] = r.hi;
        }
    }
};

template <Mode MODE>
__device__ __forceinline__ f32x4 multiply(const Frag<MODE> &w, const Frag<MODE> &x, f32x4 c)
{
    if constexpr (MODE == kFp8) {
        return mfma_fp8(join(w.v[0], w.v[1]), join(x.v[0], x.v[1]), c);
    } else {
#pragma unroll
        for (int i = 0; i < (MODE == kWide ? 4 : 2); ++i)
            c = mfma_bf16(w.v[i], x.v[i], c);
        return c;
    }
}

template <Mode MODE, bool GATED, int BM, int STAGES>
__global__ __launch_bounds__(kThreads, 1) void grouped_kernel(GroupedArgs a)
{
    using S = Shape<MODE, GATED, BM, STAGES>;
    constexpr int MF = S::kMF;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    char *const scales = smem + STAGES * S::kStage;
    float *const row_amax = reinterpret_cast<float *>(scales + STAGES * S::kScale);
    int *const tiles_before = reinterpret_cast<int *>(scales + STAGES * S::kScale + S::kAmax);
    int *const wave_tiles = tiles_before + S::kTiles / 4;
    int *const ring = wave_tiles + 16;  // [kRing][8] tiles on their way

    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int g4 = lane >> 4, l16 = lane & 15;
    const int wm = wave & (kWM - 1), wn = wave / kWM;

    // row tiles of every expert, as running totals (L <= kThreads)
    static_assert(EPX_MAX_EXPERTS <= kThreads && EPX_MAX_EXPERTS * 4 + 4 <= S::kTiles, "");
    {
        int n = 0;
        if (tid < a.L) {
            int64_t first;
            bool bad;
            n = (expert_rows(a, tid, first, bad) + BM - 1) / BM;
            if (bad && blockIdx.x == 0)
                flag_error(a.err, EPX_DEV_OVERFLOW);
        }
        const int incl = wave_inclusive_sum(n);
        if (lane == 63)
            wave_tiles[wave] = incl;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < wave; ++w)
            before += wave_tiles[w];
        if (tid < a.L)
            tiles_before[tid + 1] = before + incl;
        if (tid == 0)
            tiles_before[0] = 0;
        __syncthreads();
    }
    constexpr int kCols = GATED ? kBN / 2 : kBN;  // output columns of a tile
    const int nt = (a.N + kCols - 1) / kCols;
    const int64_t total = (int64_t)uniform(tiles_before[a.L]) * nt;
    const int wrows = GATED ? 2 * a.N : a.N;
    const int kb_n = a.K >> 7, nb_n = (wrows + 127) >> 7;
    const int64_t kbytes = (int64_t)a.K * S::kEsize;
    const int steps = (int)((kbytes + kRow - 1) / kRow);
    const int tail = (int)(kbytes % kRow);  // bytes of a partial last step

    // The tile a block takes in its round r. Blocks are dealt to the eight
    // XCDs in turn: in a full round an XCD's blocks get consecutive tiles, so
    // tiles that share rows or weights share an L2.
    const int G = gridDim.x, b = blockIdx.x;
    const auto tile_number = [&](int64_t r) -> int64_t {
        const int64_t base = r * G;
        if (G % 8 == 0 && total - base >= G)
            return base + (b % 8) * (G / 8) + b / 8;
        return base + b;
    };
    // Tiles of an expert: four row tiles at a time, over all columns, row
    // tiles fastest: 32 neighbours read 4 row tiles and 8 weight tiles.
    const auto find_tile = [&](int64_t t, Tile &o) {
        const int mt = (int)(t / nt);
        int e = 0;
        for (int step = 512; step; step >>= 1)
            if (e + step < a.L && tiles_before[e + step] <= mt)
                e += step;
        e = uniform(e);
        const int before = uniform(tiles_before[e]);
        const int mts = uniform(tiles_before[e + 1]) - before;
        const int q = (int)(t - (int64_t)before * nt);
        const int group = q / (4 * nt), gm = min(4, mts - group * 4);
        const int r = q - group * 4 * nt;
        int64_t first;
        bool bad;
        const int rows = uniform(expert_rows(a, e, first, bad));
        o.first = (int64_t)uniform64((uint64_t)first);
        o.e = e;
        o.m0 = (group * 4 + r % gm) * BM;
        o.n0 = r / gm * kCols;
        o.rows = min(BM, rows - o.m0);
    };

    // ---- loads: the state of the tile being loaded
    Tile lt;
    int64_t lround = 0;
    int lstep = steps, lbuf = 0, lgroup = 0, ltile = 0;
    // buffers: rows, weights, row scales, weight scales
    i32x4 xr{0, 0, 0, 0x00020000}, wr = xr, sr = xr, vr = xr;
    uint32_t xoff[S::kALoads], woff[S::kWLoads], soff = 0;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    const int r8 = lane >> 3, c8 = lane & 7;  // a load's row and 16-byte piece
    const auto open_tile = [&](int64_t t) {
        find_tile(t, lt);
        if (tid == 0) {
            int *p = ring + ltile * 8;
            p[0] = (int)(uint32_t)lt.first;
            p[1] = (int)(lt.first >> 32);
            p[2] = lt.e;
            p[3] = lt.m0;
            p[4] = lt.rows;
            p[5] = lt.n0;
        }
        ltile = ltile + 1 == S::kRing ? 0 : ltile + 1;
        // base: the first row a load may name (regions: the expert's)
        const bool gather = !a.off && a.R_buf > 1;
        const int64_t base = lt.first + (gather ? 0 : lt.m0);
        xr = buffer_of(static_cast<const char *>(a.x) + base * kbytes, (a.n_rows - base) * kbytes);
#pragma unroll
        for (int i = 0; i < S::kALoads; ++i) {
            const int lr = (i * kWaves + wave) * 8 + r8;  // row of the tile
            const int m = min(lr, lt.rows - 1);
            const int row = gather ? expert_row(a, lt.e, lt.m0 + m) : m;
            xoff[i] = (uint32_t)((int64_t)row * kbytes) + (uint32_t)((c8 ^ (lr & 7)) * 16);
            if (lr >= ((lt.rows + 15) & ~15))
                xoff[i] = kNowhere;
        }
        const int64_t wbase = (int64_t)lt.e * wrows + lt.n0;
        wr = buffer_of(static_cast<const char *>(a.w) + wbase * kbytes,
                       ((int64_t)a.L * wrows - wbase) * kbytes);
#pragma unroll
        for (int i = 0; i < S::kWLoads; ++i) {
            const int lr = (wave * S::kWLoads + i) * 8 + r8;
            const int col = GATED ? lr & 127 : lr;
            const int n = min(col, a.N - 1 - lt.n0) + (GATED && lr >= 128 ? a.N : 0);
            const int key = (lr & 3) | (lr >> (GATED ? 1 : 2) & 4);
            woff[i] = (uint32_t)((int64_t)n * kbytes) + (uint32_t)((c8 ^ key) * 16);
        }
        if constexpr (S::kFp8Rows) {
            const int st = scale_stride(a.K);
            if (wave < BM / kWave) {
                sr = buffer_of(a.xs + base * st, (a.n_rows - base) * st * 4);
                const int m = min(wave * kWave + lane, lt.rows - 1);
                const int row = gather ? expert_row(a, lt.e, lt.m0 + m) : m;
                soff = (uint32_t)((int64_t)row * st * 4);
            } else if (wave == BM / kWave) {
                const int64_t sb = ((int64_t)lt.e * nb_n + (lt.n0 >> 7)) * kb_n;
                vr = buffer_of(a.ws + sb, ((int64_t)a.L * nb_n * kb_n - sb) * 4);
                // lane 1: the up rows' block, or the tile's second block
                const int blk = lane == 1 ? (GATED ? a.N >> 7 : 1) : 0;
                soff = (uint32_t)(blk * kb_n * 4);
            }
        }
        lstep = 0;
    };
    // The next step's loads: begin_load, then load_piece(0 .. kLoads-1), then
    // end_load. Behind the last tile they go on from nowhere (zeros into LDS
    // that is not read again), so every step issues the same number.
    uint32_t lat = 0, lkk = 0;
    const auto begin_load = [&]() {
        if (lstep == steps) {
            const int64_t t = tile_number(lround++);
            if (t < total) {
                open_tile(t);
            } else {
                xr[2] = wr[2] = sr[2] = vr[2] = 0;  // empty buffers
                lstep = 0;
            }
        }
        if constexpr (S::kFp8Rows) {
            if ((lstep & 3) == 0) {
                const uint32_t at = lds0 + STAGES * S::kStage + lgroup * S::kScale;
                if (wave < BM / kWave)
                    load_lds(uniform(at + wave * 1024), sr, soff, lstep * 4);
                else if (wave == BM / kWave)
                    load_lds(uniform(at + BM * 16), vr, soff, lstep * 4);
                lgroup = lgroup + 1 == STAGES ? 0 : lgroup + 1;
            }
        } else if (tail && lstep == steps - 1) {  // a partial last step of its tile
#pragma unroll
            for (int i = 0; i < S::kALoads; ++i)
                if ((c8 ^ r8) * 16 >= tail)
                    xoff[i] = kNowhere;
#pragma unroll
            for (int i = 0; i < S::kWLoads; ++i) {
                const int lr = (wave * S::kWLoads + i) * 8 + r8;
                if ((c8 ^ ((lr & 3) | (lr >> (GATED ? 1 : 2) & 4))) * 16 >= tail)
                    woff[i] = kNowhere;
            }
        }
        lat = lds0 + lbuf * S::kStage + wave * 1024;
        lkk = (uint32_t)lstep * kRow;
    };
    const auto load_piece = [&](int i) {
        if (i < S::kALoads)
            load_lds(uniform(lat + i * kWaves * 1024), xr, xoff[i], lkk);
        else
            load_lds(uniform(lat + BM * kRow + wave * (S::kWLoads - 1) * 1024 +
                             (i - S::kALoads) * 1024),
                     wr, woff[i - S::kALoads], lkk);
    };
    const auto end_load = [&]() {
        lbuf = lbuf + 1 == STAGES ? 0 : lbuf + 1;
        ++lstep;
    };

    // ---- products
    const int pos = (g4 ^ (l16 & 7)) * 16;  // the lane's first piece of its row, swizzled
    // weight rows of a wave, arranged so that a lane's results over its
    // fragments j are consecutive columns: fragment row l16 is column
    // 16 (l16 / 4) + 4 j + l16 % 4 (gated: 8 (l16 / 4) + 4 j + l16 % 4)
    const int wrow = GATED ? wn * 32 + (l16 >> 2) * 8 + (l16 & 3) : wn * 64 + (l16 >> 2) * 16 + (l16 & 3);
    const char *const xlane = smem + (wm * 16 + l16) * kRow;
    const char *const wlane = smem + (BM + wrow) * kRow;

    f32x4 acc[4][MF];
    Tile o;
    int64_t round = 0;
    int mf = 0, s = 0, buf = 0, group = 0, tile = 0;
    if (tile_number(0) >= total)
        return;
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) {
        begin_load();
#pragma unroll
        for (int p = 0; p < S::kLoads; ++p)
            load_piece(p);
        end_load();
    }
    for (;;) {
        // the step to multiply has arrived when only the loads of the steps
        // after it are under way
        wait_and_meet<(STAGES - 2) * S::kLoads>();
        if (s == 0) {
            const int *p = ring + tile * 8;
            tile = tile + 1 == S::kRing ? 0 : tile + 1;
            o.first = (int64_t)((uint64_t)(uint32_t)uniform(p[0]) |
                                (uint64_t)(uint32_t)uniform(p[1]) << 32);
            o.e = uniform(p[2]), o.m0 = uniform(p[3]), o.rows = uniform(p[4]), o.n0 = uniform(p[5]);
            mf = (((o.rows + 15) >> 4) - wm + kWM - 1) / kWM;  // fragments of this wave
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < MF; ++i)
                    acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const char *const sc = scales + group * S::kScale + (s & 3) * 4;
        const char *const xb = xlane + buf * S::kStage, *const wb = wlane + buf * S::kStage;
        Raw x = Raw::read(xb, pos);
        Frag<MODE> w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = Frag<MODE>(Raw::read(wb + (GATED ? (j >> 1) * 128 + (j & 1) * 4 : j * 4) * kRow,
                                        pos));
        float sw[2] = {0.0f, 0.0f};
        if constexpr (S::kFp8Rows) {
            sw[0] = *reinterpret_cast<const float *>(sc + (BM + (GATED ? 0 : wn >> 1)) * 16);
            if (GATED)
                sw[1] = *reinterpret_cast<const float *>(sc + (BM + 1) * 16);
        }
        begin_load();
        // The wave's row fragments in two halves, the second left out where
        // the tile has no rows for it; the next step's loads go between the
        // first half's products. Fragment i + 1 is read while the matrix unit
        // works on fragment i; FP8 sums are scaled and added kLag products
        // after their own.
        const auto half = [&](auto from, auto to, auto loads) {
            constexpr int I0 = decltype(from)::value, I1 = decltype(to)::value;
            constexpr int kPer = (decltype(loads)::value + I1 - I0 - 1) / (I1 - I0);
            float sx[I1 - I0];
            if constexpr (S::kFp8Rows) {
#pragma unroll
                for (int i = I0; i < I1; ++i)
                    sx[i - I0] =
                        *reinterpret_cast<const float *>(sc + ((i * kWM + wm) * 16 + l16) * 16);
            }
            if (I0 > 0)
                x = Raw::read(xb + I0 * kWM * 16 * kRow, pos);
            constexpr int kLag = 3;
            f32x4 d[kLag + 1];
            const auto add = [&](int q) {
                const int i = q >> 2, j = q & 3;
                const float sc_ = sx[i] * sw[GATED && j >= 2];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[j][I0 + i][c] =
                        __builtin_fmaf(sc_, d[q % (kLag + 1)][c], acc[j][I0 + i][c]);
                // keeps the sums here: moved behind the branch between the
                // halves, they would hold their operands until then
                asm volatile("" : "+v"(acc[j][I0 + i]));
            };
#pragma unroll
            for (int i = I0; i < I1; ++i) {
                Raw next = x;
                if (i + 1 < I1)
                    next = Raw::read(xb + (i + 1) * kWM * 16 * kRow, pos);
                const Frag<MODE> xf(x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (S::kFp8Rows) {
                        const int q = (i - I0) * 4 + j;
                        d[q % (kLag + 1)] = multiply<MODE>(w[j], xf, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                        if (q >= kLag)
                            add(q - kLag);
                        __builtin_amdgcn_sched_barrier(0);
                    } else {
                        acc[j][i] = multiply<MODE>(w[j], xf, acc[j][i]);
                    }
                }
#pragma unroll
                for (int p = (i - I0) * kPer; p < (i - I0 + 1) * kPer; ++p)
                    if (p < decltype(loads)::value)
                        load_piece(p);
                x = next;
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (S::kFp8Rows) {
#pragma unroll
                for (int q = (I1 - I0) * 4 - kLag; q < (I1 - I0) * 4; ++q)
                    add(q);
            }
        };
        half(Const<0>{}, Const<(MF + 1) / 2>{}, Const<S::kLoads>{});
        end_load();
        if constexpr (MF > 1) {
            if (mf > (MF + 1) / 2)
                half(Const<(MF + 1) / 2>{}, Const<MF>{}, Const<0>{});
        }
        buf = buf + 1 == STAGES ? 0 : buf + 1;
        if ((s & 3) == 3 || s + 1 == steps)
            group = group + 1 == STAGES ? 0 : group + 1;
        if (++s < steps)
            continue;
        s = 0;

        // ---- epilogue: lane l holds consecutive columns of rows (2 i + wm) * 16 + l16
        const auto out_row = [&](int m) -> int64_t {
            return o.first + expert_row(a, o.e, o.m0 + m);
        };
        if constexpr (!GATED) {
            const int n = o.n0 + wn * 64 + g4 * 16;
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const int m = (i * kWM + wm) * 16 + l16;
                if (i < mf && m < o.rows) {
                    uint16_t *p = static_cast<uint16_t *>(a.out) + out_row(m) * a.N + n;
                    u32x4 v[2];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            v[j >> 1][2 * (j & 1) + c] =
                                f32_to_bf16(acc[j][i][2 * c]) |
                                (f32_to_bf16(acc[j][i][2 * c + 1]) << 16);
                    if (n < a.N)  // N is a multiple of 8
                        *reinterpret_cast<u32x4 *>(p) = v[0];
                    if (n + 8 < a.N)
                        *reinterpret_cast<u32x4 *>(p + 8) = v[1];
                }
            }
        } else {
            const int n = o.n0 + wn * 32 + g4 * 8;
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[j][i][c] = silu_mul(acc[j][i][c], acc[2 + j][i][c]);
            if constexpr (!S::kFp8Rows) {
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int m = (i * kWM + wm) * 16 + l16;
                    if (i < mf && m < o.rows && n < a.N) {
                        u32x4 v;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                v[2 * j + c] = f32_to_bf16(acc[j][i][2 * c]) |
                                               (f32_to_bf16(acc[j][i][2 * c + 1]) << 16);
                        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) +
                                                   out_row(m) * a.N + n) = v;
                    }
                }
            } else {
                // a row's 128 columns are spread over the four waves wn
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    float v = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            v = amax_of(v, acc[j][i][c]);
                    v = amax_of(v, __shfl_xor(v, 16, kWave));
                    v = amax_of(v, __shfl_xor(v, 32, kWave));
                    if (g4 == 0)
                        row_amax[wn * BM + (i * kWM + wm) * 16 + l16] = v;
                }
                meet();
                const int st = scale_stride(a.N);
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int m = (i * kWM + wm) * 16 + l16;
                    if (i < mf && m < o.rows) {
                        float v = row_amax[m];
#pragma unroll
                        for (int w = 1; w < kWN; ++w)
                            v = amax_of(v, row_amax[w * BM + m]);
                        const float s = group_scale(v);
                        uint32_t q[2] = {0, 0};
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                q[j] |= e4m3_of_quotient(acc[j][i][c], s) << (8 * c);
                        const int64_t row = out_row(m);
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + row * a.N + n) =
                            uint2{q[0], q[1]};
                        float *os = a.out_s + row * st;
                        if (wn == 0 && g4 == 0)
                            os[o.n0 >> 7] = s;
                        if (o.n0 + 128 >= a.N)  // the last columns' tile clears the padding too
                            for (int p = (a.N >> 7) + wn * 4 + g4; p < st; p += 16)
                                os[p] = 0.0f;
                    }
                }
                // (the next write of row_amax is behind the next tile's barriers)
            }
        }
        if (tile_number(++round) >= total)
            break;
    }
    // no load may reach LDS after the block has given it back
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <Mode MODE, bool GATED, int BM, int STAGES>
hipError_t launch(const GroupedArgs &a, hipStream_t stream)
{
    using S = Shape<MODE, GATED, BM, STAGES>;
    static_assert(S::kLds <= 160 * 1024, "");
    const auto k = grouped_kernel<MODE, GATED, BM, STAGES>;
    const int64_t cols = GATED ? kBN / 2 : kBN;
    const int64_t most = (a.n_rows / BM + a.L) * ((a.N + cols - 1) / cols);  // tiles there can be
    const int64_t blocks = most < a.cus ? most : a.cus;
    hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(kThreads), S::kLds, stream, a);
    return hipGetLastError();
}

template <Mode MODE, bool GATED>
hipError_t pick(const GroupedArgs &a, hipStream_t stream)
{
    if constexpr (MODE != kWide) {
        if (a.off && a.n_rows > 128ll * a.L)
            return launch<MODE, GATED, 256, 2>(a, stream);
    }
    return launch<MODE, GATED, 128, 3>(a, stream);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs &a, bool fp8, bool gated, hipStream_t stream)
{
    if (a.n_rows == 0)
        return hipSuccess;
    if (fp8)
        return gated ? pick<kWide, true>(a, stream) : pick<kFp8, false>(a, stream);
    return gated ? pick<kBf16, true>(a, stream) : pick<kBf16, false>(a, stream);
}

}  // namespace epx
