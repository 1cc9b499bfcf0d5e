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
// memory straight into LDS (buffer loads with the LDS as destination), one or
// two steps ahead and across tile boundaries, so the next tile's first steps
// arrive while this tile's epilogue runs. One barrier per
// step: it publishes the step's data and tells that the buffer to be loaded
// next has been read by every wave.
//
// Bound by: with few rows the weights from HBM (256 regions of 4 rows, 4096 x
// 7168 codes, FP8 gated: 1231 us, 6.0 TB/s). With many, the products and the
// loads beside them (49 152 rows of 64 experts, 4096 x 2048 weights, FP8: 490
// us, 1.68 PFLOP/s; 29 811 rows of 8 experts, 7168 x 2048, bf16: 783 us, 1.12
// PFLOP/s): without loads behind the first steps the same launches take 361
// and 567 us, the loads alone 324 and 552, and both with all operands in the
// L2 434 and 717. The matrix unit is busy for 40% and 54% of the time: every
// step begins with fragment reads behind its barrier, and at this tile size
// 160 KB of LDS leave room for one step of loads ahead, too little for the
// L2's misses.
#include "experts_device.h"

namespace epx {
namespace {

// How a step's 128 bytes are multiplied.
//  kBf16: 64 channels, two 16x16x32 bf16 instructions per pair of operands.
//  kFp8:  128 channels, one 16x16x128 instruction. It cuts each product towards
//         zero to a multiple of 2^(m - 13), m the largest exponent sum of the
//         products of eight neighbouring channels (measured; the tests hold it
//         to that), and adds in fp32: a result is off by about 1e-5 of its
//         products' magnitudes, 7 * 2^-13 of each eight's largest at most.
//         Taken for the twice as fast instruction: the e4m3 operands have
//         been rounded by up to 2^-4 each, and the result is rounded to bf16.
//  kWide: FP8 codes widened to bf16 (exact) in registers, four bf16
//         instructions, whose sums are full fp32: for the gated FP8 form,
//         whose scales are fp32 results (with kFp8 they were off by 1.2e-5;
//         256 experts of 128 rows took 1540 us with it, and take 2330).
enum Mode { kBf16, kFp8, kWide };

constexpr int kBN = 256;   // weight rows of a tile
constexpr int kWaves = 8, kThreads = kWaves * kWave;
constexpr int kWM = 2, kWN = 4;          // wave grid: rows x weight rows
constexpr int kRow = 128;                // bytes of a row in LDS
constexpr int kMostTiles = 0x7FFF0000;   // of a call: tile numbers go a few grids past them
constexpr uint32_t kNowhere = 0xFFFFFF00u;  // a buffer offset past every range: reads as zero

template <Mode MODE, bool GATED, int BM, int XBUF, int WBUF>
struct Shape {
    static constexpr bool kFp8Rows = MODE != kBf16;
    static constexpr int kEsize = kFp8Rows ? 1 : 2;
    static constexpr int kMF = BM / 16 / kWM;      // row fragments of a wave
    // 8-row loads of a wave and step (the last one not of every wave, if BM
    // is no multiple of 64)
    static constexpr int kALoads = (BM + 63) / 64;
    static constexpr int kWLoads = kBN / 8 / kWaves;
    static constexpr int kLoads = kALoads + kWLoads;
    static constexpr int kXStep = BM * kRow, kWStep = kBN * kRow;  // bytes of a step
    // Loads run XA and WA steps ahead; a step is there when only these loads,
    // issued after its own, are under way (an iteration issues rows, then weights).
    static constexpr int XA = XBUF - 1, WA = WBUF - 1;
    static_assert(WA >= XA && XA >= 1, "");
    static constexpr int kUnderWay = (XA - 1) * (BM / 64 + kWLoads) + (WA > XA ? kWLoads : 0);
    static constexpr int kScaleRows = (BM + kWave - 1) / kWave * kWave;
    static constexpr int kScale = kFp8Rows ? (kScaleRows + kWave) * 16 : 0;  // 4 steps of scales
    static constexpr int kAmax = GATED && kFp8Rows ? kWN * BM * 4 : 0;
    static constexpr int kTiles = 2064;            // running row tiles of the experts
    static constexpr int kRing = WBUF + 1;         // tiles opened and not yet finished
    static constexpr int kScaleAt = XBUF * kXStep + WBUF * kWStep;
    static constexpr int kAmaxAt = kScaleAt + XBUF * kScale;
    static constexpr int kTilesAt = kAmaxAt + kAmax;
    static constexpr int kRingAt = kTilesAt + kTiles + 64;
    static constexpr int kLds = kRingAt + kRing * 32;
};

// 64 lanes x 16 bytes from a buffer into LDS at lds (wave-uniform), lane l's
// bytes at lds + 16 l. Not tracked by the compiler: wait with wait_and_meet.
// A vector memory instruction may read a scalar register no earlier than five
// wait states after a vector instruction wrote it (v_readfirstlane for the
// descriptor, v_readlane where one was spilled), and the compiler does not
// look inside the block: the block's first two instructions are those five,
// and the one that m0 needs.
__device__ __forceinline__ void load_lds(uint32_t lds, i32x4 rsrc, uint32_t voff, uint32_t soff)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rsrc[i] = __builtin_amdgcn_readfirstlane(rsrc[i]);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                     lds),
                 "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
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

// Eight results; STREAM: past the L2, which would write them back at the
// launch's end.
template <bool STREAM>
__device__ __forceinline__ void store_result(uint16_t *p, u32x4 v)
{
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
    else
        *reinterpret_cast<u32x4 *>(p) = v;
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
    static constexpr int kProducts = MODE == kFp8 ? 1 : MODE == kBf16 ? 2 : 4;
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

// The k-th of a step's kProducts instructions for a pair of fragments.
template <Mode MODE>
__device__ __forceinline__ f32x4 multiply(const Frag<MODE> &w, const Frag<MODE> &x, int k, f32x4 c)
{
    if constexpr (MODE == kFp8)
        return mfma_fp8(join(w.v[0], w.v[1]), join(x.v[0], x.v[1]), c);
    else
        return mfma_bf16(w.v[k], x.v[k], c);
}

template <Mode MODE, bool GATED, int BM, int XBUF, int WBUF>
__global__ __launch_bounds__(kThreads, 1) void grouped_kernel(GroupedArgs a)
{
    using S = Shape<MODE, GATED, BM, XBUF, WBUF>;
    constexpr int MF = S::kMF, kScaleWaves = (BM + kWave - 1) / kWave;
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    float *const row_amax = reinterpret_cast<float *>(smem + S::kAmaxAt);
    int *const tiles_before = reinterpret_cast<int *>(smem + S::kTilesAt);
    int *const wave_tiles = tiles_before + S::kTiles / 4;
    int *const ring = reinterpret_cast<int *>(smem + S::kRingAt);  // [kRing][8] opened tiles

    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int g4 = lane >> 4, l16 = lane & 15;
    const int wm = wave & (kWM - 1), wn = wave / kWM;

    // row tiles of every expert, as running totals (L <= kThreads)
    static_assert(EPX_MAX_EXPERTS <= kThreads && EPX_MAX_EXPERTS * 4 + 4 <= S::kTiles, "");
    const bool gather = !a.off && a.R_buf > 1;  // an expert's rows lie in several regions
    {
        int n = 0;
        bool bad = false;
        if (gather) {
            if (tid < a.L)
                tiles_before[tid] = 0;
            __syncthreads();
            for (int i = tid; i < a.L * a.R_buf; i += kThreads)
                atomicAdd(&tiles_before[i / a.R_buf], region_rows(a, i, bad));
            __syncthreads();
            n = tid < a.L ? tiles_before[tid] : 0;
        } else if (tid < a.L) {
            int64_t first;
            n = expert_rows(a, tid, first, bad);
        }
        if (bad && blockIdx.x == 0)
            flag_error(a.err, EPX_DEV_OVERFLOW);
        n = n / BM + (n % BM != 0);
        const int incl = wave_inclusive_sum(n);
        if (lane == 63)
            wave_tiles[wave] = incl;
        __syncthreads();
        // offsets that overlap can name more tiles than 32 bits hold: such
        // totals stop at kMost (a wave's own total stays below 2^30 + 64)
        constexpr int kMost = 0x38000000;
        int before = 0;
        for (int w = 0; w < wave; ++w)
            before = min(before + wave_tiles[w], kMost);
        if (tid < a.L)
            tiles_before[tid + 1] = min(before + incl, kMost);
        if (tid == 0)
            tiles_before[0] = 0;
        __syncthreads();
    }
    constexpr int kCols = GATED ? kBN / 2 : kBN;  // output columns of a tile
    const int nt = (a.N + kCols - 1) / kCols;
    // (what valid offsets can reach is checked by the launcher)
    const int total = uniform((int)min((int64_t)tiles_before[a.L] * nt, (int64_t)kMostTiles));
    const int wrows = GATED ? 2 * a.N : a.N;
    const int kb_n = a.K >> 7, nb_n = (wrows + 127) >> 7;
    const int64_t kbytes = (int64_t)a.K * S::kEsize;
    const int steps = (int)((kbytes + kRow - 1) / kRow);
    const int tail = (int)(kbytes % kRow);  // bytes of a partial last step

    // The tile a block takes in its round r. Blocks are dealt to the eight
    // XCDs in turn: in a full round an XCD's blocks get consecutive tiles, so
    // tiles that share rows or weights share an L2.
    const int G = gridDim.x, b = blockIdx.x;
    const auto tile_number = [&](int r) {
        const int base = r * G;
        if (G % 8 == 0 && total - base >= G)
            return base + (b % 8) * (G / 8) + b / 8;
        return base + b;
    };
    // Tiles of an expert: four row tiles at a time, over all columns, row
    // tiles fastest: 32 neighbours read 4 row tiles and 8 weight tiles.
    const auto find_tile = [&](int t, Tile &o) {
        const int mt = t / nt;
        int e = -1;  // the last expert whose tiles begin at or before mt
        for (int e0 = 0; e0 < a.L; e0 += kWave)
            e += __builtin_popcountll(
                __ballot(e0 + lane < a.L && tiles_before[min(e0 + lane, a.L)] <= mt));
        e = uniform(e);
        const int before = uniform(tiles_before[e]);
        const int mts = uniform(tiles_before[e + 1]) - before;
        const int q = t - before * nt;
        const int group = q / (4 * nt), gm = min(4, mts - group * 4);
        const int r = q - group * 4 * nt;
        int64_t first = (int64_t)e * a.R_buf * a.cap;
        bool bad = false;
        int rows;
        if (gather) {
            Regions g;
            g.load(a, e);
            rows = g.rows();
        } else {
            rows = uniform(expert_rows(a, e, first, bad));
        }
        o.first = (int64_t)uniform64((uint64_t)first);
        o.e = e;
        o.m0 = (group * 4 + r % gm) * BM;
        o.n0 = r / gm * kCols;
        o.rows = min(BM, rows - o.m0);
    };

    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    const int r8 = lane >> 3, c8 = lane & 7;  // a load's row and 16-byte piece
    // Behind the last tile the loads go on from empty buffers (zeros into LDS
    // that is not read again), so every step issues the same number.

    // ---- weight loads: they open the tiles
    Tile wt{};
    int wround = 0;
    int wstep = steps, wbuf = 0, wtile = 0;
    i32x4 wr{0, 0, 0, 0x00020000};
    uint32_t woff[S::kWLoads] = {};
    const auto wkey = [&](int lr) { return (lr & 3) | (lr >> 1 & 4); };
    const auto begin_weights = [&]() {
        if (wstep == steps) {
            wstep = 0;
            const int t = tile_number(wround++);
            if (t < total) {
                find_tile(t, wt);
                const int64_t base = (int64_t)wt.e * wrows + wt.n0;
                wr = buffer_of(static_cast<const char *>(a.w) + base * kbytes,
                               ((int64_t)a.L * wrows - base) * kbytes);
#pragma unroll
                for (int i = 0; i < S::kWLoads; ++i) {
                    const int lr = (wave * S::kWLoads + i) * 8 + r8;
                    const int col = GATED ? lr & 127 : lr;
                    const int n = min(col, a.N - 1 - wt.n0) + (GATED && lr >= 128 ? a.N : 0);
                    woff[i] = (uint32_t)((int64_t)n * kbytes) + (uint32_t)((c8 ^ wkey(lr)) * 16);
                }
            } else {
                wt.rows = 0;
                wr[2] = 0;
            }
            if (tid == 0) {
                int *p = ring + wtile * 8;
                p[0] = (int)(uint32_t)wt.first;
                p[1] = (int)(wt.first >> 32);
                p[2] = wt.e;
                p[3] = wt.m0;
                p[4] = wt.rows;
                p[5] = wt.n0;
            }
            wtile = wtile + 1 == S::kRing ? 0 : wtile + 1;
        }
        if (MODE == kBf16 && tail && wstep == steps - 1) {  // a partial last step
#pragma unroll
            for (int i = 0; i < S::kWLoads; ++i)
                if ((c8 ^ wkey((wave * S::kWLoads + i) * 8 + r8)) * 16 >= tail)
                    woff[i] = kNowhere;
        }
    };
    const auto load_weights = [&](int i) {
        load_lds(uniform(lds0 + XBUF * S::kXStep + wbuf * S::kWStep +
                         (wave * S::kWLoads + i) * 1024),
                 wr, woff[i], (uint32_t)wstep * kRow);
    };
    const auto end_weights = [&]() {
        wbuf = wbuf + 1 == WBUF ? 0 : wbuf + 1;
        ++wstep;
    };

    const auto ring_tile = [&](int i) {
        const int *p = ring + i * 8;
        Tile o;
        o.first = (int64_t)((uint64_t)(uint32_t)uniform(p[0]) |
                            (uint64_t)(uint32_t)uniform(p[1]) << 32);
        o.e = uniform(p[2]), o.m0 = uniform(p[3]), o.rows = uniform(p[4]), o.n0 = uniform(p[5]);
        return o;
    };

    // ---- row loads, with the scales of four steps at a time
    int xstep = steps, xbuf = 0, xtile = 0, xgroup = 0;
    i32x4 xr{0, 0, 0, 0x00020000}, sr = xr;  // rows; row scales or weight scales
    uint32_t xoff[S::kALoads] = {}, soff = 0;
    const auto begin_rows = [&]() {
        if (xstep == steps) {
            xstep = 0;
            const Tile o = S::XA == S::WA ? wt : ring_tile(xtile);
            xtile = xtile + 1 == S::kRing ? 0 : xtile + 1;
            if (o.rows > 0) {
                // base: the first row a load may name (regions: the expert's)
                const int64_t base = o.first + (gather ? 0 : o.m0);
                Regions g{};
                if (gather)
                    g.load(a, o.e);
                xr = buffer_of(static_cast<const char *>(a.x) + base * kbytes,
                               (a.n_rows - base) * kbytes);
#pragma unroll
                for (int i = 0; i < S::kALoads; ++i) {
                    const int lr = (i * kWaves + wave) * 8 + r8;  // row of the tile
                    const int m = min(lr, o.rows - 1);
                    const int row = gather ? g.row(a, o.m0 + m) : m;
                    xoff[i] = (uint32_t)((int64_t)row * kbytes) + (uint32_t)((c8 ^ r8) * 16);
                    if (lr >= ((o.rows + 15) & ~15))
                        xoff[i] = kNowhere;
                }
                if constexpr (S::kFp8Rows) {
                    const int st = scale_stride(a.K);
                    if (wave < kScaleWaves) {
                        sr = buffer_of(a.xs + base * st, (a.n_rows - base) * st * 4);
                        const int m = min(wave * kWave + lane, o.rows - 1);
                        const int row = gather ? g.row(a, o.m0 + m) : m;
                        soff = (uint32_t)((int64_t)row * st * 4);
                    } else {
                        const int64_t sb = ((int64_t)o.e * nb_n + (o.n0 >> 7)) * kb_n;
                        sr = buffer_of(a.ws + sb, ((int64_t)a.L * nb_n * kb_n - sb) * 4);
                        // lane 1: the up rows' block, or the tile's second block
                        const int blk = lane == 1 ? (GATED ? a.N >> 7 : 1) : 0;
                        soff = (uint32_t)(blk * kb_n * 4);
                    }
                }
                // the compiler would wait for loads made here wherever their
                // results are used, behind loads it does not know of
                if (gather)
                    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
            } else {
                xr[2] = sr[2] = 0;
            }
        }
        if constexpr (S::kFp8Rows) {
            if ((xstep & 3) == 0) {
                if (wave <= kScaleWaves)
                    load_lds(uniform(lds0 + S::kScaleAt + xgroup * S::kScale + wave * 1024), sr,
                             soff, (uint32_t)xstep * 4);
                xgroup = xgroup + 1 == XBUF ? 0 : xgroup + 1;
            }
        } else if (tail && xstep == steps - 1) {
#pragma unroll
            for (int i = 0; i < S::kALoads; ++i)
                if ((c8 ^ r8) * 16 >= tail)
                    xoff[i] = kNowhere;
        }
    };
    const auto load_rows = [&](int i) {
        if (BM % 64 && (i * kWaves + wave) * 8 >= BM)
            return;
        load_lds(uniform(lds0 + xbuf * S::kXStep + (i * kWaves + wave) * 1024), xr, xoff[i],
                 (uint32_t)xstep * kRow);
    };
    const auto end_rows = [&]() {
        xbuf = xbuf + 1 == XBUF ? 0 : xbuf + 1;
        ++xstep;
    };

    // ---- products
    const int pos = (g4 ^ (l16 & 7)) * 16;  // the lane's first piece of its row, swizzled
    // weight rows of a wave, arranged so that a lane's results of fragments j
    // and j + 1 (j even) are eight consecutive columns, and those of its row's
    // four lanes 64 bytes or more together: fragment row l16 is column
    // 8 (l16 / 4) + 4 (j % 2) + l16 % 4 of the fragment pair's 32 (gated: one
    // pair gate columns, one the up rows of the same)
    const int wrow = wn * (GATED ? 32 : 64) + (l16 >> 2) * 8 + (l16 & 3);
    constexpr int kPairRows = GATED ? 128 : 32;
    const char *const xlane = smem + (wm * 16 + l16) * kRow;
    const char *const wlane = smem + XBUF * S::kXStep + wrow * kRow;

    f32x4 acc[4][MF];
    Tile o{};
    int mf = 0, s = 0, xcur = 0, wcur = 0, group = 0, tile = 0;
#pragma unroll 1
    for (int it = -S::WA; it < 0; ++it) {  // fill the buffers
        meet();
        begin_weights();
        if (it + S::XA >= 0) {
            begin_rows();
#pragma unroll
            for (int p = 0; p < S::kALoads; ++p)
                load_rows(p);
            end_rows();
        }
#pragma unroll
        for (int p = 0; p < S::kWLoads; ++p)
            load_weights(p);
        end_weights();
    }
    for (;;) {
        wait_and_meet<S::kUnderWay>();
        if (s == 0) {
            o = ring_tile(tile);
            if (o.rows == 0)
                break;
            tile = tile + 1 == S::kRing ? 0 : tile + 1;
            mf = (((o.rows + 15) >> 4) - wm + kWM - 1) / kWM;  // fragments of this wave
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < MF; ++i)
                    acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const char *const sc = smem + S::kScaleAt + group * S::kScale + (s & 3) * 4;
        const char *const xb = xlane + xcur * S::kXStep, *const wb = wlane + wcur * S::kWStep;
        // A wave without rows widens no weights, which would hold up its
        // neighbour (128-row tiles, 256 regions of four rows: 1230 us against
        // 1330). Not in the others: 64-row tiles 1235 against 1280 for four rows
        // an expert but 1380 against 1335 for thirty, 160-row tiles 1% slower.
        const bool busy = MODE != kWide || BM != 128 || mf > 0;
        Raw x{};
        Frag<MODE> w[4];
        if (busy) {
            x = Raw::read(xb, pos);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = Frag<MODE>(Raw::read(wb + ((j >> 1) * kPairRows + (j & 1) * 4) * kRow,
                                            pos));
        }
        float sw[2] = {0.0f, 0.0f};
        if constexpr (S::kFp8Rows) {
            sw[0] = *reinterpret_cast<const float *>(sc + (S::kScaleRows + (GATED ? 0 : wn >> 1)) * 16);
            if (GATED)
                sw[1] = *reinterpret_cast<const float *>(sc + (S::kScaleRows + 1) * 16);
        }
        begin_weights();
        begin_rows();
        // The wave's row fragments two at a time, as far as the tile has rows.
        // Fragment i + 1 is read while the matrix unit works on fragment i.
        // The step's loads go between the products: where there is time for
        // them to arrive, evenly, as a wave that issues them faster than 64
        // bytes a cycle and compute unit waits; with two buffers, early.
        constexpr int kOver = XBUF >= 3 || MODE == kWide ? MF : 2;  // fragments
        const auto piece_at = [&](int i) {
            return (i < kOver ? i : kOver) * S::kLoads / kOver;
        };
        const auto load_piece = [&](int p) {
            if (p < S::kALoads)
                load_rows(p);
            else
                load_weights(p - S::kALoads);
        };
        const auto part = [&](auto from, auto count) {
            constexpr int I0 = decltype(from)::value, I1 = I0 + decltype(count)::value;
            float sx[I1 - I0];
            if constexpr (S::kFp8Rows) {
#pragma unroll
                for (int i = I0; i < I1; ++i)
                    sx[i - I0] =
                        *reinterpret_cast<const float *>(sc + ((i * kWM + wm) * 16 + l16) * 16);
            }
            // an FP8 fragment's products are scaled and added between the
            // products of the next one
            f32x4 d[2][4];
            const auto add = [&](int i, int j) {
                const float sc_ = sx[i - I0] * sw[GATED && j >= 2];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float v = __builtin_fmaf(sc_, d[i & 1][j][c], acc[j][i][c]);
                    // keeps the sum here: moved behind a branch between the
                    // parts, it would hold its operands until then
                    asm volatile("" : "+v"(v));
                    acc[j][i][c] = v;
                }
            };
#pragma unroll
            for (int i = I0; i < I1; ++i) {
                const Frag<MODE> xf(x);
                if (i + 1 < MF)
                    x = Raw::read(xb + (i + 1) * kWM * 16 * kRow, pos);
                if constexpr (MODE == kFp8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        d[i & 1][j] = multiply<MODE>(w[j], xf, 0, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                        if (i > I0)
                            add(i - 1, j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else if constexpr (MODE == kWide) {
                    // four chains of four products, so that no product waits
                    // for the one before it
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        d[i & 1][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            d[i & 1][j] = multiply<MODE>(w[j], xf, k, d[i & 1][j]);
                        if (i > I0)
                            add(i - 1, k);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < Frag<MODE>::kProducts; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[j][i] = multiply<MODE>(w[j], xf, k, acc[j][i]);
                }
#pragma unroll
                for (int p = piece_at(i); p < piece_at(i + 1); ++p)
                    load_piece(p);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (S::kFp8Rows) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    add(I1 - 1, j);
            }
        };
        // the loads of the parts left out
        const auto rest = [&](int i0) {
#pragma unroll
            for (int p = 0; p < S::kLoads; ++p)
                if (p >= piece_at(i0))
                    load_piece(p);
        };
        if (busy)
            part(Const<0>{}, Const<2>{});
        else
            rest(0);
        if (MF > 2 && mf > 2) {
            part(Const<(MF > 2 ? 2 : 0)>{}, Const<2>{});
            if (MF > 4 && mf > 4) {
                part(Const<(MF > 4 ? 4 : 0)>{}, Const<(MF > 5 ? 2 : 1)>{});
                if (MF > 6 && mf > 6)
                    part(Const<(MF > 6 ? 6 : 0)>{}, Const<2>{});
                else if (MF > 6)
                    rest(6);
            } else if (MF > 4) {
                rest(4);
            }
        } else if (MF > 2 && busy) {
            rest(2);
        }
        end_rows();
        end_weights();
        xcur = xcur + 1 == XBUF ? 0 : xcur + 1;
        wcur = wcur + 1 == WBUF ? 0 : wcur + 1;
        if ((s & 3) == 3 || s + 1 == steps)
            group = group + 1 == XBUF ? 0 : group + 1;
        if (++s < steps)
            continue;
        s = 0;

        // ---- epilogue: lane l holds columns of rows (2 i + wm) * 16 + l16
        Regions regions{};
        if (gather)
            regions.load(a, o.e);
        const auto out_row = [&](int m) -> int64_t {  // (every lane of the wave calls it)
            return o.first + (gather ? regions.row(a, min(o.m0 + m, o.m0 + o.rows - 1)) : o.m0 + m);
        };
        if constexpr (!GATED) {
            const int n = o.n0 + wn * 64 + g4 * 8;
            // Short tiles' whole lines go past the L2: written back at the
            // launch's end they cost 41 us against 34 (FP8, 256 regions of four
            // rows, 7168 columns) and 832 against 805 (256 experts of 120). Not
            // lines that several rows share (N = 1000: 56 us against 42), and
            // not beside 256-row tiles (bf16, 3700 rows an expert: 810 against
            // 790) or gated results, of which a wave has half lines.
            // (Two loops: the compiler would join two stores and drop the hint.)
            const auto store = [&](auto stream) {
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    const int m = (i * kWM + wm) * 16 + l16;
                    const int64_t row = out_row(m);
                    if (i < mf && m < o.rows) {
                        uint16_t *p = static_cast<uint16_t *>(a.out) + row * a.N + n;
                        u32x4 v[2];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                v[j >> 1][2 * (j & 1) + c] =
                                    f32_to_bf16(acc[j][i][2 * c]) |
                                    (f32_to_bf16(acc[j][i][2 * c + 1]) << 16);
                        if (n < a.N)  // N is a multiple of 8
                            store_result<decltype(stream)::value>(p, v[0]);
                        if (n + 32 < a.N)
                            store_result<decltype(stream)::value>(p + 32, v[1]);
                    }
                }
            };
            if (BM < 256 && a.N % 64 == 0)
                store(Const<(BM < 256)>{});
            else
                store(Const<0>{});
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
                    const int64_t row = out_row(m);
                    if (i < mf && m < o.rows && n < a.N) {
                        u32x4 v;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                v[2 * j + c] = f32_to_bf16(acc[j][i][2 * c]) |
                                               (f32_to_bf16(acc[j][i][2 * c + 1]) << 16);
                        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + row * a.N +
                                                   n) = v;
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
                    const int64_t row = out_row(m);
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
    }
    // no load may reach LDS after the block has given it back
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <Mode MODE, bool GATED, int BM, int XBUF, int WBUF>
hipError_t launch(const GroupedArgs &a, hipStream_t stream)
{
    using S = Shape<MODE, GATED, BM, XBUF, WBUF>;
    static_assert(S::kLds <= 160 * 1024, "");
    const int64_t cols = GATED ? kBN / 2 : kBN;
    const int64_t most = (a.n_rows / BM + a.L) * ((a.N + cols - 1) / cols);  // tiles there can be
    const int64_t blocks = most < a.cus ? most : a.cus;
    if (most > kMostTiles)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((grouped_kernel<MODE, GATED, BM, XBUF, WBUF>), dim3((unsigned)blocks),
                       dim3(kThreads), S::kLds, stream, a);
    return hipGetLastError();
}

// Tile height and buffers by the rows an expert has on average, as far as the
// host knows them: n_rows / L, for regions their capacity, however few rows
// they hold. (The pairs of times are from when each choice was made.) Few
// rows: the weights' stream decides, and three steps of both operands in LDS
// keep more of it under way (256 regions of 4 rows, FP8 gated: capacity 128
// 1237 us; capacity 129 and more, 160 rows with two steps of rows and three of
// weights, 1598); with at most 64, or 48 on average, 64-row tiles load less
// that is not used (8 experts of 16 rows, 4096 x 1024, bf16 gated: 15.3 us,
// against 22.3 for 160-row tiles; FP8 gated, 64 experts of 32 rows, 4096 x 2048:
// 107, against 112 for 128-row tiles). Around 128 rows: one tile per expert
// (gated FP8, 256 experts of 128 rows: 2230 us, against 2900 for 128-row
// tiles; product over regions of 128 rows: 34 against 52; bf16 has room for
// three steps of 160 rows: 345 us for 94 rows on average, against 362 for
// 128-row tiles). Many: the fewest bytes per product (bf16, 3700 rows: 770 us
// against 830 for 160-row tiles; FP8, 770 rows: 483 against 517).
template <Mode MODE, bool GATED>
hipError_t pick(const GroupedArgs &a, hipStream_t stream)
{
    const int64_t per = a.n_rows / a.L;
    if constexpr (MODE != kWide) {
        if (a.off && per > 384)
            return launch<MODE, GATED, 256, 2, 2>(a, stream);
    }
    if (per <= (a.off ? 48 : 64))
        return launch<MODE, GATED, 64, 3, 3>(a, stream);
    if constexpr (MODE == kBf16)
        return launch<MODE, GATED, 160, 3, 3>(a, stream);
    else
        return per <= (a.off ? 96 : 128) ? launch<MODE, GATED, 128, 3, 3>(a, stream)
                                         : launch<MODE, GATED, 160, 2, 3>(a, stream);
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
