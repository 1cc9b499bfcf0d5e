"""The experts' arithmetic on the GPU -- weight quantiser, grouped products,
gated products, low-latency regions, the whole layer for a few tokens --
against 64-bit results on the CPU within derived bounds (tests/_experts.py)."""
import ctypes

import numpy as np
import pytest
import torch

import _experts as X
from _gpu import CANARY, say

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def epx():
    import combine_get_dispatch_counts_amd as m

    return m


def gpu(*ts):
    r = [None if t is None else t.to(DEV) for t in ts]
    return r[0] if len(r) == 1 else r


def canary(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(CANARY)
    return t


def untouched(t, rows):
    """Rows of t whose mask is set still hold the canary."""
    b = t[rows].contiguous().view(torch.uint8)
    return bool((b == CANARY).all())


# ------------------------------------------------------------- quantiser

@pytest.mark.parametrize("E,N,K", [(1, 8, 128), (3, 5, 256), (2, 128, 640), (2, 129, 128),
                                   (1, 264, 1024), (5, 256, 512)])
def test_quantize_weights(E, N, K):
    w = X.randn((E, N, K), 11, 0.02)
    w[0, 0, :128] = 0.0
    w[-1, N // 2:, -128:] *= 1000.0
    w[-1, -1, 0] = 1e-30
    say(f"quantize_weights {E}x{N}x{K}")
    q, s = epx().quantize_weights(gpu(w))
    up = -(-N // 128) * 128
    b = torch.zeros((E, up, K))
    b[:, :N] = w.float()
    b = b.view(E, up // 128, 128, K // 128, 128)
    sr = b.abs().amax(dim=(2, 4)).clamp_min(1e-4) / 448.0      # fp32 throughout
    qr = (b / sr[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(s.cpu().view(torch.int32), sr.view(torch.int32))
    assert torch.equal(q.cpu(), qr.view(E, up, K)[:, :N])


def test_quantize_weights_non_finite():
    """Inf and NaN stay in their block: amax over the values that compare, an
    Inf block has an Inf scale and zero codes, NaN quotients are 0x7F."""
    w = X.randn((1, 256, 384), 12)
    w[0, 3, 5] = float("nan")                # block (0, 0): a NaN among finite values
    w[0, 130, 200] = float("-inf")           # block (1, 1)
    say("quantize_weights non-finite")
    q, s = (t.cpu() for t in epx().quantize_weights(gpu(w)))
    b = w.float().view(2, 128, 3, 128)
    ok = torch.where(b.isnan(), torch.zeros(()), b.abs())
    sr = ok.amax(dim=(1, 3)).clamp_min(1e-4) / 448.0
    v = b / sr[:, None, :, None]
    qr = torch.where(v.isnan(), torch.full((), 0x7F, dtype=torch.uint8),
                     v.to(torch.float8_e4m3fn).view(torch.uint8)).view(256, 384)
    assert torch.equal(s[0].view(torch.int32), sr.view(torch.int32))
    assert torch.equal(q[0], qr)


# -------------------------------------------------------------- products

COUNTS = {
    "one row": [1],
    "empty experts": [0, 3, 0, 0, 17, 0],
    "ragged": [65, 1, 64, 130, 0, 7],
    "no rows at all": [0, 0],
    "long": [300, 5],
    "many": [2, 0, 1, 5] * 40,
}


def _operands(fp8, n, L, rows_w, K, seed):
    if fp8:
        x, xs = X.fp8_rows((n, K), seed)
        w, ws = X.fp8_weights((L, rows_w, K), seed + 1)
        return x, xs, w, ws
    return X.randn((n, K), seed), None, X.randn((L, rows_w, K), seed + 1, K ** -0.5), None


def _check_rows(gated, fp8, out, out_s, rows_of, x, xs, w, ws):
    """rows_of[e]: the row numbers of expert e."""
    for e, r in enumerate(rows_of):
        if len(r) == 0:
            continue
        r = torch.as_tensor(r, dtype=torch.long)
        xe = X.rows64(x[r], None if xs is None else xs[r])
        we = X.weights64(w[e], None if ws is None else ws[e])
        if not gated:
            y, tol = X.product(xe, we)
            if fp8:
                tol = tol + X.cut(x[r], xs[r], w[e], ws[e])
        else:
            y, tol = X.gated(xe, we)
            if fp8:
                X.assert_codes(out[r.to(DEV)], out_s[r.to(DEV)], y, tol, f"expert {e}")
                continue
        X.assert_close(out[r.to(DEV)], y, tol + X.BF16 * (y.abs() + tol), f"expert {e}")


def _run(gated, fp8, counts, N, K, seed, lead=0, tail=0):
    off = X.offsets(counts, lead)
    n, L = int(off[-1]) + tail, len(counts)
    x, xs, w, ws = _operands(fp8, n, L, 2 * N if gated else N, K, seed)
    # rows of no expert may hold anything
    dead = torch.ones(n, dtype=torch.bool)
    dead[lead:off[-1]] = False
    if fp8:
        x[dead] = 0x7F
    else:
        x[dead] = float("nan")
    xd, xsd, wd, wsd = gpu(x, xs, w, ws)
    offd = torch.from_numpy(off).to(DEV)
    out = canary((n, N), torch.uint8 if gated and fp8 else torch.bfloat16)
    out_s = canary((n, X.stride(N)), torch.float32) if gated and fp8 else None
    if gated:
        epx().grouped_swiglu(xd, wd, offd, xsd, wsd, out=out, out_scales=out_s)
    else:
        epx().grouped_gemm(xd, wd, offd, xsd, wsd, out=out)
    assert epx().get_error() == 0
    _check_rows(gated, fp8, out, out_s,
                [np.arange(off[e], off[e + 1]) for e in range(L)], x, xs, w, ws)
    assert untouched(out, dead.to(DEV))
    if out_s is not None:
        assert untouched(out_s, dead.to(DEV))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("which", list(COUNTS))
def test_grouped_rows(which, gated, fp8):
    say(f"grouped {which} gated={gated} fp8={fp8}")
    _run(gated, fp8, COUNTS[which], 256, 256, 21, lead=3, tail=5)


SIZES = [(8, 8), (24, 40), (136, 72), (264, 1416), (120, 128), (520, 2048)]
SIZES_FP8 = [(8, 128), (24, 384), (136, 640), (264, 1152), (1000, 2176)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_sizes_bf16(N, K, gated):
    say(f"grouped bf16 N={N} K={K} gated={gated}")
    _run(gated, False, [5, 0, 70, 129], N, K, 31)


@pytest.mark.parametrize("N,K", SIZES_FP8)
def test_grouped_sizes_fp8(N, K):
    say(f"grouped fp8 N={N} K={K}")
    _run(False, True, [5, 0, 70, 129], N, K, 32)


@pytest.mark.parametrize("N,K", [(128, 128), (384, 128), (128, 1152), (640, 2176), (4224, 384)])
def test_grouped_swiglu_sizes_fp8(N, K):
    say(f"grouped swiglu fp8 f={N} K={K}")
    _run(True, True, [5, 0, 70, 129], N, K, 33)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_many_tiles(fp8, gated):
    """More output tiles than the device holds at once, uneven experts."""
    say(f"grouped many tiles fp8={fp8} gated={gated}")
    rng = np.random.default_rng(5)
    counts = [int(c) for c in rng.integers(0, 190, 24)] + [900, 1]
    _run(gated, fp8, counts, 2176, 256, 41)


TALL = {
    # heights of a tile, one row less and one more; on average above 384 rows
    "tall": [256, 257, 1023, 0, 511],
    "medium": [159, 160, 161, 321, 97],
    "short": [127, 128, 129, 1, 0, 31],
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("which", list(TALL))
def test_grouped_tile_heights(which, gated, fp8):
    N, K = (384, 640) if fp8 else (264, 200)
    say(f"grouped {which} gated={gated} fp8={fp8}")
    _run(gated, fp8, TALL[which], N, K, 43, lead=2, tail=7)


@pytest.mark.parametrize("fp8,K", [(False, 64), (False, 40), (False, 128), (True, 128)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows", [70, 150, 500])
def test_grouped_one_step_many_tiles(rows, gated, fp8, K):
    """One or two steps of channels, several tiles a block: the loads run more
    tiles ahead than a tile has steps."""
    say(f"grouped rows={rows} K={K} gated={gated} fp8={fp8}")
    rng = np.random.default_rng(6)
    counts = [int(c) for c in rng.integers(rows - 60, rows + 60, 16)]
    _run(gated, fp8, counts, 5120 if rows < 200 else 2688, K, 44)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,K", [(128, 65536), (65536, 128)])
def test_grouped_largest_sizes(N, K, fp8):
    say(f"grouped N={N} K={K} fp8={fp8}")
    for gated in (False, True):
        _run(gated, fp8, [2, 0, 17], N, K, 45, lead=1)


def test_fp8_products_are_cut_as_stated():
    """The plain FP8 product against sums of products that are cut the way
    its instruction cuts them: random codes, and pairs that cancel beside
    small products."""
    say("fp8 sums")
    n, K = 512, 128
    g = torch.Generator().manual_seed(46)
    for scale in (110.0, 4.0, 0.02):
        x = (torch.randn((n, K), generator=g) * 110).clamp(-448, 448)
        w = (torch.randn((n, K), generator=g) * scale).clamp(-448, 448)
        x[::2, 1::8], w[::2, 1::8] = -x[::2, ::8], w[::2, ::8]      # cancel in every second row
        x[::2, 2::8] /= 64
        x, w = (v.to(torch.float8_e4m3fn).view(torch.uint8) for v in (x, w))
        off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        out = epx().grouped_gemm(gpu(x), gpu(w[None]), off,
                                 torch.ones((n, X.stride(K)), device=DEV),
                                 torch.ones((1, n // 128, 1), device=DEV))
        y, mag = X.cut_product(x, w)
        tol = (K + 8) * X.U32 * mag
        X.assert_close(out.diagonal(), y, tol + X.BF16 * (y.abs() + tol), f"scale {scale}")


# --------------------------------------------------- low-latency regions

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("L,R,cap,most", [(1, 1, 1, 1), (5, 1, 33, 33), (3, 4, 20, 20),
                                          (2, 64, 9, 4), (300, 1, 3, 3), (2, 8, 100, 100),
                                          (3, 1, 128, 12), (3, 1, 128, 128), (4, 2, 64, 20)])
def test_ll_grouped(L, R, cap, most, gated, fp8):
    say(f"ll grouped L={L} R={R} cap={cap} gated={gated} fp8={fp8}")
    N, K = 256, 384
    rng = np.random.default_rng(51 + L)
    counts = rng.integers(-1, most + 1, L * R).astype(np.int32)
    counts[rng.random(L * R) < 0.3] = -1
    counts[0], counts[-1] = most, 1
    n = L * R * cap
    x, xs, w, ws = _operands(fp8, n, L, 2 * N if gated else N, K, 52)
    live = (np.arange(cap)[None, :] < counts[:, None]).reshape(-1)
    dead = torch.from_numpy(~live)
    x[dead] = 0x7F if fp8 else float("nan")
    xd, xsd, wd, wsd = gpu(x, xs, w, ws)
    out = canary((n, N), torch.uint8 if gated and fp8 else torch.bfloat16)
    out_s = canary((n, X.stride(N)), torch.float32) if gated and fp8 else None
    cd = torch.from_numpy(counts).to(DEV)
    if gated:
        epx().ll_grouped_swiglu(xd, wd, cd, cap, xsd, wsd, out=out, out_scales=out_s)
    else:
        epx().ll_grouped_gemm(xd, wd, cd, cap, xsd, wsd, out=out)
    assert epx().get_error() == 0
    rows = [np.flatnonzero(live[e * R * cap:(e + 1) * R * cap]) + e * R * cap for e in range(L)]
    if L > 8:  # a sample of the experts, the first and the last among them
        rows = [r if e % 37 == 0 or e == L - 1 else r[:0] for e, r in enumerate(rows)]
    _check_rows(gated, fp8, out, out_s, rows, x, xs, w, ws)
    assert untouched(out, dead.to(DEV))
    if out_s is not None:
        assert untouched(out_s, dead.to(DEV))


def test_ll_grouped_far_rows():
    """Regions whose byte offsets pass 32 bits: only the last expert has rows."""
    L, cap, N, K = 256, 2100, 4096, 8192     # 4.4 GB of codes and of results
    say("ll grouped far rows")
    x = torch.empty((L * cap, K), dtype=torch.uint8, device=DEV)
    xs = torch.empty((L * cap, X.stride(K)), device=DEV)
    xr, xsr = X.fp8_rows((3, K), 61)
    first = (L - 1) * cap
    x[first:first + 3], xs[first:first + 3] = gpu(xr, xsr)
    w1, ws1 = X.fp8_weights((1, N, K), 62)
    w = torch.empty((L, N, K), dtype=torch.uint8, device=DEV)      # 8.6 GB
    ws = torch.empty((L, N // 128, K // 128), device=DEV)
    w[-1:], ws[-1:] = gpu(w1, ws1)
    counts = torch.zeros(L, dtype=torch.int32, device=DEV)
    counts[-1] = 3
    out = torch.empty((L * cap, N), dtype=torch.bfloat16, device=DEV)
    epx().ll_grouped_gemm(x, w, counts, cap, xs, ws, out=out)
    assert epx().get_error() == 0
    y, tol = X.product(X.rows64(xr, xsr), X.weights64(w1[0], ws1[0]))
    X.assert_close(out[first:first + 3], y, tol + X.BF16 * (y.abs() + tol), "far rows")


# ------------------------------------------------------ values and errors

@pytest.mark.parametrize("fp8", [False, True])
def test_non_finite_rows_stay_alone(fp8):
    """A row holding NaN or Inf, and an expert whose weights hold one, spoil
    their own results only."""
    say(f"non-finite rows fp8={fp8}")
    counts, N, K = [9, 20, 70], 256, 256
    off = X.offsets(counts)
    x, xs, w, ws = _operands(fp8, 99, 3, 2 * N, K, 71)
    x[4, 7] = 0x7F if fp8 else float("inf")       # expert 0, row 4
    w[2, 5, 0] = 0x7F if fp8 else float("nan")    # expert 2, gate column 5
    xd, xsd, wd, wsd = gpu(x, xs, w, ws)
    act, act_s = epx().grouped_swiglu(xd, wd, torch.from_numpy(off).to(DEV), xsd, wsd)
    assert epx().get_error() == 0
    good = [np.array([0, 1, 2, 3, 5, 6, 7, 8]), np.arange(9, 29)]
    _check_rows(True, fp8, act, act_s, good + [[]], x, xs, w, ws)
    if fp8:
        v = act.cpu().view(torch.float8_e4m3fn).float()
        assert v[29:, 5].isnan().all()
        assert not v[29:, :5].isnan().any() and not v[29:, 6:].isnan().any()
        assert v[4].isnan().all()
    else:
        v = act.cpu().float()
        assert v[29:, 5].isnan().all()
        assert not v[29:, :5].isnan().any() and not v[29:, 6:].isnan().any()


def test_extreme_gates():
    """Gates far outside exp's range: silu goes to 0 or to the gate itself,
    in a fp8 row the group's scale follows its largest value and an all-zero
    group has the floor's scale."""
    say("extreme gates")
    K = N = 128
    x = torch.zeros((4, K), dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([-3e4, 3e4, 0.0, -100.0])
    x[:, 1] = 1.0
    w = torch.zeros((1, 2 * N, K), dtype=torch.bfloat16)
    w[0, :N, 0] = 1.0
    w[0, N:, 1] = 2.0
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    act, _ = epx().grouped_swiglu(gpu(x), gpu(w), off)
    a = act.float().cpu()
    assert (a[0] == 0).all() and (a[2] == 0).all() and (a[3].abs() < 1e-30).all()
    assert ((a[1] - 6e4).abs() <= 6e4 * X.BF16).all()
    xq = torch.zeros((4, K), dtype=torch.uint8)
    xq[:, 0] = torch.tensor([0xFE, 0x7E, 0x00, 0xFE], dtype=torch.uint8)   # -448, 448, 0, -448
    xq[:, 1] = 0x38                                                        # 1
    xs = torch.zeros((4, X.stride(K)))
    xs[:, 0] = torch.tensor([100.0, 100.0, 1.0, 1.0])
    wq = torch.where(w == 1, 0x38, torch.where(w == 2, 0x40, 0)).to(torch.uint8)
    ws = torch.ones((1, 2, 1))
    q, s = epx().grouped_swiglu(gpu(xq), gpu(wq), off, gpu(xs), gpu(ws))
    s, v = s.cpu(), q.cpu().view(torch.float8_e4m3fn).float()
    floor = np.float32(1e-4) / np.float32(448)
    assert s[0, 0] == floor and s[2, 0] == floor and s[3, 0] == floor
    assert (v[[0, 2, 3]] == 0).all()
    assert (v[1] == 448).all()
    assert abs(float(s[1, 0]) * 448 - 44800.0 * 200.0) <= 44800.0 * 200.0 * 8 * X.U32


def test_bad_offsets_are_flagged_and_clamped():
    say("bad offsets")
    N, K, n = 64, 64, 40
    x, w = X.randn((n, K), 81), X.randn((3, N, K), 82)
    buf = canary((n + 64, N), torch.bfloat16)
    for bad in ([0, 10, 5, 40], [0, 10, 20, 4000], [-7, 10, 20, 40], [2 ** 31 - 1, 0, 0, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        epx().grouped_gemm(gpu(x), gpu(w), off, out=buf[:n])
        assert epx().get_error() == 2, bad
        epx().grouped_swiglu(gpu(x), gpu(w), off, out=buf[:n, :].view(-1)[:n * N // 2].view(n, N // 2))
        assert epx().get_error() == 2, bad
        assert untouched(buf, torch.arange(n, n + 64, device=DEV))
    counts = torch.tensor([1, 99, -5], dtype=torch.int32, device=DEV)
    buf = canary((30 + 64, N), torch.bfloat16)
    epx().ll_grouped_gemm(gpu(x[:30]), gpu(w), counts, 10, out=buf[:30])
    assert epx().get_error() == 2
    assert untouched(buf, torch.arange(30, 94, device=DEV))


def test_size_limits():
    """What the kernels cannot address is refused before any launch: the
    pointers are never followed."""
    from combine_get_dispatch_counts_amd import _lib
    from combine_get_dispatch_counts_amd.api import _ctx

    say("size limits")
    lib, ctx, p = _lib.load(), _ctx(DEV), ctypes.c_void_p(256)

    def gemm(n, K, L, N, fp8):
        return lib.epx_grouped_gemm(ctx, p, p, n, K, p, p, L, N, fp8, p, p, None)

    def swiglu(n, K, L, f, fp8):
        return lib.epx_grouped_swiglu(ctx, p, p, n, K, p, p, L, f, fp8, p, p, p, None)

    def ll(K, N, fp8, R, cap, L=1):
        return lib.epx_ll_grouped_gemm(ctx, p, p, K, p, p, L, N, fp8, p, R, cap, p, None)

    for bad in ((1, 65536, 1, 32768, 0), (1, 65536, 1, 65536, 1), (1, 65536 + 128, 1, 8, 0),
                (1, 8, 1, 65536 + 8, 0), (2 ** 31, 8, 1, 8, 0), (-1, 8, 1, 8, 0), (1, 8, 0, 8, 0),
                (1, 8, 513, 8, 0)):
        assert gemm(*bad) == -1, bad
    for bad in ((1, 65536, 1, 16384, 0), (1, 65536, 1, 32768, 1)):
        assert swiglu(*bad) == -1, bad
    assert ll(8192, 8, 0, 64, 8192) == -1            # 8.6 GB of one expert's rows
    assert ll(65536, 8, 1, 2, 32000) == -1           # with the scales above 4 GB
    assert ll(8, 8, 0, 65, 1) == -1 and ll(8, 8, 0, 0, 1) == -1 and ll(8, 8, 0, 1, 0) == -1
    assert ll(8, 8, 0, 64, 65536, L=512) == -1       # 2^31 rows
    assert epx().get_error() == 0


def test_refusals():
    say("refusals")
    m = epx()
    E = m.EpxError
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)     # noqa: E731
    f32 = lambda *s: torch.zeros(s, device=DEV)                       # noqa: E731
    x, w = bf(4, 64), bf(2, 32, 64)
    for call in (m.grouped_gemm, m.grouped_swiglu):
        with pytest.raises(TypeError):
            call(x.float(), w, off)
        with pytest.raises(TypeError):
            call(x, u8(2, 32, 64), off)
        with pytest.raises(TypeError):
            call(x, w, off.long())
        with pytest.raises(ValueError):
            call(x, w, off[:2])
        with pytest.raises(ValueError):
            call(x, bf(2, 32, 56), off)
        with pytest.raises(ValueError):
            call(bf(4, 128)[:, ::2], w, off)
        with pytest.raises(ValueError):
            call(x, w, off, f32(4, 32), f32(2, 1, 1))       # scales without FP8
        with pytest.raises(ValueError):
            call(u8(4, 128), u8(2, 128, 128), off)          # FP8 without scales
        with pytest.raises(E) as ex:
            call(u8(4, 64), w.view(torch.uint8)[:, :, :64].contiguous(), off, f32(4, 32),
                 f32(2, 1, 1))                              # K % 128
        assert ex.value.code == -3
        with pytest.raises(E) as ex:
            call(bf(4, 60), bf(2, 32, 60), off)             # K % 8
        assert ex.value.code == -1
        with pytest.raises(E) as ex:
            call(x, bf(2, 24, 64) if call is m.grouped_swiglu else bf(2, 12, 64), off)  # N % 8
        assert ex.value.code == -1
    with pytest.raises(E) as ex:
        m.grouped_swiglu(u8(4, 128), u8(2, 128, 128), off, f32(4, 32), f32(2, 1, 1))    # f = 64
    assert ex.value.code == -3
    with pytest.raises(ValueError):
        m.grouped_swiglu(x, bf(2, 31, 64), off)
    with pytest.raises(ValueError):
        m.grouped_gemm(x, w, off, out=bf(4, 31))
    shifted = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=DEV)[1:4 * 64 + 1].view(4, 64)
    with pytest.raises(E) as ex:
        m.grouped_gemm(shifted, w, off)
    assert ex.value.code == -1
    with pytest.raises(E):
        m.grouped_gemm(x, bf(513, 8, 64), torch.zeros(514, dtype=torch.int32, device=DEV))
    counts = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (dict(cap=3), dict(cap=0)):
        with pytest.raises(ValueError):
            m.ll_grouped_gemm(x, w, counts, **bad)
    with pytest.raises(ValueError):
        m.ll_grouped_gemm(x, w, counts[:3], 1)
    with pytest.raises(E) as ex:
        m.quantize_weights(bf(1, 8, 64))
    assert ex.value.code == -3
    with pytest.raises(TypeError):
        m.quantize_weights(f32(1, 8, 128))
    with pytest.raises(ValueError):
        m.quantize_weights(bf(8, 128))
    idx = torch.zeros((2, 2), dtype=torch.int64, device=DEV)
    tw = f32(2, 2)
    xx, w13, w2 = bf(2, 64), bf(3, 48, 64), bf(3, 64, 24)
    m.moe_decode(xx, idx, tw, w13, w2)
    with pytest.raises(TypeError):
        m.moe_decode(xx, idx.int(), tw, w13, w2)
    with pytest.raises(ValueError):
        m.moe_decode(xx, idx, tw[:, :1], w13, w2)
    with pytest.raises(ValueError):
        m.moe_decode(xx, idx, tw, w13, bf(3, 64, 32))
    with pytest.raises(ValueError):
        m.moe_decode(xx, idx, tw, w13, w2, w13_scales=f32(3, 1, 1))
    with pytest.raises(E) as ex:
        m.moe_decode(xx, idx, tw, w13, w2, workspace=u8(64))
    assert ex.value.code == -2
    with pytest.raises(E) as ex:
        m.moe_decode(bf(65, 64), idx[:1].repeat(65, 1), f32(65, 2), w13, w2)
    assert ex.value.code == -2
    with pytest.raises(E) as ex:
        m.moe_decode(xx, idx, tw, u8(3, 48, 64), u8(3, 64, 24), f32(3, 1, 0), f32(3, 1, 0))
    assert ex.value.code == -3
    assert m.get_error() == 0


# ------------------------------------------------------- few-token layer

def _decode_inputs(T, K, E, h, f, fp8, seed, p_drop=0.0, skew=False):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)) + (np.arange(E) * 0.2 if skew else 0), axis=1)[:, :K]
    idx = idx.astype(np.int64)
    idx[rng.random(idx.shape) < p_drop] = -1
    w13 = X.fp8_weights((E, 2 * f, h), seed + 1) if fp8 else (X.randn((E, 2 * f, h), seed + 1, h ** -0.5), None)
    w2 = X.fp8_weights((E, h, f), seed + 2) if fp8 else (X.randn((E, h, f), seed + 2, f ** -0.5), None)
    top = torch.from_numpy(rng.random((T, K)).astype(np.float32))
    return X.randn((T, h), seed + 3), torch.from_numpy(idx), top, w13, w2


def _decode_ref(x, idx, top, w13, w2):
    x = x.double()
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(w13[0].shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        a, da = X.gated(x[t], X.weights64(w13[0][e], None if w13[1] is None else w13[1][e]))
        da = da + X.BF16 * (a.abs() + da)          # the activation's rounding to bf16
        w = X.weights64(w2[0][e], None if w2[1] is None else w2[1][e])
        y, dy = X.product(a, w)
        dy = dy + da @ w.abs().T * (1 + (a.shape[1] + 8) * X.U32)
        tw = top[t, k].double()[:, None]
        out.index_add_(0, t, tw * y)
        tol.index_add_(0, t, tw.abs() * (dy + 64 * X.U32 * y.abs()))   # weights and sums
    return out, tol + X.BF16 * (out.abs() + tol)


def _check_decode(x, idx, top, w13, w2, **kw):
    xd, id_, td, a, sa, b, sb = gpu(x, idx, top, w13[0], w13[1], w2[0], w2[1])
    got = epx().moe_decode(xd, id_, td, a, b, sa, sb, **kw)
    assert epx().get_error() == 0
    ref, tol = _decode_ref(x, idx, top, w13, w2)
    X.assert_close(got, ref, tol, "decode")
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K,E,h,f", [(1, 1, 1, 128, 128), (1, 8, 32, 512, 256), (3, 2, 8, 128, 384),
                                       (7, 8, 300, 256, 128), (64, 2, 4, 384, 256),
                                       (33, 6, 64, 1024, 128), (17, 1, 1, 256, 640),
                                       (64, 32, 512, 128, 128), (2, 2, 3, 2176, 1152)])
def test_moe_decode(T, K, E, h, f, fp8):
    say(f"decode T={T} K={K} E={E} h={h} f={f} fp8={fp8}")
    _check_decode(*_decode_inputs(T, K, E, h, f, fp8, 91 + T))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("h,f", [(65536, 128), (128, 65536)])
def test_moe_decode_largest_sizes(h, f, fp8):
    say(f"decode h={h} f={f} fp8={fp8}")
    _check_decode(*_decode_inputs(3, 2, 2, h, f, fp8, 96))


@pytest.mark.parametrize("h,f", [(8, 8), (72, 24), (264, 1000), (1000, 136)])
def test_moe_decode_odd_sizes(h, f):
    say(f"decode bf16 h={h} f={f}")
    _check_decode(*_decode_inputs(5, 3, 6, h, f, False, 95))


@pytest.mark.parametrize("fp8", [False, True])
def test_moe_decode_routing(fp8):
    """Dropped entries, a token without any, an expert repeated by a token,
    one expert with every token."""
    say(f"decode routing fp8={fp8}")
    x, idx, top, w13, w2 = _decode_inputs(40, 4, 6, 256, 128, fp8, 101, p_drop=0.3)
    idx[5] = -1
    idx[6] = torch.tensor([2, 2, -1, 2])
    idx[7] = 3
    got = _check_decode(x, idx, top, w13, w2)
    assert (got[5] == 0).all()
    idx[:, 1] = 5
    _check_decode(x, idx, top, w13, w2)
    idx[:] = -1
    xd, td, a, sa, b, sb = gpu(x, top, w13[0], w13[1], w2[0], w2[1])
    out = canary((40, 256), torch.bfloat16)
    epx().moe_decode(xd, gpu(idx), td, a, b, sa, sb, out=out)
    assert (out == 0).all() and epx().get_error() == 0


def test_moe_decode_bad_route():
    say("decode bad route")
    x, idx, top, w13, w2 = _decode_inputs(6, 2, 4, 128, 128, False, 103)
    ref = idx.clone()
    idx[1, 0], idx[3, 1], idx[4, 0] = 4, -2, 2 ** 40
    ref[1, 0] = ref[3, 1] = ref[4, 0] = -1
    got = epx().moe_decode(*gpu(x, idx, top, w13[0], w2[0]))
    assert epx().get_error() == 1
    r, tol = _decode_ref(x, ref, top, w13, w2)
    X.assert_close(got, r, tol, "decode")


def test_moe_decode_no_tokens():
    say("decode no tokens")
    x, idx, top, w13, w2 = _decode_inputs(1, 2, 4, 128, 128, False, 104)
    out = epx().moe_decode(gpu(x)[:0], gpu(idx)[:0], gpu(top)[:0], gpu(w13[0]), gpu(w2[0]))
    assert out.shape == (0, 128) and epx().get_error() == 0


def test_moe_decode_non_finite():
    """A token with a NaN spoils its own row; so does a weight matrix for the
    tokens routed to it."""
    say("decode non-finite")
    x, idx, top, w13, w2 = _decode_inputs(20, 2, 4, 128, 128, False, 105)
    idx[:, 0], idx[:, 1] = 0, 1
    idx[10:, 1] = 2
    x[3, 5] = float("nan")
    w2[0][2, 9, 0] = float("inf")
    got = epx().moe_decode(*gpu(x, idx, top, w13[0], w2[0])).cpu().float()
    assert got[3].isnan().all()
    w2[0][2, 9, 0] = 0.0
    ref, tol = _decode_ref(x, idx, top, w13, w2)
    ok = torch.ones(20, dtype=torch.bool)
    ok[3] = False
    X.assert_close(got[ok][:9], ref[ok][:9], tol[ok][:9], "finite tokens")
    cols = [c for c in range(128) if c != 9]
    X.assert_close(got[10:][:, cols], ref[10:][:, cols], tol[10:][:, cols], "finite columns")
    assert not got[10:, 9].isfinite().any()


# -------------------------------------------------- together, streams, graphs

def _layer_inputs(T, K, E, h, f, seed):
    x, idx, top, _, _ = _decode_inputs(T, K, E, 128, 128, False, seed, p_drop=0.1)
    return (X.randn((T, h), seed), idx, top, X.randn((E, 2 * f, h), seed + 1, h ** -0.5),
            X.randn((E, h, f), seed + 2, f ** -0.5))


def _layer64(x, idx, top, w13, w2):
    x, out = x.double(), torch.zeros(x.shape, dtype=torch.float64)
    for e in range(w13.shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            a, _ = X.gated(x[t], w13[e].double())
            out.index_add_(0, t, top[t, k].double()[:, None] * (a @ w2[e].double().T))
    return out


def _rel(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ll", [False, True])
def test_layer_from_dispatch_to_combine(fp8, ll):
    """dispatch, gated product, product, combine -- both layouts, both row
    formats -- against the layer in 64 bits. Independent roundings of relative
    size r leave a sum's relative error near r: two roundings to e4m3 of each
    operand of the products (2^-4 at most) and a few to bf16."""
    say(f"layer fp8={fp8} ll={ll}")
    m = epx()
    T, K, E, R, h, f = 150, 4, 16, 4, 512, 384
    x, idx, top, w13, w2 = _layer_inputs(T, K, E, h, f, 111)
    xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
    sa = sb = None
    if fp8:
        (a, sa), (b, sb) = m.quantize_weights(a), m.quantize_weights(b)
    if ll:
        d = m.ll_dispatch(xd, id_, E, R, 0, T, R_buf=1, fp8=fp8)
        act, act_s = m.ll_grouped_swiglu(d.ll_x, a, d.ll_count, T, d.ll_scales, sa)
        y = m.ll_grouped_gemm(act, b, d.ll_count, T, act_s, sb)
        out = m.combine(y, d.pos_ll, td)
    else:
        d = m.dispatch(xd, id_, td, E, R, fp8=fp8)
        act, act_s = m.grouped_swiglu(d.recv_x, a, d.layout.exp_off, d.recv_scales, sa)
        y = m.grouped_gemm(act, b, d.layout.exp_off, act_s, sb)
        out = m.combine(y, d.pos_exp, td)
    assert m.get_error() == 0
    ref = _layer64(x, idx, top, w13, w2)
    assert _rel(out, ref) <= (4 * X.E4M3 if fp8 else 4 * X.BF16)
    few = m.moe_decode(xd[:64], id_[:64], td[:64], a, b, sa, sb)
    assert _rel(few, ref[:64]) <= (2 * X.E4M3 if fp8 else 4 * X.BF16)


def test_receiver_permute_then_products():
    """recv_permute's blocks into the products: capacity rows past the last
    expert stay as they were."""
    say("receiver permute then products")
    m = epx()
    N, K, L, h, f = 200, 3, 4, 256, 128
    rng = np.random.default_rng(121)
    idx = rng.integers(-1, L, (N, K)).astype(np.int64)
    rows = X.randn((N, h), 122)
    w = X.randn((L, 2 * f, h), 123, h ** -0.5)
    rec = m.recv_permute(gpu(rows), torch.from_numpy(idx).to(DEV), L)
    act = canary((N * K, f), torch.bfloat16)
    m.grouped_swiglu(rec.x, gpu(w), rec.layout.exp_off, out=act)
    assert m.get_error() == 0
    off = rec.layout.exp_off.cpu().numpy()
    _check_rows(True, False, act, None, [np.arange(off[e], off[e + 1]) for e in range(L)],
                rec.x.cpu(), None, w, None)
    assert untouched(act, torch.arange(int(off[-1]), N * K, device=DEV))


def test_same_bytes_twice():
    say("same bytes twice")
    m = epx()
    x, idx, top, w13, w2 = _layer_inputs(48, 6, 24, 512, 256, 131)
    xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
    one = m.moe_decode(xd, id_, td, a, b)
    d = m.dispatch(xd, id_, td, 24, 4)
    y1 = m.grouped_swiglu(d.recv_x, a, d.layout.exp_off)[0]
    for _ in range(4):
        assert torch.equal(m.moe_decode(xd, id_, td, a, b), one)
        assert torch.equal(m.grouped_swiglu(d.recv_x, a, d.layout.exp_off)[0], y1)


def test_on_another_stream():
    say("another stream")
    m = epx()
    x, idx, top, w13, w2 = _layer_inputs(20, 4, 8, 256, 128, 141)
    xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
    one = m.moe_decode(xd, id_, td, a, b)
    q, s = m.quantize_weights(a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        two = m.moe_decode(xd, id_, td, a, b)
        q2, s2 = m.quantize_weights(a)
    three = m.moe_decode(xd, id_, td, a, b)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(one, three)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_two_streams_at_once():
    """Different calls of the same operators side by side: nothing is shared."""
    say("two streams")
    m = epx()
    sets = []
    for seed in (161, 162):
        x, idx, top, w13, w2 = _layer_inputs(60, 4, 16, 512, 256, seed)
        xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
        d = m.dispatch(xd, id_, td, 16, 4)
        sets.append((xd, id_, td, a, b, d))

    def layer(xd, id_, td, a, b, d):
        act, _ = m.grouped_swiglu(d.recv_x, a, d.layout.exp_off)
        return (m.quantize_weights(a)[0], act, m.grouped_gemm(act, b, d.layout.exp_off),
                m.moe_decode(xd, id_, td, a, b))

    want = [layer(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(layer(*sets[i]))
    torch.cuda.synchronize()
    n = [int(s[5].layout.exp_off[-1]) for s in sets]
    for i in range(2):
        for g in got[i]:
            for j, (u, v) in enumerate(zip(g, want[i])):
                live = slice(0, n[i]) if j in (1, 2) else slice(None)
                assert torch.equal(u[live], v[live]), (i, j)


def test_graph_replays_follow_the_inputs():
    """Both layers captured; every replay against the eager result on new
    tokens and a new routing, eager calls in between."""
    say("graph replays")
    m = epx()
    T, K, E, h, f = 24, 4, 16, 256, 128
    x, idx, top, w13, w2 = _layer_inputs(T, K, E, h, f, 151)
    xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
    (aq, asc), (bq, bsc) = m.quantize_weights(a), m.quantize_weights(b)
    buf = m.alloc_ll(E, 1, T, h, T, K, True, DEV)

    def both():
        few = m.moe_decode(xd, id_, td, a, b)
        d = m.ll_dispatch(xd, id_, E, 4, 0, T, R_buf=1, fp8=True, buf=buf)
        act, act_s = m.ll_grouped_swiglu(d.ll_x, aq, d.ll_count, T, d.ll_scales, asc)
        y = m.ll_grouped_gemm(act, bq, d.ll_count, T, act_s, bsc)
        return few, m.combine(y, d.pos_ll, td)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for r in range(4):
        x2, idx2, top2, _, _ = _layer_inputs(T, K, E, h, f, 160 + r)
        xd.copy_(x2)
        id_.copy_(idx2)
        td.copy_(top2)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        eager = both()
        torch.cuda.synchronize()
        for u, v in zip(kept, eager):
            assert torch.equal(u, v), f"replay {r}"
    assert m.get_error() == 0
