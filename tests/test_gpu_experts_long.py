"""The experts' arithmetic over many channels, on sums that are exact
(tests/_experts_exact.py): every step of every tile height counts once, with
its own scales, up to the largest K, h and f; and the layer in FP8 against the
same roundings made on the CPU."""
import numpy as np
import pytest
import torch

import _experts as X
import _experts_exact as XE
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


def _check(gated, out, out_s, rows_of, x, xs, w, ws):
    for e, r in enumerate(rows_of):
        if len(r) == 0:
            continue
        r = torch.as_tensor(r, dtype=torch.long)
        y = XE.sums(x[r], None if xs is None else xs[r], w[e], None if ws is None else ws[e])
        assert (y.float().double() == y).all()
        got = out[r.to(DEV)]
        if gated:
            XE.assert_activation(got, None if out_s is None else out_s[r.to(DEV)], y, f"expert {e}")
        else:
            XE.assert_sums(got, y, f"expert {e}")


def _outputs(gated, fp8, n, N):
    if gated and fp8:
        return canary((n, N), torch.uint8), canary((n, X.stride(N)), torch.float32)
    return canary((n, N), torch.bfloat16), None


# Rows of the experts by the tile height that their average takes.
COUNTS = {
    "64": [5, 0, 17, 64],
    "128": [70, 97, 60],          # FP8; bf16 rows take 160 here too
    "160": [120, 161, 40, 90],
    "256": [300, 511],
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("which", list(COUNTS))
@pytest.mark.parametrize("K", [1152, 20608, 65536])
def test_grouped_long_channels(K, which, gated, fp8):
    if K == 65536 and which == "256":
        K -= 128 if fp8 else 8                # an odd number of steps; bf16: a partial last one
    say(f"long channels K={K} {which} gated={gated} fp8={fp8}")
    N = 128 if gated else 264
    off = X.offsets(COUNTS[which])
    n, L = int(off[-1]), len(off) - 1
    x, xs, w, ws = XE.operands(fp8, n, L, 2 * N if gated else N, K, 21 + K % 11,
                               XE.UNIT if gated else 0)
    out, out_s = _outputs(gated, fp8, n, N)
    xd, xsd, wd, wsd, od = gpu(x, xs, w, ws, torch.from_numpy(off))
    if gated:
        epx().grouped_swiglu(xd, wd, od, xsd, wsd, out=out, out_scales=out_s)
    else:
        epx().grouped_gemm(xd, wd, od, xsd, wsd, out=out)
    assert epx().get_error() == 0
    _check(gated, out, out_s, [np.arange(off[e], off[e + 1]) for e in range(L)], x, xs, w, ws)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R,cap", [(1, 30), (1, 100), (1, 200), (8, 30)])
def test_ll_grouped_long_channels(R, cap, gated, fp8):
    say(f"long channels, regions R={R} cap={cap} gated={gated} fp8={fp8}")
    L, K, N = 3, 20608, 128
    rng = np.random.default_rng(31)
    counts = rng.integers(-1, cap + 1, L * R).astype(np.int32)
    counts[0] = cap
    n = L * R * cap
    live = (np.arange(cap)[None, :] < counts[:, None]).reshape(-1)
    x, xs, w, ws = XE.operands(fp8, n, L, 2 * N if gated else N, K, 32, XE.UNIT if gated else 0)
    out, out_s = _outputs(gated, fp8, n, N)
    xd, xsd, wd, wsd, cd = gpu(x, xs, w, ws, torch.from_numpy(counts))
    if gated:
        epx().ll_grouped_swiglu(xd, wd, cd, cap, xsd, wsd, out=out, out_scales=out_s)
    else:
        epx().ll_grouped_gemm(xd, wd, cd, cap, xsd, wsd, out=out)
    assert epx().get_error() == 0
    rows = [np.flatnonzero(live[e * R * cap:(e + 1) * R * cap]) + e * R * cap for e in range(L)]
    _check(gated, out, out_s, rows, x, xs, w, ws)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_grouped_wide_results(gated, fp8):
    """65536 columns: every one is computed and every scale in its place."""
    N, K, L = 65536, 256, 2
    say(f"wide results gated={gated} fp8={fp8}")
    off = X.offsets([3, 18])
    x, xs, w, ws = XE.operands(fp8, 21, L, 2 * N if gated else N, K, 41, 3 if gated else 0)
    out, out_s = _outputs(gated, fp8, 21, N)
    xd, xsd, wd, wsd, od = gpu(x, xs, w, ws, torch.from_numpy(off))
    if gated:
        epx().grouped_swiglu(xd, wd, od, xsd, wsd, out=out, out_scales=out_s)
    else:
        epx().grouped_gemm(xd, wd, od, xsd, wsd, out=out)
    assert epx().get_error() == 0
    _check(gated, out, out_s, [np.arange(off[e], off[e + 1]) for e in range(L)], x, xs, w, ws)


# --------------------------------------------------------- few-token layer

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,h", [(5, 20608), (3, 65536), (40, 20608)])
def test_moe_decode_long_h(T, h, fp8):
    """One expert a token, and w2 picks one activation a column with weight
    1: the activation, rounded to bf16, then halved (exact)."""
    say(f"decode T={T} h={h} fp8={fp8}")
    E, f = 2, 128
    x, _, w13, s13 = XE.operands(fp8, T, E, 2 * f, h, 51, XE.UNIT)
    if fp8:
        x = XE.signs((T, h), torch.Generator().manual_seed(52)).to(torch.bfloat16)
    pick = torch.zeros((E, h, f))
    pick[:, torch.arange(h), torch.arange(h) % f] = 1.0
    w2 = pick.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else pick.to(torch.bfloat16)
    s2 = torch.ones((E, -(-h // 128), f // 128)) if fp8 else None
    idx = torch.arange(T)[:, None] % E
    top = torch.full((T, 1), 0.5)
    xd, id_, td, a, sa, b, sb = gpu(x, idx, top, w13, s13, w2, s2)
    got = epx().moe_decode(xd, id_, td, a, b, sa, sb)
    assert epx().get_error() == 0
    for e in range(E):
        t = torch.nonzero(idx[:, 0] == e)[:, 0]
        y = XE.sums(x[t], None, w13[e], None if s13 is None else s13[e])
        assert (y.float().double() == y).all()
        wide = got[t.to(DEV)].float()[:, :h - h % f].view(len(t), -1, f) * 2
        assert (wide == wide[:, :1]).all()        # the same activation in every place
        XE.assert_activation(wide[:, 0], None, y, f"expert {e}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,K,E,f", [(5, 1, 2, 20608), (3, 2, 2, 65536), (40, 2, 3, 20608),
                                     (20, 6, 12, 4096)])
def test_moe_decode_long_f(T, K, E, f, fp8):
    """Gates of 32, whose silu is 32 in fp32 (1 + exp(-32) is 1), and up values
    that make every activation -1, 0 or 1 (FP8: times 1/2, 1 or 2): the second
    product's sums, times powers of two, are exact."""
    say(f"decode T={T} K={K} E={E} f={f} fp8={fp8}")
    h = 128
    rng = np.random.default_rng(61)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int64))
    top = torch.from_numpy((2.0 ** rng.integers(-2, 1, (T, K))).astype(np.float32))
    x = torch.zeros((T, h))
    x[:, 0] = 1.0
    x[torch.arange(T), 1 + torch.arange(T)] = 1.0
    _, _, up, su = XE.operands(fp8, 1, E, f, h, 62)
    _, _, w2, s2 = XE.operands(fp8, 1, E, h, f, 63)
    one = torch.zeros((E, f, h))
    one[:, :, 0] = 32.0
    if fp8:
        up[:, :, 0] = 0
        w13 = torch.cat([one.to(torch.float8_e4m3fn).view(torch.uint8), up], 1)
        s13 = torch.cat([torch.ones_like(su), su / 32], 1)
    else:
        up[:, :, 0] = 0.0
        w13, s13 = torch.cat([one.to(torch.bfloat16), up / 32], 1), None
    x = x.to(torch.bfloat16)
    xd, id_, td, a, sa, b, sb = gpu(x, idx, top, w13, s13, w2, s2)
    got = epx().moe_decode(xd, id_, td, a, b, sa, sb)
    assert epx().get_error() == 0
    want = torch.zeros((T, h), dtype=torch.float64)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        act = XE.sums(x[t], None, w13[e], None if s13 is None else s13[e])
        act = act[:, :f] * act[:, f:]
        y = act @ X.weights64(w2[e], None if s2 is None else s2[e]).T
        want.index_add_(0, t, top[t, k].double()[:, None] * y)
    assert (want.float().double() == want).all()
    XE.assert_sums(got, want, "decode")


# ----------------------------------------------------------- layer in FP8

@pytest.mark.parametrize("ll", [False, True])
def test_fp8_layer_against_the_same_roundings(ll):
    """dispatch to combine, and the few-token layer, with rows, weights and
    activations rounded to e4m3 on the CPU by the same formulas. What is left
    are the roundings of y and of the result to bf16, each at most 2^-8 of its
    value and independent, so sqrt(2) 2^-8 of the norm at most (the few-token
    layer: of the activations and of the result), the FP8 product's cuts (some
    1e-5 of the magnitudes), and the few codes whose quotient lies within a
    fp32 rounding of a border. Some 2^-9 is expected, 2 * 2^-8 allowed."""
    say(f"fp8 layer ll={ll}")
    m = epx()
    T, K, E, R, h, f = 150, 4, 16, 4, 512, 384
    rng = np.random.default_rng(71)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int64))
    idx[torch.from_numpy(rng.random((T, K)) < 0.1)] = -1
    top = torch.from_numpy(rng.random((T, K)).astype(np.float32))
    x = X.randn((T, h), 72)
    w13, w2 = X.randn((E, 2 * f, h), 73, h ** -0.5), X.randn((E, h, f), 74, f ** -0.5)
    xd, id_, td, a, b = gpu(x, idx, top, w13, w2)
    (a, sa), (b, sb) = m.quantize_weights(a), m.quantize_weights(b)
    if ll:
        d = m.ll_dispatch(xd, id_, E, R, 0, T, R_buf=1, fp8=True)
        act, act_s = m.ll_grouped_swiglu(d.ll_x, a, d.ll_count, T, d.ll_scales, sa)
        y = m.ll_grouped_gemm(act, b, d.ll_count, T, act_s, sb)
        out = m.combine(y, d.pos_ll, td)
    else:
        d = m.dispatch(xd, id_, td, E, R, fp8=True)
        act, act_s = m.grouped_swiglu(d.recv_x, a, d.layout.exp_off, d.recv_scales, sa)
        y = m.grouped_gemm(act, b, d.layout.exp_off, act_s, sb)
        out = m.combine(y, d.pos_exp, td)
    few = m.moe_decode(xd[:64], id_[:64], td[:64], a, b, sa, sb)
    assert m.get_error() == 0

    q13, s13 = XE.quantized_weights(w13.float())
    q2, s2 = XE.quantized_weights(w2.float())
    rows = XE.values(*XE.quantized_rows(x.float()))
    want, want_few = (torch.zeros((T, h), dtype=torch.float64) for _ in range(2))
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        v13, v2 = X.weights64(q13[e], s13[e]), X.weights64(q2[e], s2[e])
        tw = top[t, k].double()[:, None]
        act64, _ = XE.activation(rows[t] @ v13.T)
        want.index_add_(0, t, tw * (XE.values(*XE.quantized_rows(act64.float())) @ v2.T))
        act64, _ = XE.activation(x[t].double() @ v13.T)
        want_few.index_add_(0, t, tw * (act64 @ v2.T))
    rel = lambda got, ref: float((got.double().cpu() - ref).norm() / ref.norm())  # noqa: E731
    say(f"relative error {rel(out, want):.5f}, few tokens {rel(few, want_few[:64]):.5f}")
    assert rel(out, want) <= 2 * X.BF16
    assert rel(few, want_few[:64]) <= 2 * X.BF16


def test_gates_where_silu_leaves_fp32():
    """Gates around -88 beside huge up values: the stated error down to where
    the quotient is said to be zero, zero from there on."""
    say("gates around -88")
    gates = torch.tensor([-60.0, -80.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -100.0, -3e38])
    n, K, N = len(gates), 8, 8
    x = torch.zeros((n, K))
    x[:, 0], x[:, 1] = gates, 1.0
    w = torch.zeros((1, 2 * N, K))
    w[0, :N, 0], w[0, N:, 1] = 1.0, 2.0 ** 100
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    act, _ = epx().grouped_swiglu(gpu(x.to(torch.bfloat16)), gpu(w.to(torch.bfloat16)), off)
    assert epx().get_error() == 0
    act = act.cpu().float()
    assert (act[4:] == 0).all(), act[:, 0]
    g = x[:4, :1].to(torch.bfloat16).double()
    a = g / (1 + torch.exp(-g)) * 2.0 ** 100
    a, tol = a.expand(4, N), ((8 + g.abs()) * X.U32 * a.abs()).expand(4, N)
    X.assert_close(act[:4], a, tol + X.BF16 * (a.abs() + tol), "gates above -87.3")
