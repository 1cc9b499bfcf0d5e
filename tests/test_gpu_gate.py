"""The residual norm, the router's choice, the balance loss and the gradients
on the GPU, against 64-bit results on the CPU within derived bounds
(tests/_gate.py)."""
import ctypes

import numpy as np
import pytest
import torch

import _experts as X
import _gate as G
import synth
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


def is_canary(t):
    return bool((t.contiguous().view(torch.uint8) == CANARY).all())


def flags(*bits):
    """The device error word is exactly the sum of the bits."""
    assert epx().get_error() == sum(bits)


def same(a, b, what):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 8), (3, 136), (2, 1016), (5, 1024), (7, 1032), (300, 1416), (4, 4096),
               (6, 7168), (2, 16384), (3, 16392), (2, 32768)]


def _norm_case(T, h, residual, bf16, fp8, w_dtype, seed=50, eps=1e-6):
    x, r = G.rows((T, h), seed), G.rows((T, h), seed + 1, 3.0) if residual else None
    x[:, ::97] *= 50
    w = (1.0 + 0.1 * torch.randn(h, generator=G.gen(seed + 2))).to(w_dtype)
    say(f"rms_norm T={T} h={h} residual={residual} bf16={bf16} fp8={fp8} weight={w_dtype}")
    # rows behind the T stay as they were
    full = epx().alloc_norm(T + 1, h, residual, bf16, fp8, DEV)
    for t in vars(full).values():
        if t is not None:
            t.view(torch.uint8).fill_(CANARY)
    buf = epx().Normed(**{k: t if t is None else t[:T] for k, t in vars(full).items()})
    epx().rms_norm(gpu(x), gpu(w), eps, residual=gpu(r), buf=buf)
    flags()
    assert all(is_canary(t[T]) for t in vars(full).values() if t is not None)
    v = x.double() if r is None else x.double() + r.double()
    y, inv = G.norm(v, w.double(), eps)
    tol = G.norm_tol(y, v, inv, w.double())
    if residual:
        same(buf.residual.cpu(), (x.float() + r.float()).to(torch.bfloat16), "residual")
    if bf16:
        X.assert_close(buf.out, y, tol + G.BF16 * (y.abs() + tol), "out")
    if fp8:
        X.assert_codes(buf.codes, buf.scales, y, tol, "rows")


@pytest.mark.parametrize("T,h", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, h, residual):
    _norm_case(T, h, residual, True, False, torch.float32 if residual else torch.bfloat16)


@pytest.mark.parametrize("T,h", [(1, 128), (3, 384), (5, 1024), (2, 1152), (9, 4224), (6, 7168),
                                 (2, 16384), (2, 16512), (1, 32768)])
@pytest.mark.parametrize("bf16", [False, True])
def test_norm_fp8(T, h, bf16):
    _norm_case(T, h, bf16, bf16, True, torch.bfloat16 if bf16 else torch.float32)


@pytest.mark.parametrize("h,fp8", [(8, False), (128, True), (136, False), (256, True), (264, False)])
def test_norm_many_rows(h, fp8):
    _norm_case(2601, h, True, True, fp8, torch.bfloat16)


def test_norm_eps_and_zero_rows():
    """eps counts where the row is small; a row of zeros gives zeros and the least scale."""
    x = G.rows((4, 256), 60, 1e-4)
    x[1] = 0
    w = torch.ones(256)
    b = epx().rms_norm(gpu(x), gpu(w), 1e-3, fp8=True)
    y, inv = G.norm(x.double(), w.double(), 1e-3)
    tol = G.norm_tol(y, x.double(), inv, w.double())
    X.assert_close(b.out, y, tol + G.BF16 * (y.abs() + tol), "out")
    X.assert_codes(b.codes, b.scales, y, tol, "rows")
    assert not b.out[1].any() and not b.codes[1].any()
    assert (b.scales[1, :2] == torch.tensor(1e-4) / 448).all()
    z = epx().rms_norm(gpu(x), gpu(w), 0.0)
    assert z.out[1].isnan().all()                     # 0 / 0, as the formula says
    flags()


def test_norm_non_finite_rows():
    """An Inf or NaN makes its own row NaN (codes 0x7F, the least scale) and no other."""
    x = G.rows((5, 512), 61)
    x[1, 3], x[3, 511] = float("inf"), float("nan")
    w = torch.ones(512, dtype=torch.bfloat16)
    b = epx().rms_norm(gpu(x), gpu(w), fp8=True)
    ok = [0, 2, 4]
    y, inv = G.norm(x[ok].double(), w.double(), 1e-6)
    tol = G.norm_tol(y, x[ok].double(), inv, w.double())
    X.assert_close(b.out[ok], y, tol + G.BF16 * (y.abs() + tol), "out")
    X.assert_codes(b.codes[ok], b.scales[ok], y, tol, "rows")
    assert b.out[3].isnan().all() and b.out[1, 3].isnan()
    assert not b.out[1, :3].any()                     # finite / inf
    assert (b.codes[3] & 0x7F == 0x7F).all() and b.codes[1, 3] & 0x7F == 0x7F
    # a weight that is not finite keeps to its channel's group
    w[130] = float("inf")
    b = epx().rms_norm(gpu(x[ok]), gpu(w), fp8=True)
    y[:, 130] = 0
    keep = [c for c in range(512) if not 128 <= c < 256]
    got = b.codes.view(torch.float8_e4m3fn).double().cpu()
    assert (got[:, keep].abs() <= 448).all() and torch.isinf(b.scales[:, 1]).all()
    assert torch.isfinite(b.scales[:, [0, 2, 3]]).all() and torch.isinf(b.out[:, 130]).all()
    flags()


def test_norm_residual_rounds_everywhere():
    """Sums of every pair of exponents, denormal ones too, rounded nearest even."""
    bits = torch.randint(0, 1 << 16, (2, 64, 4096), generator=G.gen(64)).to(torch.int16)
    x, r = bits.view(torch.bfloat16)
    x, r = (torch.where(t.isfinite(), t, torch.zeros_like(t)) for t in (x, r))
    # neighbours in size, so that both count: r's exponent within 10 of x's
    e = ((x.view(torch.int16).int() >> 7) & 0xFF) + torch.randint(-10, 11, x.shape, generator=G.gen(65))
    near = (r.view(torch.int16).int() & 0x807F) | (e.clamp(0, 254) << 7)
    r[::2] = near.to(torch.int16).view(torch.bfloat16)[::2]
    b = epx().rms_norm(gpu(x), torch.ones(4096, device=DEV), residual=gpu(r))
    same(b.residual.cpu(), (x.float() + r.float()).to(torch.bfloat16), "residual")
    assert (b.residual.float().abs() < 1e-38).any() and (b.residual != 0).any()
    flags()


def test_norm_in_place():
    """The sum over the residual, the normed rows over x."""
    x, r, w = gpu(G.rows((33, 1416), 62), G.rows((33, 1416), 63), torch.ones(1416))
    want = epx().rms_norm(x, w, residual=r)
    a, b = x.clone(), r.clone()
    epx().rms_norm(a, w, residual=b, buf=epx().Normed(out=a, residual=b))
    same(a, want.out, "out")
    same(b, want.residual, "residual")


@pytest.mark.parametrize("T,h", NORM_SHAPES + [(1500, 200), (2049, 64), (9001, 128), (4100, 256), (5000, 8), (1300, 264)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_backward(T, h, residual):
    x, dout = G.rows((T, h), 70), G.rows((T, h), 71, 0.02)
    x[:, ::97] *= 50
    dres = G.rows((T, h), 72, 0.02) if residual else None
    w = (1.0 + 0.1 * torch.randn(h, generator=G.gen(73))).to(
        torch.bfloat16 if residual else torch.float32)
    say(f"rms_norm_backward T={T} h={h} residual={residual}")
    out = canary((T + 1, h), torch.bfloat16)
    dw = canary(h + 4, torch.float32)
    epx().rms_norm_backward(gpu(dout), gpu(x), gpu(w), 1e-6, dresidual=gpu(dres),
                            out=(out[:T], dw[:h]))
    flags()
    assert is_canary(out[T]) and is_canary(dw[h:])
    dx, tol, ref_w, tol_w = G.norm_backward(dout.double(), x.double(), w.double(), 1e-6,
                                            None if dres is None else dres.double())
    X.assert_close(out[:T], dx, tol + G.BF16 * (dx.abs() + tol), "dx")
    X.assert_close(dw[:h], ref_w, tol_w, "dweight")


@pytest.mark.parametrize("h,T", [(8, (1 << 27) + 5), (264, (1 << 25) + 3)])
def test_norm_more_rows_than_a_launch(h, T):
    """Rows beyond the 2^31 threads of one launch, and offsets beyond 2^32 bytes."""
    base = G.rows((1 << 12, h), 79)
    say(f"rms_norm T={T} h={h}")
    x = torch.empty((T, h), dtype=torch.bfloat16, device=DEV)
    x[:1 << 12] = gpu(base)
    done = 1 << 12
    while done < T:                            # the same rows again and again
        n = min(done, T - done)
        x[done:done + n] = x[:n]
        done += n
    b = epx().rms_norm(x, torch.ones(h, device=DEV))
    torch.cuda.synchronize()
    flags()
    y, inv = G.norm(base.double(), torch.ones(h).double(), 1e-6)
    tol = G.norm_tol(y, base.double(), inv, torch.ones(h).double())
    for r in (0, (1 << 31) // (16 if h == 8 else 64) - 2, T - 3, 1 << 24):
        at = torch.arange(r, min(r + 3, T)) % (1 << 12)
        X.assert_close(b.out[r:r + 3], y[at], tol[at] + G.BF16 * (y[at].abs() + tol[at]), f"row {r}")
    del x, b
    torch.cuda.empty_cache()


def test_norm_backward_in_place_and_empty():
    x, dout, dres, w = gpu(G.rows((9, 264), 74), G.rows((9, 264), 75), G.rows((9, 264), 76),
                           torch.ones(264))
    dx, dw = epx().rms_norm_backward(dout, x, w, dresidual=dres)
    for over in (0, 1):
        a, b = dout.clone(), dres.clone()
        out = (b if over else a, torch.empty_like(dw))
        epx().rms_norm_backward(a, x, w, dresidual=b, out=out)
        same(out[0], dx, "dx")
        same(out[1], dw, "dweight")
    _, dw = epx().rms_norm_backward(dout[:0], x[:0], w)
    assert not dw.any()
    assert epx().rms_norm(x[:0], w).out.shape == (0, 264)
    flags()


@pytest.mark.parametrize("h", [8, 64, 128, 200, 256])
@pytest.mark.parametrize("T", [1, 33, 2601])
def test_norm_in_place_narrow(h, T):
    """Rows that go several to a wave, over their own inputs, forward and backward."""
    m = epx()
    x, r, s, w = gpu(G.rows((T, h), 191), G.rows((T, h), 192), G.rows((T, h), 193),
                     1 + 0.1 * torch.randn(h, generator=G.gen(194)))
    say(f"rms_norm and its gradient in place T={T} h={h}")
    want = m.rms_norm(x, w, residual=r)
    for swap in (False, True):                 # the sum over the residual or over x
        a, b = x.clone(), r.clone()
        to = m.Normed(out=b, residual=a) if swap else m.Normed(out=a, residual=b)
        m.rms_norm(a, w, residual=b, buf=to)
        same(to.out, want.out, "out")
        same(to.residual, want.residual, "residual")
    a = x.clone()
    m.rms_norm(a, w, buf=m.Normed(out=a))
    same(a, m.rms_norm(x, w).out, "out alone")
    dx, dw = m.rms_norm_backward(r, x, w, dresidual=s)
    for over in (0, 1):
        a, b = r.clone(), s.clone()
        out = (b if over else a, torch.empty_like(dw))
        m.rms_norm_backward(a, x, w, dresidual=b, out=out)
        same(out[0], dx, "dx")
        same(out[1], dw, "dweight")
    flags()


# ---------------------------------------------------------------- router

def _logits(T, E, seed, scale=1.5):
    return torch.randn((T, E), generator=G.gen(seed)) * scale


def _route(l, K, scoring="softmax", bias=None, G_=1, top=1, normalize=True, scale=1.0, mask=None,
           bits=()):
    T, E = l.shape
    idx, w = canary((T + 1, K), torch.int64), canary((T + 1, K), torch.float32)
    say(f"route T={T} E={E} K={K} {scoring} bias={bias is not None} groups={G_}/{top} "
        f"normalize={normalize}")
    epx().route(gpu(l), K, scoring, gpu(bias), G_, top, normalize, scale, gpu(mask),
                out=(idx[:T], w[:T]))
    flags(*bits)
    assert is_canary(idx[T]) and is_canary(w[T])
    clean = torch.where(l < torch.inf, l, -torch.inf)
    if bias is not None:
        bias = torch.where(bias < torch.inf, bias, -torch.inf)
    ri, rw, tol = G.route(clean, K, scoring, bias, G_, top, normalize, scale, mask)
    bad = (idx[:T].cpu() != ri).any(1).nonzero()
    assert not len(bad), (f"{len(bad)} tokens, first {int(bad[0])}: "
                          f"{idx[int(bad[0])].tolist()} for {ri[int(bad[0])].tolist()}")
    X.assert_close(w[:T], rw, tol, "topk_weights")


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (7, 3), (8, 2), (63, 6), (64, 8), (65, 5),
                                 (100, 32), (128, 1), (160, 6), (255, 8), (256, 8), (257, 16),
                                 (384, 8), (512, 10), (512, 32), (300, 31), (32, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route(E, K, scoring, normalize):
    _route(_logits(37, E, E), K, scoring, None, 1, 1, normalize, 1.0 if normalize else 2.5)
    bias = torch.randn(E, generator=G.gen(E + 1)) * 0.1
    _route(_logits(37, E, E + 2), K, scoring, bias, 1, 1, normalize, 2.5 if normalize else 1.0)


@pytest.mark.parametrize("E,G_,top,K", [(8, 2, 1, 3), (8, 8, 3, 3), (64, 8, 3, 6), (72, 8, 2, 9),
                                        (96, 3, 2, 8), (160, 8, 3, 6), (256, 8, 4, 8),
                                        (256, 64, 5, 8), (256, 4, 4, 8), (320, 5, 1, 32),
                                        (512, 16, 4, 8), (512, 32, 7, 20), (64, 8, 1, 10),
                                        (100, 50, 20, 30), (12, 3, 1, 4), (512, 2, 1, 16)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(E, G_, top, K, scoring, biased):
    bias = torch.randn(E, generator=G.gen(E + 3)) * 0.1 if biased else None
    _route(_logits(41, E, E + 4), K, scoring, bias, G_, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G_,top", [(1, 1), (8, 3)])
def test_route_ties(scoring, biased, G_, top):
    """Logits and biases of a few values, zeros of both signs: the lowest expert first."""
    E = 256
    l = torch.round(_logits(60, E, 80)) * 0.5
    l[::3] = torch.where(torch.rand((20, E), generator=G.gen(81)) < 0.5, 0.0, -0.0)
    bias = torch.round(torch.randn(E, generator=G.gen(82))) * 0.25 if biased else None
    _route(l, 8, scoring, bias, G_, top)
    _route(torch.zeros((3, E)), 8, scoring, None if bias is None else torch.zeros(E), G_, top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G_,top", [(1, 1), (4, 2)])
def test_route_near_ties(scoring, G_, top):
    """Biased scores that differ by less than fp32 can tell: the 64-bit order.
    The biases take back what the logits give, up to 1e-8 or so."""
    T, E = 64, 128
    l = _logits(1, E, 83, 0.5)
    s = G.scores(l.double(), scoring)
    bias = (0.6 - s[0]).float()
    near = l.repeat(T, 1)
    for t in range(1, T):     # the last place of some logits
        step = torch.randint(-1, 2, (E,), generator=G.gen(84 + t))
        near[t] = torch.nextafter(near[t], near[t] + step)
    key = (G.scores(near.double(), scoring) + bias.double()).sort(1, descending=True).values
    assert (key[:, :8] - key[:, 1:9]).median() < 2e-8          # hard, and not of equal keys
    assert (key[:, :8] - key[:, 1:9]).min() > 0
    _route(near, 8, scoring, bias, G_, top)


def test_route_saturated_scores():
    """Sigmoids that are one to fp32 still order, as do logits whose scores
    underflow; normalized weights of tiny scores are whole."""
    l = torch.cat([torch.linspace(15, 36, 32), torch.linspace(-300, -200, 32)])[None].repeat(8, 1)
    l = torch.gather(l, 1, torch.stack([torch.randperm(64, generator=G.gen(90 + i))
                                        for i in range(8)]))
    _route(l, 8, "sigmoid")
    _route(l, 8, "sigmoid", bias=torch.zeros(64))
    # some of the large ones, the others of the 32 far below them
    _route(torch.where(l > 20.0, -torch.inf, l), 32, "softmax")
    _route(l.clamp(max=-200.0), 32, "sigmoid")
    _route(l.clamp(max=-200.0), 32, "softmax", normalize=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G_,top,K", [(40, 1, 1, 6), (256, 1, 1, 8), (256, 8, 3, 8)])
def test_route_masked_experts(scoring, E, G_, top, K):
    """-inf logits and biases: never chosen, no share; rows that leave fewer than
    K, one or no expert; the lowest finite value is a live logit."""
    l = _logits(24, E, 91)
    l[torch.rand(l.shape, generator=G.gen(92)) < 0.6] = -torch.inf
    l[3] = -torch.inf
    l[4] = -torch.inf
    l[4, E - 1] = 2.0
    l[5, 1:] = -torch.inf
    l[6] = torch.finfo(torch.float32).min
    l[7, :3] = torch.finfo(torch.float32).min
    bias = torch.zeros(E)
    bias[::5] = -torch.inf
    for b in (None, bias):
        for normalize in (True, False):
            _route(l, K, scoring, b, G_, top, normalize)


def test_route_flags_bad_logits():
    l = _logits(9, 64, 93)
    l[2, 5], l[3, 7] = torch.nan, torch.inf
    _route(l, 6, bits=(16,))
    _route(l, 6, "sigmoid", bits=(16,))
    bias = torch.zeros(64)
    bias[11], bias[60] = torch.nan, torch.inf
    _route(_logits(9, 64, 94), 6, "sigmoid", bias=bias, bits=(16,))


def test_route_mask_and_rows():
    """Padded tokens (whatever their logits hold), rows that start off a 16-byte
    border, one token, none."""
    l = _logits(70, 100, 95)
    mask = torch.rand(70, generator=G.gen(96)) < 0.7
    l[~mask] = torch.nan
    _route(l, 7, mask=mask)
    _route(l, 7, mask=mask.to(torch.uint8), scoring="sigmoid")
    for E in (100, 256, 36):
        store = torch.zeros(5 * E + 1)
        store[1:] = _logits(5, E, 97).view(-1)
        d = gpu(store)[1:].view(5, E)
        idx, w = epx().route(d, 4)
        ri, rw, tol = G.route(store[1:].view(5, E), 4, "softmax")
        assert torch.equal(idx.cpu(), ri)
        X.assert_close(w, rw, tol, "topk_weights")
    _route(_logits(1, 256, 98), 8)
    idx, w = epx().route(gpu(_logits(0, 16, 99)), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    flags()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G_", [(64, 8), (72, 8), (256, 64), (12, 3), (96, 3)])
def test_route_groups_of_largest_and_lowest_biases(scoring, E, G_):
    """Biases at the ends of fp32's range, whose sums of two are beyond it: groups
    that are masked by the lowest value are live and come in their order, those of
    the largest are told apart."""
    least, most, per = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max, E // G_
    l = _logits(11, E, 185)
    bias = torch.full((E,), least)
    bias[2 * per:3 * per] = 0.0                # one group; the others follow, lowest first
    _route(l, min(per + 3, 32), scoring, bias, G_, min(3, G_))
    bias[2 * per:3 * per] = least              # nothing but masks
    _route(l, 2, scoring, bias, G_, 2)
    bias = torch.zeros(E)
    bias[0:per] = 0.7 * most                   # twice 0.7 against 1 + 0.5 and 0.6 + 0.6
    bias[per], bias[per + 1] = most, 0.5 * most
    bias[2 * per:2 * per + 2] = 0.6 * most
    _route(l, 2, scoring, bias, G_, 1)
    _route(l, 4, scoring, bias, G_, 2)
    bias[:] = -torch.inf                       # one live expert in a group: it alone
    bias[per - 1], bias[per], bias[per + 1] = least, least, least
    _route(l, 3, scoring, bias, G_, 1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [-100.0, -1e9, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("G_,top", [(1, 1), (8, 3)])
def test_route_finite_masks(scoring, mask, G_, top):
    """Experts masked by a finite bias: last, not out."""
    E = 64
    l, bias = _logits(21, E, 187), torch.zeros(E)
    bias[torch.randperm(E, generator=G.gen(188))[:20]] = mask
    _route(l, 8, scoring, bias, G_, top)
    bias[8:] = mask                            # fewer than K without a mask
    _route(l, 12, scoring, bias, G_, top)


@pytest.mark.parametrize("scale", [1e-4, 25.0, 300.0])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_narrow_and_wide_logits(scoring, scale):
    """Logits nearer than the fixed point tells, and chosen ones outside its window."""
    l = _logits(40, 256, 189, scale)
    _route(l, 8, scoring)
    _route(l, 16, scoring, normalize=False)
    _route(l, 8, scoring, torch.randn(256, generator=G.gen(190)) * 0.1, 8, 4)


# ---------------------------------------------------------- balance loss

def _choose(T, E, K, seed, drop=0.1):
    idx = torch.from_numpy(synth.random_routing(T, K, E, seed, drop)) if T else \
        torch.zeros((0, K), dtype=torch.int64)
    if T > 3:
        idx[T // 2] = -1
    return idx


def _balance(l, idx, scoring, off=None, bits=(), ref_off=None):
    T, E = l.shape
    S = 1 if off is None else len(off) - 1
    say(f"balance_loss T={T} E={E} K={idx.shape[1]} S={S} {scoring}")
    b = epx().alloc_balance(S, E, DEV)
    for t in vars(b).values():
        t.view(torch.uint8).fill_(CANARY)
    offd = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    ws = canary(epx().balance_workspace(T, E, S) + 16, torch.uint8)
    epx().balance_loss(gpu(l), gpu(idx), scoring, offd, out=b, workspace=ws[:-16])
    flags(*bits)
    assert is_canary(ws[-16:])
    clean = torch.where(l < torch.inf, l, -torch.inf)
    loss, counts, probs, n, rel = G.balance(clean, idx, scoring, off)
    assert torch.equal(b.counts.cpu(), counts) and torch.equal(b.num_tokens.cpu(), n)
    X.assert_close(b.probs, probs, rel * probs + G.TINY, "probs")
    # counts * probs: a thread's share, 6 steps of a wave, 16 waves, S sequences
    X.assert_close(b.loss, torch.tensor([loss]).double(),
                   torch.tensor([(rel + (2 + 6 + 16 + S + 4) * G.U) * loss + G.TINY]), "loss")
    return b, offd


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (63, 8, 2), (64, 64, 6), (65, 65, 3),
                                   (200, 128, 32), (300, 160, 6), (513, 256, 8), (130, 512, 10)])
def test_balance(T, E, K, scoring):
    _balance(_logits(T, E, 100 + E), _choose(T, E, K, 101), scoring)


@pytest.mark.parametrize("T,S", [(70, 70000), (20000, 9000)])
def test_balance_many_sequences(T, S):
    """More sequences than tokens or blocks, most of them empty."""
    g = G.gen(109)
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g)).values
    off = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([T])])
    l, idx = _logits(T, 16, 108), _choose(T, 16, 2, 107)
    say(f"balance_loss T={T} S={S}")
    b = epx().balance_loss(gpu(l), gpu(idx), "softmax", gpu(off.to(torch.int32)))
    flags()
    seq = torch.searchsorted(off, torch.arange(T), right=True) - 1
    p, seen = torch.softmax(l.double(), 1), (idx >= 0).any(1)
    n = torch.zeros(S, dtype=torch.int64).index_add_(0, seq, seen.long())
    counts = torch.zeros((S, 17), dtype=torch.int64)
    counts.index_put_((seq[:, None].expand_as(idx), torch.where(idx >= 0, idx, 16)),
                      torch.ones_like(idx), accumulate=True)
    probs = torch.zeros((S, 16), dtype=torch.float64).index_add_(0, seq[seen], p[seen])
    probs = probs / n.clamp(min=1)[:, None]
    assert torch.equal(b.counts.cpu().long(), counts[:, :16])
    assert torch.equal(b.num_tokens.cpu().long(), torch.cat([n, (n > 0).sum().view(1)]))
    # a sequence has few tokens here: the scores' own errors and some 20 additions
    rel = (2 * (4 + float(G.spread(l).max())) + 14 + 6 + 64) * G.U
    X.assert_close(b.probs, probs, rel * probs + G.TINY, "probs")
    each = (counts[:, :16] * probs).sum(1) * 16 / (2 * n.clamp(min=1))
    loss = each[n > 0].mean()
    # the losses of S sequences in a thread's turn, a block's threads, its waves
    X.assert_close(b.loss, loss.view(1), ((rel + (S / 1024 + 64) * G.U) * loss + G.TINY).view(1),
                   "loss")


SEQUENCES = {
    "uneven": [0, 1, 64, 64, 130, 131, 400],
    "short, padding behind": [0, 3, 5, 5, 5, 9, 60],
    "one token each": list(range(0, 201)),
    "starts late": [70, 128, 192, 192, 300],
    "none has a token": [5, 5, 5],
}


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("which", list(SEQUENCES))
@pytest.mark.parametrize("T", [60, 400])
def test_balance_sequences(which, T, scoring):
    off = [min(v, T) for v in SEQUENCES[which]]
    l = _logits(T, 72, 110)
    idx = _choose(T, 72, 4, 111)
    # tokens of no sequence may hold anything in their logits
    out = torch.ones(T, dtype=torch.bool)
    out[off[0]:off[-1]] = False
    l[out] = torch.nan
    _balance(l, idx, scoring, off)


def test_balance_no_routes():
    """No tokens, no routes, experts that are masked, a token without a live one."""
    _balance(_logits(0, 8, 112), _choose(0, 8, 2, 1), "softmax")
    _balance(_logits(90, 8, 112), torch.full((90, 2), -1), "softmax", [0, 40, 90])
    l = _logits(100, 16, 113)
    l[torch.rand(l.shape, generator=G.gen(114)) < 0.5] = -torch.inf
    l[7] = -torch.inf
    idx = _choose(100, 16, 2, 115)
    for scoring in ("softmax", "sigmoid"):
        _balance(l, idx, scoring)


def test_balance_flags():
    """Routes outside the experts are skipped, NaN and +inf logits taken as masked."""
    l, idx = _logits(80, 24, 116), _choose(80, 24, 3, 117)
    idx[5, 1], idx[70, 0] = 24, -2
    ref = idx.clone()
    ref[5, 1] = ref[70, 0] = -1
    for i, bits in ((idx, (1,)), (ref, ())):
        _balance(l, i, "softmax", bits=bits)
    l[9, 3], l[66, 4] = torch.nan, torch.inf
    idx[9, 0] = idx[66, 0] = 2
    idx[5, 1] = idx[70, 0] = -1
    _balance(l, idx, "sigmoid", bits=(16,))


@pytest.mark.parametrize("off", [[0, 50, 20, 80], [-5, 40, 80], [0, 40, 1000], [90, 95, 100],
                                 [80, 0]])
def test_balance_bad_offsets(off):
    """Offsets that decrease or leave the batch: flagged, nothing outside the buffers."""
    l, idx = _logits(80, 24, 118), _choose(80, 24, 3, 119)
    S = len(off) - 1
    b = epx().alloc_balance(S + 1, 24, DEV)
    ws = canary(epx().balance_workspace(80, 24, S) + 4096, torch.uint8)
    for t in vars(b).values():
        t.view(torch.uint8).fill_(CANARY)
    part = epx().Balance(b.loss, b.counts[:S], b.probs[:S], b.num_tokens[:S + 1])
    say(f"balance_loss offsets {off}")
    epx().balance_loss(gpu(l), gpu(idx), "softmax",
                       torch.tensor(off, dtype=torch.int32, device=DEV), out=part,
                       workspace=ws[:-4096])
    flags(2)
    assert is_canary(ws[-4096:]) and is_canary(b.counts[S]) and is_canary(b.probs[S])
    assert is_canary(b.num_tokens[S + 1:])


# -------------------------------------------------------------- gradient

def _route_backward(l, idx, scoring, normalize, scale, weights, off=None, bal=True, bits=()):
    T, E = l.shape
    K = idx.shape[1]
    d = torch.randn((T, K), generator=G.gen(120)) if weights else None
    say(f"route_backward T={T} E={E} K={K} {scoring} normalize={normalize} weights={weights} "
        f"balance={bal} sequences={off}")
    b = offd = dloss = None
    if bal:
        offd = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
        b = epx().balance_loss(gpu(l), gpu(idx), scoring, offd)
        epx().get_error()
        dloss = torch.tensor([0.7], device=DEV)
    out = canary((T + 1, E), torch.float32)
    epx().route_backward(gpu(l), gpu(idx), scoring, normalize, scale, gpu(d), b, dloss, offd,
                         out=out[:T])
    flags(*bits)
    assert is_canary(out[T])
    clean = torch.where(l < torch.inf, l, -torch.inf)
    counts = n = None
    if bal:
        _, counts, _, n, _ = G.balance(clean, idx, scoring, off)
    ref, tol = G.route_backward(clean, idx, scoring, normalize, scale, d, counts, n,
                                float(torch.tensor(0.7)), off)
    X.assert_close(out[:T], ref, tol, "dlogits")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("weights,bal", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,E,K", [(1, 2, 1), (5, 8, 2), (67, 65, 6), (30, 160, 32), (130, 256, 8),
                                   (33, 512, 10)])
def test_route_backward(T, E, K, scoring, normalize, weights, bal):
    _route_backward(_logits(T, E, 121), _choose(T, E, K, 122), scoring, normalize, 2.5, weights,
                    bal=bal)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("which", list(SEQUENCES))
def test_route_backward_sequences(which, scoring):
    off = [min(v, 400) for v in SEQUENCES[which]]
    _route_backward(_logits(400, 36, 123), _choose(400, 36, 4, 124), scoring, True, 1.0, True, off)


def test_route_backward_one_weight_is_constant():
    """A normalised weight alone is 1 whatever its logit: no gradient, exactly."""
    l, idx = gpu(_logits(50, 40, 125)), gpu(_choose(50, 40, 1, 126, 0.0))
    d = torch.randn((50, 1), generator=G.gen(127)).to(DEV)
    for scoring in ("softmax", "sigmoid"):
        assert not epx().route_backward(l, idx, scoring, dtopk_weights=d).any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_backward_masked_experts(scoring, normalize):
    """-inf logits get no gradient, chosen or not; an expert named twice gets
    both entries'; bad entries are flagged and skipped."""
    l = _logits(40, 24, 128)
    l[torch.rand(l.shape, generator=G.gen(129)) < 0.4] = -torch.inf
    l[3] = -torch.inf
    l[4] = torch.finfo(torch.float32).min
    idx = _choose(40, 24, 4, 130, 0.0)
    idx[8, 1] = idx[8, 0]
    l[8, idx[8, 0]] = 1.0
    _route_backward(l, idx, scoring, normalize, 1.0, True)
    l[9, 5] = torch.nan
    idx[10, 2] = 24
    _route_backward(l, idx, scoring, normalize, 1.0, True, bits=(1, 16))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_backward_against_differences(scoring):
    """The gradient beside differences of the forward calls themselves."""
    T, E, K = 6, 24, 3
    l = _logits(T, E, 131, 1.0)
    idx = _choose(T, E, K, 132, 0.0)
    d = torch.randn((T, K), generator=G.gen(133))

    def total(l):
        """Weights of a fixed choice (everything else masked) and the loss."""
        only = torch.full_like(l, -torch.inf).scatter(1, idx.clamp(min=0), l.gather(1, idx.clamp(min=0)))
        ci, cw = (t.cpu() for t in epx().route(gpu(only), K, scoring))
        v = 0.0
        for t in range(T):
            for k in range(K):
                if idx[t, k] >= 0:
                    at = (ci[t] == idx[t, k]).nonzero()
                    v += float(d[t, k]) * float(cw[t, int(at)])
        return v + 3.0 * float(epx().balance_loss(gpu(l), gpu(idx), scoring).loss)

    b = epx().balance_loss(gpu(l), gpu(idx), scoring)
    got = epx().route_backward(gpu(l), gpu(idx), scoring, dtopk_weights=gpu(d), balance=b,
                               dloss=torch.full((1,), 3.0, device=DEV)).cpu()
    step = 2.0 ** -5
    # central differences: fp32 values of some 10 are off by 1e-5 or less, over
    # 2^-4, and the third derivative (below 20) times step^2 / 6
    tol = 1e-5 / (2 * step) + 20 * step ** 2 / 6
    for t, e in [(0, int(idx[0, 0])), (0, 1), (2, int(idx[2, 1])), (4, int(idx[4, 2])), (5, 20)]:
        up, dn = l.clone(), l.clone()
        up[t, e] += step
        dn[t, e] -= step
        diff = (total(up) - total(dn)) / float(up[t, e] - dn[t, e])
        assert abs(diff - float(got[t, e])) <= tol, (t, e, diff, float(got[t, e]))


def _far_apart(T, E, top, low, seed):
    """Logits near `low`, of which three a token (experts 0 to 2) are near `top`."""
    l = low + _logits(T, E, seed, 0.5)
    l[:, :3] += top - low
    return l


@pytest.mark.parametrize("top,low", [(-59.0, -95.0), (-30.0, -95.0), (-4.0, -89.0), (-59.0, -130.0),
                                     (-61.0, -95.0), (-75.0, -79.0), (20.0, -95.0)])
@pytest.mark.parametrize("E,K", [(40, 8), (256, 20)])
def test_sigmoids_below_their_underflow(top, low, E, K):
    """Sigmoids that leave fp32's range beside others that do not: normalised weights,
    shares and their gradients are whole, in both directions."""
    l = _far_apart(9, E, top, low, 180)
    l[4] = _logits(1, E, 181)[0]               # an ordinary token beside them
    _route(l, K, "sigmoid")
    idx = G.route(l, K, "sigmoid")[0]
    idx[2] = -1
    _route_backward(l, idx, "sigmoid", True, 2.5, True, bal=False)
    _route_backward(l, idx, "sigmoid", True, 2.5, False)
    _route_backward(l, idx, "sigmoid", True, 2.5, True, [0, 3, 9])
    keep = [t for t in range(9) if t != 4]     # (it would hide the others' mean shares)
    _balance(l[keep], idx[keep], "sigmoid")


def test_router_results_do_not_depend_on_the_wave():
    """A token among others of far smaller scores gives the bytes that it gives alone."""
    E, K = 40, 6
    l = _far_apart(8, E, -59.0, -95.0, 182)
    l[5] = -6.0 + _logits(1, E, 183)[0]
    d = torch.randn((8, K), generator=G.gen(184)).to(DEV)
    say("route, route_backward, balance_loss of one token, alone and among others")
    idx, w = epx().route(gpu(l), K, "sigmoid")
    one = torch.ones(1, device=DEV)
    off = torch.arange(9, dtype=torch.int32, device=DEV)
    b = epx().balance_loss(gpu(l), idx, "sigmoid", off)
    dl = epx().route_backward(gpu(l), idx, "sigmoid", dtopk_weights=d, balance=b, dloss=one * 8,
                              seq_off=off)
    for n in (1, 4):                           # four are a wave of it
        l1, off1 = gpu(l[5:6].repeat(n, 1)), off[:n + 1]
        i1, w1 = epx().route(l1, K, "sigmoid")
        b1 = epx().balance_loss(l1, i1, "sigmoid", off1)
        d1 = epx().route_backward(l1, i1, "sigmoid", dtopk_weights=d[5:6].repeat(n, 1), balance=b1,
                                  dloss=one * n, seq_off=off1)
        flags()
        for a, c, what in ((idx[5:6], i1, "idx"), (w[5:6], w1, "weights"),
                           (b.probs[5:6], b1.probs, "shares"), (dl[5:6], d1, "gradient")):
            for row in c:
                same(a[0], row, what)


# -------------------------------------------------------- combine's gradient

@pytest.mark.parametrize("T,h,K", [(1, 8, 1), (5, 128, 2), (9, 1032, 3), (4, 2056, 9), (6, 4096, 6),
                                   (5, 4104, 1), (7, 7168, 8), (3, 7176, 32), (2, 16392, 2),
                                   (130, 256, 8), (33, 136, 3), (17, 264, 5), (900, 4096, 8)])
def test_combine_backward(T, h, K):
    E = max(K, 8)
    idx = _choose(T, E, K, 140, 0.15 if T > 2 else 0.0)
    lay = epx().get_dispatch_layout(gpu(idx), E, 1)
    w = torch.rand((T, K), generator=G.gen(141))
    d = epx().dispatch(gpu(torch.zeros((T, h), dtype=torch.bfloat16)), gpu(idx), gpu(w), E, 1,
                       layout=lay)
    n = int((idx >= 0).sum())
    pos = d.pos_exp
    dout, y = G.rows((T, h), 142), G.rows((n + 3, h), 143)
    say(f"combine_backward T={T} h={h} K={K} rows={n}")
    dy, dw = canary((n + 3, h), torch.bfloat16), canary((T + 1, K), torch.float32)
    epx().combine_backward(gpu(dout), gpu(y), pos, gpu(w), out=(dy, dw[:T]))
    flags()
    ref, named, rw, tol = G.combine_backward(dout, y, pos.cpu(), w)
    same(dy.cpu()[named], ref[named], "d_expert_out")
    assert is_canary(dy[(~named).to(DEV)]) and is_canary(dw[T])
    X.assert_close(dw[:T], rw, tol, "d_topk_weights")
    assert not dw[:T].cpu()[idx < 0].any()
    # either alone
    a, _ = epx().combine_backward(gpu(dout), None, pos, gpu(w), out=(torch.empty_like(dy), None))
    same(a.cpu()[named], ref[named], "d_expert_out alone")
    _, b = epx().combine_backward(gpu(dout), gpu(y), pos, gpu(w), out=(None, torch.empty_like(dw[:T])))
    same(b, dw[:T], "d_topk_weights alone")


@pytest.mark.parametrize("T,h,K", [((1 << 21) + 5, 8, 2), ((1 << 21) + 3, 264, 1)])
def test_combine_backward_more_tokens_than_a_launch(T, h, K):
    g = torch.Generator(device="cuda").manual_seed(148)
    n = T * K
    pos = torch.randperm(n, generator=g, device=DEV).to(torch.int32).view(T, K)
    w = torch.rand((T, K), generator=g, device=DEV)
    dout = torch.randn((T, h), generator=g, device=DEV).bfloat16()
    y = torch.randn((n, h), generator=g, device=DEV).bfloat16()
    say(f"combine_backward T={T} h={h} K={K}")
    dy, dw = epx().combine_backward(dout, y, pos, w)
    flags()
    for k in range(K):
        for t in torch.arange(T, device=DEV).split(1 << 20):
            r = pos[t, k].long()
            same(dy[r], (w[t, k][:, None] * dout[t].float()).to(torch.bfloat16), "d_expert_out")
            x = dout[t].double() * y[r].double()
            tol = (h / 64 + 14) * G.U * x.abs().sum(1)
            assert bool(((dw[t, k].double() - x.sum(1)).abs() <= tol).all())


@pytest.mark.parametrize("h", [8192, 8200, 12296])
def test_combine_backward_long_rows_in_two_launches(h):
    """Rows of one step and more, whole and in part, sums and scaled rows a launch each."""
    T, K = 600, 6
    dout, y = G.rows((T, h), 204), G.rows((T * K, h), 205)
    w = torch.rand((T, K), generator=G.gen(206))
    pos = torch.randperm(T * K, generator=G.gen(207)).to(torch.int32).view(T, K)
    say(f"combine_backward T={T} h={h} K={K}")
    dy, dw = epx().combine_backward(gpu(dout), gpu(y), gpu(pos), gpu(w))
    flags()
    ref, named, rw, tol = G.combine_backward(dout, y, pos, w)
    assert named.all()
    same(dy.cpu(), ref, "d_expert_out")
    X.assert_close(dw, rw, tol, "d_topk_weights")


def test_combine_backward_bad_handle():
    dout, y, w = gpu(G.rows((3, 64), 144), G.rows((4, 64), 145), torch.rand((3, 2)))
    pos = torch.tensor([[0, 4], [-7, 1], [3, 2]], dtype=torch.int32)
    dy, dw = epx().combine_backward(dout, y, gpu(pos), w)
    flags(4)
    ref, named, rw, tol = G.combine_backward(dout.cpu(), y.cpu(), pos, w.cpu())
    same(dy.cpu()[named], ref[named], "d_expert_out")
    X.assert_close(dw, rw, tol, "d_topk_weights")
    z = epx().combine_backward(dout[:0], y, gpu(pos)[:0], w[:0])
    assert z[1].shape == (0, 2)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    _, dw = epx().combine_backward(dout, y[:0], none, w)
    assert not dw.any()
    flags()


@pytest.mark.parametrize("h", [64, 520])
def test_combine_backward_no_expert_rows(h):
    """No expert rows at all, each gradient alone and both."""
    dout, w = gpu(G.rows((3, h), 186), torch.rand((3, 2)))
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    y = torch.empty((0, h), dtype=torch.bfloat16, device=DEV)
    say(f"combine_backward of no rows h={h}")
    dy, _ = epx().combine_backward(dout, None, none, w, out=(y, None))
    assert dy.shape == (0, h)
    _, dw = epx().combine_backward(dout, y, none, w, out=(None, torch.ones_like(w)))
    assert not dw.any()
    dy, dw = epx().combine_backward(dout, y, none, w)
    assert dy.shape == (0, h) and not dw.any()
    flags()
    epx().combine_backward(dout, None, none + 1, w, out=(y, None))
    flags(4)


# ------------------------------------------------------------ as they are used

def _step(x, r, wn, wr, w13, w2, K, off, dnext, dtop_stream):
    """One training step of a layer: everything this file tests, with dispatch,
    products and combine between, and back to the router's and norm's inputs."""
    m = epx()
    E, f = w13.shape[0], w13.shape[1] // 2
    n = m.rms_norm(x, wn, residual=r)
    # (as sums of products: library products may not replay)
    logits = (n.out.float()[:, None] * wr.float()).sum(2)
    idx, top = m.route(logits, K, "sigmoid", num_groups=4, topk_groups=2, scale=2.0)
    bal = m.balance_loss(logits, idx, "sigmoid", off)
    lay = m.get_dispatch_layout(idx, E, 4)
    d = m.dispatch(n.out, idx, top, E, 4, layout=lay, exact=False)
    act, _ = m.grouped_swiglu(d.recv_x, w13, lay.exp_off)
    y = m.grouped_gemm(act, w2, lay.exp_off)
    out = m.combine(y, d.pos_exp, top)
    dy, dtop = m.combine_backward(dnext, y, d.pos_exp, top)
    dl = m.route_backward(logits, idx, "sigmoid", scale=2.0, dtopk_weights=dtop, balance=bal,
                          dloss=torch.full((1,), 0.1, device=DEV), seq_off=off)
    dn = (dl[:, :, None] * wr.float()).sum(1).to(torch.bfloat16)
    dx, dwn = m.rms_norm_backward(dn, n.residual, wn, dresidual=dtop_stream)
    return dict(n=n, logits=logits, idx=idx, top=top, bal=bal, y=y, out=out, dy=dy, dtop=dtop,
                dl=dl, dn=dn, dx=dx, dwn=dwn, pos=d.pos_exp)


def _step_inputs(T=200, h=256, E=32, f=64):
    x, r, dnext, dstream = (G.rows((T, h), 150 + i) for i in range(4))
    wn = (1 + 0.1 * torch.randn(h, generator=G.gen(155))).to(torch.bfloat16)
    wr = G.rows((E, h), 156, h ** -0.5)
    w13, w2 = G.rows((E, 2 * f, h), 157, h ** -0.5), G.rows((E, h, f), 158, f ** -0.5)
    off = torch.tensor([0, 77, 77, 190], dtype=torch.int32)
    return [t.to(DEV) for t in (x, r, wn, wr, w13, w2)], off.to(DEV), dnext.to(DEV), dstream.to(DEV)


def test_step_against_differentiation():
    """The chain's gradients beside automatic differentiation in 64 bits of the
    same formulas, from the same choice: norm -> router -> weights -> combine,
    and the loss."""
    (x, r, wn, wr, w13, w2), off, dnext, dstream = _step_inputs()
    s = _step(x, r, wn, wr, w13, w2, 4, off, dnext, dstream)
    flags()
    v = s["n"].residual.cpu().double().requires_grad_()
    w = wn.cpu().double().requires_grad_()
    n, _ = G.norm(v, w, 1e-6)
    logits = n @ wr.cpu().double().T
    logits.retain_grad()
    idx = s["idx"].cpu()
    sig = torch.sigmoid(logits)
    top = torch.gather(sig, 1, idx)
    top = 2.0 * top / top.sum(1, keepdim=True)
    y = s["y"].cpu().double()[s["pos"].cpu().long()]
    out = (top[:, :, None] * y).sum(1)
    p = sig / sig.sum(1, keepdim=True)
    _, counts, _, seen, _ = G.balance(logits.detach(), idx, "sigmoid", off.tolist())
    loss, o = 0.0, off.tolist()
    for q in range(3):
        if int(seen[q]):
            loss = loss + (counts[q].double() * p[o[q]:o[q + 1]].mean(0)).sum() * 32 / (4 * int(seen[q])) / int(seen[3])
    ((out * dnext.cpu().double()).sum() + 0.1 * loss + (v * dstream.cpu().double()).sum()).backward()
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    # the router reads bf16 rows: 2^-8 of each channel at most, a random walk
    # over them; the gradients then follow the logits
    loss = float(loss.detach())
    assert abs(float(s["bal"].loss) - loss) <= 2.0 ** -8 * loss
    assert rel(s["top"], top.detach()) < 2.0 ** -8
    assert rel(s["out"], out.detach()) < 2.0 ** -7
    assert rel(s["dl"], logits.grad) < 2.0 ** -6
    # dn is rounded to bf16 once more on its way
    assert rel(s["dx"], v.grad) < 2.0 ** -6
    assert rel(s["dwn"], w.grad) < 2.0 ** -5


def test_norm_fp8_rows_reach_the_products():
    """The normed FP8 rows through an expert that every token visits: what the
    quantised weights make of them, beside 64 bits from the same codes."""
    m = epx()
    T, h, f = 130, 512, 256
    x, r = G.rows((T, h), 195), G.rows((T, h), 196, 3.0)
    wn = (1 + 0.1 * torch.randn(h, generator=G.gen(197))).to(torch.bfloat16)
    w13, w2 = G.rows((1, 2 * f, h), 198, h ** -0.5), G.rows((1, h, f), 199, f ** -0.5)
    say("rms_norm's FP8 rows through grouped_swiglu and grouped_gemm")
    n = m.rms_norm(gpu(x), gpu(wn), residual=gpu(r), fp8=True)
    q13, s13 = m.quantize_weights(gpu(w13))
    q2, s2 = m.quantize_weights(gpu(w2))
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    up = m.grouped_gemm(n.codes, q13, off, n.scales, s13)
    act, act_s = m.grouped_swiglu(n.codes, q13, off, n.scales, s13)
    y = m.grouped_gemm(act, q2, off, act_s, s2)
    flags()
    rows, w64 = X.rows64(n.codes.cpu(), n.scales.cpu()), X.weights64(q13[0].cpu(), s13[0].cpu())
    want, tol = X.product(rows, w64)
    tol = tol + X.cut(n.codes.cpu(), n.scales.cpu(), q13[0].cpu(), s13[0].cpu())
    X.assert_close(up, want, tol + X.BF16 * (want.abs() + tol), "product")
    # through both products, beside the layer from the unrounded normed rows: four
    # roundings to e4m3, 2^-4 each at most, which add in squares
    v = x.double() + r.double()
    v, _ = G.norm(v, wn.double(), 1e-6)
    g, u = (v @ w13[0].double().T).split(f, 1)
    ref = (torch.nn.functional.silu(g) * u) @ w2[0].double().T
    assert float((y.cpu().double() - ref).norm() / ref.norm()) <= 2.0 ** -3


def _flat(s):
    return [t for t in (s["n"].out, s["n"].residual, s["idx"], s["top"], s["bal"].loss,
                        s["bal"].counts, s["bal"].probs, s["bal"].num_tokens, s["out"], s["dy"],
                        s["dtop"], s["dl"], s["dx"], s["dwn"])]


def test_step_is_repeatable_and_replays():
    """The same bytes from the same inputs, on another stream, and from a
    captured graph replayed between other work."""
    args, off, dnext, dstream = _step_inputs()
    run = lambda: _step(*args, 4, off, dnext, dstream)  # noqa: E731
    ref = [t.clone() for t in _flat(run())]
    for a, b in zip(_flat(run()), ref):
        same(a, b, "second run")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _flat(run())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        same(a, b, "another stream")
    say("capture of the step")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _flat(run())
    for replay in range(3):
        for t in held:
            t.view(torch.uint8).fill_(CANARY)
        torch.randn(1 << 20, device=DEV).sum()
        run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        flags()
        for a, b in zip(held, ref):
            same(a, b, f"replay {replay}")


def test_dispatch_gradient_is_a_combine():
    """A token's row goes to each of its entries' rows, so the gradient that comes
    back is their sum: a combine with weights of one."""
    m = epx()
    T, h, E, K = 90, 264, 16, 4
    idx = _choose(T, E, K, 200)
    x, dr = G.rows((T, h), 201), G.rows((int((idx >= 0).sum()), h), 202)
    w = torch.rand((T, K), generator=G.gen(203))
    say("dispatch's gradient")
    d = m.dispatch(gpu(x), gpu(idx), gpu(w), E, 1)
    got = m.combine(gpu(dr), d.pos_exp, torch.ones((T, K), device=DEV))
    flags()
    same(d.recv_x.cpu(), x[d.recv_src.cpu().long()], "recv_x")
    v = x.double().requires_grad_()
    (v[d.recv_src.cpu().long()] * dr.double()).sum().backward()
    # K terms in fp32, then bf16
    mag = torch.zeros((T, h)).double().index_add_(0, d.recv_src.cpu().long(), dr.double().abs())
    tol = K * G.U * mag
    X.assert_close(got, v.grad, tol + G.BF16 * (v.grad.abs() + tol), "dx")


def _repeated(base, T):
    """T rows: those of base again and again."""
    out = torch.empty((T, base.shape[1]), dtype=base.dtype, device=DEV)
    out[:len(base)] = gpu(base)
    done = len(base)
    while done < T:
        n = min(done, T - done)
        out[done:done + n] = out[:n]
        done += n
    return out


def test_router_takes_rows_off_16_bytes():
    """Tensors that start 4 bytes behind a 16-byte boundary give the same bytes."""
    def off(t):
        flat = torch.empty(t.numel() + 4, dtype=t.dtype, device=DEV)
        view = flat[1:1 + t.numel()].view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 16 != 0
        return view

    T, E, K = 70, 64, 6
    l, bias = gpu(_logits(T, E, 176)), gpu(_logits(1, E, 177, 0.1)[0])
    say("router's calls on unaligned tensors")
    idx, w = epx().route(l, K, "sigmoid", bias, 8, 4)
    bal = epx().balance_loss(l, idx, "sigmoid")
    d, one = torch.randn((T, K), generator=G.gen(178)).to(DEV), torch.ones(1, device=DEV)
    dl = epx().route_backward(l, idx, "sigmoid", dtopk_weights=d, balance=bal, dloss=one)
    i2, w2 = epx().route(off(l), K, "sigmoid", off(bias), 8, 4, out=(off(idx), off(w)))
    b2 = epx().balance_loss(off(l), i2, "sigmoid",
                            out=epx().Balance(**{k: off(t) for k, t in vars(bal).items()}))
    dl2 = epx().route_backward(off(l), i2, "sigmoid", dtopk_weights=off(d), balance=b2,
                               dloss=off(one), out=off(dl))
    flags()
    for a, b in zip([idx, w, dl, *vars(bal).values()], [i2, w2, dl2, *vars(b2).values()]):
        same(a, b, "unaligned")


def test_router_beyond_32_bit_offsets():
    """More than 2^31 logits: a token's results do not depend on where it is."""
    T, E, K, B = (1 << 23) + 5, 264, 3, 4096
    base = gpu(_logits(B, E, 170))
    l = _repeated(base, T)
    say(f"route, balance_loss, route_backward T={T} E={E}")
    bi, bw = epx().route(base, K)
    idx, w = epx().route(l, K)
    d = torch.randn((B, K), generator=G.gen(171)).to(DEV)
    dd = _repeated(d, T)
    bl = epx().route_backward(base, bi, dtopk_weights=d)
    dl = epx().route_backward(l, idx, dtopk_weights=dd)
    b = epx().balance_loss(l, idx)
    flags()
    for r in (0, (1 << 31) // E // B * B, T // B * B):
        n = min(B, T - r)
        same(idx[r:r + n], bi[:n], f"topk_idx from {r}")
        same(w[r:r + n], bw[:n], f"topk_w from {r}")
        same(dl[r:r + n], bl[:n], f"dlogits from {r}")
    counts = torch.bincount(bi.flatten(), minlength=E) * (T // B)
    counts += torch.bincount(bi[:T % B].flatten(), minlength=E)
    assert torch.equal(b.counts[0].long(), counts) and b.num_tokens.tolist() == [T, 1]
    del l, idx, w, dl, dd
    torch.cuda.empty_cache()


def test_norm_backward_beyond_32_bit_offsets():
    T, h, B = (1 << 18) + 5, 8200, 512
    base, dbase = G.rows((B, h), 172), G.rows((B, h), 173)
    w = torch.ones(h, device=DEV)
    say(f"rms_norm_backward T={T} h={h}")
    want, _ = epx().rms_norm_backward(gpu(dbase), gpu(base), w)
    x, dout = _repeated(base, T), _repeated(dbase, T)
    dx, dw = epx().rms_norm_backward(dout, x, w)
    flags()
    for r in (0, (1 << 31) // h // B * B, T // B * B):
        n = min(B, T - r)
        same(dx[r:r + n], want[:n], f"dx from {r}")
    v = base.double()
    term = dbase.double() * v * (v.square().mean(1, keepdim=True) + 1e-6) ** -0.5
    times = torch.full((B, 1), T // B).double()
    times[:T % B] += 1
    # a thread adds a row after the other, T / 256 of them or fewer, then come the
    # groups, the blocks and the error of a row's own sum (below 200 in all)
    tol = (T / 256 + 200) * G.U * (times * term.abs()).sum(0)
    X.assert_close(dw, (times * term).sum(0), tol, "dweight")
    del x, dout, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,h,K", [((1 << 16) + 1, 4104, 8), (300001, 7168, 1)])
def test_combine_backward_beyond_32_bit_offsets(T, h, K):
    """More than 2^31 elements of expert rows, in one launch and in two."""
    n = T * K
    g = torch.Generator(device="cuda").manual_seed(174)
    pos = torch.randperm(n, generator=g, device=DEV).to(torch.int32).view(T, K)
    w = torch.rand((T, K), generator=g, device=DEV)
    dout = torch.randn((T, h), generator=g, device=DEV).bfloat16()
    y = _repeated(torch.randn((1024, h), generator=G.gen(175)).bfloat16(), n)
    say(f"combine_backward T={T} h={h} K={K}")
    dy, dw = epx().combine_backward(dout, y, pos, w)
    flags()
    inverse = torch.empty(n, dtype=torch.int64, device=DEV)
    inverse[pos.flatten().long()] = torch.arange(n, device=DEV)
    for r in (0, (1 << 31) // h - 1000, n - 2000):
        tk = inverse[r:r + 2000]
        d = dout[tk // K]
        same(dy[r:r + 2000], (w.flatten()[tk][:, None] * d.float()).to(torch.bfloat16), f"rows from {r}")
        x = d.double() * y[r:r + 2000].double()
        tol = (h / 64 + 14) * G.U * x.abs().sum(1)
        assert bool(((dw.flatten()[tk].double() - x.sum(1)).abs() <= tol).all())
    del dout, y, dy
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    l = [gpu(_logits(3000, 64, 160 + i)) for i in range(2)]
    idx = [gpu(_choose(3000, 64, 6, 162 + i)) for i in range(2)]
    off = gpu(torch.tensor([0, 1000, 2500], dtype=torch.int32))
    x = [gpu(G.rows((3000, 512), 164 + i)) for i in range(2)]
    w = gpu(torch.ones(512))
    want = [(epx().balance_loss(l[i], idx[i], seq_off=off),
             epx().rms_norm_backward(x[i], x[1 - i], w)) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = (epx().balance_loss(l[i], idx[i], seq_off=off),
                          epx().rms_norm_backward(x[i], x[1 - i], w))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(vars(got[i][0]).values(), vars(want[i][0]).values()):
            same(a, b, "balance")
        for a, b in zip(got[i][1], want[i][1]):
            same(a, b, "norm backward")
    flags()


# ---------------------------------------------------------------- refusals

def test_binding_refuses():
    m = epx()
    x, w = gpu(G.rows((4, 256), 170)), torch.ones(256, device=DEV)
    l, idx = gpu(_logits(4, 16, 171)), torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    top, pos = torch.zeros((4, 2), device=DEV), torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    b = m.balance_loss(l, idx)
    one, b16 = torch.ones(1, device=DEV), x.clone()
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    for err, call in [
        (TypeError, lambda: m.rms_norm(x.float(), w)),
        (TypeError, lambda: m.rms_norm(x, w.half())),
        (ValueError, lambda: m.rms_norm(x, w[:128])),
        (ValueError, lambda: m.rms_norm(x.t(), w)),
        (ValueError, lambda: m.rms_norm(x[:, :128], w[:128])),
        (ValueError, lambda: m.rms_norm(x, w, residual=x[:3])),
        (ValueError, lambda: m.rms_norm(x, w, bf16=False)),
        (ValueError, lambda: m.rms_norm(x, w, residual=x, buf=m.Normed(out=x.clone()))),
        (ValueError, lambda: m.rms_norm(x, w, buf=m.Normed(out=x.clone(), residual=x.clone()))),
        (ValueError, lambda: m.rms_norm(x, w, buf=m.Normed(out=x.clone(), scales=w))),
        (m.EpxError, lambda: m.rms_norm(x, w, residual=x, buf=m.Normed(out=b16, residual=b16))),
        (ValueError, lambda: m.rms_norm(x, w.cpu())),
        (ValueError, lambda: m.rms_norm_backward(x[:3], x, w)),
        (ValueError, lambda: m.rms_norm_backward(x, x, w, dresidual=x[:1])),
        (TypeError, lambda: m.rms_norm_backward(x, x, w, out=(x.clone(), w.bfloat16()))),
        (TypeError, lambda: m.route(l.bfloat16(), 2)),
        (ValueError, lambda: m.route(l, 2, "argmax")),
        (ValueError, lambda: m.route(l, 2, bias=w)),
        (TypeError, lambda: m.route(l, 2, mask=one.repeat(4))),
        (ValueError, lambda: m.route(l, 2, out=(idx[:3], top))),
        (ValueError, lambda: m.route(l.t().contiguous().t(), 2)),
        (ValueError, lambda: m.balance_loss(l, idx[:3])),
        (ValueError, lambda: m.balance_loss(l, idx.view(-1))),
        (TypeError, lambda: m.balance_loss(l, idx.int())),
        (TypeError, lambda: m.balance_loss(l, idx, seq_off=off.long())),
        (ValueError, lambda: m.balance_loss(l, idx, seq_off=off[:1])),
        (ValueError, lambda: m.balance_loss(l, idx, seq_off=off, out=m.alloc_balance(2, 16, DEV))),
        (ValueError, lambda: m.route_backward(l, idx)),
        (ValueError, lambda: m.route_backward(l, idx, balance=b)),
        (ValueError, lambda: m.route_backward(l, idx, dtopk_weights=top, dloss=one)),
        (ValueError, lambda: m.route_backward(l, idx, dtopk_weights=top, seq_off=off)),
        (ValueError, lambda: m.route_backward(l, idx, balance=b, dloss=w)),
        (ValueError, lambda: m.route_backward(l, idx, dtopk_weights=top[:, :1])),
        (ValueError, lambda: m.combine_backward(x, x[:, :128].contiguous(), pos, top)),
        (ValueError, lambda: m.combine_backward(x, None, pos, top)),
        (ValueError, lambda: m.combine_backward(x, x, pos, top, out=(None, None))),
        (ValueError, lambda: m.combine_backward(x, None, pos, top, out=(x.clone(), top))),
        (TypeError, lambda: m.combine_backward(x, x, pos.long(), top)),
    ]:
        with pytest.raises(err):
            call()
    for code, call in [
        (-1, lambda: m.rms_norm(x.view(-1)[:12].view(1, 12), w[:12])),
        (-3, lambda: m.scale_stride(264)),
        (-1, lambda: m.rms_norm(x, w, -1.0)),
        (-1, lambda: m.rms_norm(x, w, float("nan"))),
        (-1, lambda: m.rms_norm(torch.zeros((1, 32776), dtype=torch.bfloat16, device=DEV),
                                torch.ones(32776, device=DEV))),
        (-2, lambda: m.rms_norm_backward(x, x, w, workspace=torch.empty(16, dtype=torch.uint8,
                                                                        device=DEV))),
        (-1, lambda: m.route(l, 17)),
        (-1, lambda: m.route(l, 0)),
        (-1, lambda: m.route(l, 2, num_groups=3)),
        (-1, lambda: m.route(l, 2, num_groups=4, topk_groups=5)),
        (-1, lambda: m.route(l, 2, num_groups=4, topk_groups=0)),
        (-1, lambda: m.route(l, 2, scale=float("inf"))),
        (-1, lambda: m.route(torch.zeros((1, 513), device=DEV), 2)),
        (-1, lambda: m.route(torch.zeros((1, 40), device=DEV), 33)),
        (-2, lambda: m.balance_loss(l.repeat(20, 1), idx.repeat(20, 1),
                                    workspace=torch.empty(32, dtype=torch.uint8, device=DEV))),
    ]:
        with pytest.raises(m.EpxError) as e:
            call()
        assert e.value.code == code
    flags()


def test_c_abi_refuses():
    from combine_get_dispatch_counts_amd import _lib, api

    lib, ctx = _lib.load(), api._ctx(DEV)
    t = torch.zeros(4096, device=DEV)
    p = ctypes.c_void_p(t.data_ptr())
    odd = ctypes.c_void_p(t.data_ptr() + 4)
    norm = lambda x=p, r=None, w=p, h=128, ro=None, o=p, c=None, s=None: lib.epx_rms_norm(  # noqa: E731
        ctx, x, r, w, 0, 1, h, 1e-6, ro, o, c, s, None)
    assert norm() == 0
    for bad in (dict(x=None), dict(w=None), dict(o=None), dict(r=p), dict(ro=p), dict(c=p),
                dict(s=p), dict(x=odd), dict(o=odd), dict(w=odd), dict(r=odd, ro=p), dict(h=4)):
        assert norm(**bad) == -1, bad
    assert norm(h=136, c=p, s=p) == -3
    bal = lambda off=None, S=1, ws=p, loss=p, T=0: lib.epx_balance_loss(  # noqa: E731
        ctx, p, p, off, T, 8, 2, S, 0, loss, p, p, p, ws, 16384, None)
    assert bal() == 0 and bal(ws=None) == 0 and bal(ws=None, T=65) == -1 and bal(T=1 << 20) == -2
    assert bal(S=2) == -1 and bal(S=0) == -1 and bal(ws=odd) == -1 and bal(loss=None) == -1
    back = lambda d=p, c=None, n=None, dl=None, off=None, S=1, sc=0: lib.epx_route_backward(  # noqa: E731
        ctx, p, p, 0, 8, 2, sc, 1, 1.0, d, c, n, dl, off, S, p, None)
    assert back() == 0 and back(c=p, n=p, dl=p) == 0
    assert back(d=None) == -1 and back(c=p) == -1 and back(c=p, n=p) == -1
    assert back(c=p, n=p, dl=p, S=2) == -1 and back(n=p) == -1 and back(sc=2) == -1
    comb = lambda y=p, rows=1, dy=p, dw=p, d=p: lib.epx_combine_backward(  # noqa: E731
        ctx, d, y, rows, 8, p, p, 1, 1, dy, dw, None)
    assert comb(y=None) == -1 and comb(dy=None, dw=None) == -1 and comb(d=odd) == -1
    assert comb(rows=-1) == -1 and comb(y=odd) == -1 and comb(dy=odd) == -1
    torch.cuda.synchronize()
    flags()
    assert np.isfinite(t.cpu().numpy()).all()
