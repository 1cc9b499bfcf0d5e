"""The experts' arithmetic in 64 bits on the CPU, with the error each result
may have, for the GPU tests. Every bound is derived, none is fitted:

 * rounding to a type is off by at most half a step: bf16 2^-8, e4m3 2^-4 of
   the value (2^-10 of the scale in its subnormal range);
 * a sum of K exact products in fp32, in any order and with truncating adds,
   is off by at most K 2^-23 times the sum of the products' magnitudes; the
   FP8 form multiplies by two scales and adds again, covered by K + 8;
 * the plain FP8 product's instruction cuts each product towards zero to a
   multiple of 2^(m - 13), m the largest exponent sum of the eight products
   of channels 8 i .. 8 i + 7 (subnormal codes have exponent -6): the largest
   is kept whole (its last bit is 2^(m - 6)), each of the seven others loses
   less than 2^(m - 13) (cut below; cut_product is the cut sum itself);
 * exp2 and the reciprocal are within an ulp, the argument of exp2 is rounded
   once: (8 + |g|) 2^-23 of silu(g) u.
"""
from __future__ import annotations

import numpy as np
import torch

U32, BF16, E4M3 = 2.0 ** -23, 2.0 ** -8, 2.0 ** -4


def stride(k: int) -> int:
    return (k // 128 + 31) // 32 * 32


def randn(shape, seed, scale=1.0) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def fp8_rows(shape, seed):
    """Random codes (no NaN) with scales: (codes, padded scales [rows, stride])."""
    n, k = shape
    g = torch.Generator().manual_seed(seed)
    c = (torch.randn(shape, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.full((n, stride(k)), float("nan"))
    s[:, :k // 128] = (torch.rand((n, k // 128), generator=g) + 0.5) / 110
    return c.view(torch.uint8), s


def fp8_weights(shape, seed):
    E, n, k = shape
    g = torch.Generator().manual_seed(seed)
    c = (torch.randn(shape, generator=g) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand((E, -(-n // 128), k // 128), generator=g) + 0.5) / 110 * k ** -0.5
    return c.view(torch.uint8), s


def rows64(x, xs=None):
    if xs is None:
        return x.double()
    k = x.shape[1]
    return x.view(torch.float8_e4m3fn).double() * xs[:, :k // 128].double().repeat_interleave(128, 1)


def weights64(w, ws=None):
    """One expert's matrix [n, k]."""
    if ws is None:
        return w.double()
    s = ws.double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:w.shape[0]]
    return w.view(torch.float8_e4m3fn).double() * s


def product(x, w):
    """x [m, k] @ w [n, k].T in 64 bits and the fp32 sum's bound."""
    return x @ w.T, (x.shape[1] + 8) * U32 * (x.abs() @ w.abs().T)


def cut(x, xs, w, ws):
    """What cutting can take from the sums of x's rows [m, k] with one expert's
    rows w [n, k] (codes and scales): 7 times 2^-13 of each eight's largest."""
    big = lambda v: v.abs().clamp(min=2.0 ** -6).view(v.shape[0], -1, 8).amax(-1)  # noqa: E731
    k = x.shape[1]
    gx = big(x.view(torch.float8_e4m3fn).double()) * xs[:, :k // 128].double().repeat_interleave(16, 1)
    one = torch.full_like(w, 0x38)                                 # codes of 1: the scales
    gw = big(w.view(torch.float8_e4m3fn).double()) * weights64(one, ws)[:, ::8]
    return 7 * 2.0 ** -13 * (gx @ gw.T)


def cut_product(x, w):
    """Row i of x times row i of w, codes [n, 128], each product cut."""
    x, w = (c.view(torch.float8_e4m3fn).double() for c in (x, w))
    p = (x * w).view(-1, 16, 8)
    m = sum(torch.floor(torch.log2(c.abs().clamp(min=2.0 ** -6))) for c in (x, w)).view(-1, 16, 8)
    m = torch.where(p == 0, torch.full_like(m, -99.0), m).amax(-1, keepdim=True)
    step = 2.0 ** (m - 13)
    return (torch.trunc(p / step) * step).sum((1, 2)), p.abs().sum((1, 2))


def gated(x, w):
    """silu(gate) * up of one expert, and its bound before any rounding to a
    narrower type."""
    f = w.shape[0] // 2
    g, dg = product(x, w[:f])
    u, du = product(x, w[f:])
    a = g * torch.sigmoid(g) * u
    return a, 1.1 * dg * (u.abs() + du) + g.abs() * du + (8 + g.abs()) * U32 * a.abs()


def assert_close(got, ref, tol, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {ref[bad][0]} "
                           f"(allowed {tol[bad][0]})")


def assert_codes(q, s, ref, tol, what):
    """e4m3 codes [m, f] (uint8) and scales [m, stride] against values with a
    bound: the scales, the padding's zeros, and every dequantised value."""
    m, f = q.shape
    q, s = q.cpu(), s.cpu()
    groups, gt = ref.view(m, -1, 128).abs().amax(-1), tol.view(m, -1, 128).amax(-1)
    s64 = groups.clamp(min=1e-4) / 448
    assert_close(s[:, :f // 128], s64, gt / 448 + 2 * U32 * s64, what + " scales")
    assert (s[:, f // 128:] == 0).all() and not torch.signbit(s[:, f // 128:]).any(), \
        what + " padding"
    wide = s[:, :f // 128].double().repeat_interleave(128, 1)
    got = q.view(torch.float8_e4m3fn).double() * wide
    # half a step around the unrounded value, whose quotient is rounded once to fp32
    near = ref.abs() + tol
    assert_close(got, ref, tol + E4M3 * near + 2.0 ** -10 * wide + U32 * near, what + " values")


def offsets(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)
