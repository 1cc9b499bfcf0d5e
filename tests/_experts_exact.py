"""Operands whose products' sums are exact in fp32 whatever their order, so
that a result over thousands of channels has one right value and a lost, a
repeated or a wrongly scaled step shows.

Values are -1, 0 and 1 (FP8: their codes, with scales 1/2, 1 and 2 per row and
128 channels and per 128 x 128 block of weights). A sum of K <= 65536 such
products is a multiple of 1/4 of at most 4 K = 2^18: 20 bits. The FP8
instruction loses nothing either: the products of eight channels are all 0 or
of the same size. For the gated form everything is 2^-UNIT smaller, which
brings gate and up to a few units; they are exact, and the activation is
g / (1 + exp(-g)) * u up to (8 + |g|) 2^-23 (exp2's argument is rounded, and
exp2, the reciprocal, the sum and two products are within an ulp each).
"""
from __future__ import annotations

import torch

import _experts as X

UNIT = 6


def signs(shape, g):
    return torch.randint(-1, 2, shape, generator=g, dtype=torch.int8)


def powers(shape, g):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g).float())


def operands(fp8, n, L, rows_w, K, seed, unit=0):
    """x, xs, w, ws as the calls take them; 2^-unit is the weights' share."""
    g = torch.Generator().manual_seed(seed)
    x, w = signs((n, K), g).to(torch.bfloat16), signs((L, rows_w, K), g).to(torch.bfloat16)
    if not fp8:
        return x, None, w * 2.0 ** -unit, None
    xs = torch.full((n, X.stride(K)), float("nan"))
    xs[:, :K // 128] = powers((n, K // 128), g)
    ws = powers((L, -(-rows_w // 128), K // 128), g) * 2.0 ** -unit
    code = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    return code(x), xs, code(w), ws


def sums(x, xs, w, ws):
    """One expert's rows times its weights, in 64 bits."""
    return X.rows64(x, xs) @ X.weights64(w, ws).T


def activation(y):
    """The gated activation of sums [m, 2 f] and its bound before rounding."""
    f = y.shape[1] // 2
    g, u = y[:, :f], y[:, f:]
    a = g * torch.sigmoid(g) * u
    return a, (8 + g.abs()) * X.U32 * a.abs()


def assert_sums(got, y, what):
    """bf16 results against exact sums: equal once those are rounded."""
    want = y.float().to(torch.bfloat16)
    bad = got.cpu() != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ"


def assert_activation(got, got_s, y, what):
    a, tol = activation(y)
    if got_s is None:
        X.assert_close(got, a, tol + X.BF16 * (a.abs() + tol), what)
    else:
        X.assert_codes(got, got_s, a, tol, what)


def quantized_rows(x):
    """The dispatch's FP8 rows of fp32 values [n, K]: codes and scales."""
    v = x.view(x.shape[0], -1, 128)
    s = v.abs().amax(-1).clamp_min(1e-4) / 448.0
    q = (v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(x.shape), s


def quantized_weights(w):
    """quantize_weights of fp32 values [E, N, K], N a multiple of 128."""
    E, N, K = w.shape
    b = w.view(E, N // 128, 128, K // 128, 128)
    s = b.abs().amax(dim=(2, 4)).clamp_min(1e-4) / 448.0
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(E, N, K), s


def values(q, s):
    """Codes [n, K] with scales [n, K / 128], in 64 bits."""
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, -1)
