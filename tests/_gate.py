"""The norm, the router's choice, the balance loss and the gradients in 64 bits
on the CPU, with the error that each result may have, for the GPU tests. Every
bound is derived, none is fitted; U = 2^-24 is half a step of fp32.

 * a row's sum over its channels: a thread adds at most 32 terms, a wave six
   more times and a block at most 16: 56 roundings beside the terms' own;
 * 1 / sqrt(mean + eps) halves the mean's error and adds a rounding for the
   division by h, the eps, the root and the reciprocal: INV = 34 in all;
 * exp is within two units of the last place (4 U) of its argument's, which is a
   rounded difference of logits: (4 + |x|) U;
 * rounding to bf16 is off by at most 2^-8 of the value.
"""
from __future__ import annotations

import torch

U, BF16 = 2.0 ** -24, 2.0 ** -8
INV = 34
TINY = 2.0 ** -125      # what falls below fp32's normal range may be lost


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(torch.bfloat16)


# ------------------------------------------------------------------ norm

def norm(v, w, eps):
    """v [T, h] and w [h] in 64 bits -> (y, inv)."""
    inv = (v.square().mean(1, keepdim=True) + eps) ** -0.5
    return v * inv * w, inv


def norm_tol(y, v, inv, w):
    """Before any rounding to a narrower type: v's own rounding (of a sum of two
    bf16 values), inv's error, two products."""
    return (INV + 3) * U * y.abs() + U * (v.abs() * inv * w.abs())


def norm_backward(dout, v, w, eps, dres=None):
    """(dx, its bound before rounding, dweight, its bound) of 64-bit inputs."""
    T, h = v.shape
    inv = (v.square().mean(1, keepdim=True) + eps) ** -0.5
    n, g = v * inv, dout * w
    dx = inv * (g - n * (g * n).mean(1, keepdim=True))
    # the mean's terms: 57 roundings and inv twice; then products and additions
    mag = inv * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    tol = (57 + 3 * INV + 8) * U * mag
    if dres is not None:
        dx = dx + dres
        tol = tol + U * (mag + dres.abs())
    # rows in turn (at least 256 blocks share them), then as many blocks
    adds = -(-T // 256) + 1024 / 16 + 16
    dw = (dout * n).sum(0)
    return dx, tol, dw, (adds + INV + 3) * U * (dout * n).abs().sum(0) + TINY


# ---------------------------------------------------------------- router

def scores(l, scoring):
    """Scores [T, E] of 64-bit logits; experts at -inf get 0."""
    if scoring == "sigmoid":
        return torch.sigmoid(l)
    m = l.amax(1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    e = torch.exp(l - m)
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def shares(l, scoring):
    if scoring == "softmax":
        return scores(l, scoring)
    # relative to the largest, so that no sum of tiny scores vanishes
    ls = torch.nn.functional.logsigmoid(l)
    return scores(ls, "softmax")


def spread(l):
    """Largest distance of a live logit from its row's largest (or from 0)."""
    live = torch.where(l.isinf(), torch.zeros_like(l), l)
    return 2.0 * live.abs().amax(1, keepdim=True).clamp(max=110.0)


def route(l, K, scoring, bias=None, G=1, top=1, normalize=True, scale=1.0, mask=None):
    """(topk_idx, topk_w, bound of topk_w), expert by expert in plain Python."""
    l = l.double()
    T, E = l.shape
    s = scores(l, scoring)
    key = s if bias is None else s + bias.double()
    live = ~l.isinf() if bias is None else ~l.isinf() & ~bias.isinf()
    idx = torch.full((T, K), -1, dtype=torch.int64)
    w = torch.zeros((T, K), dtype=torch.float64)
    tol = torch.zeros_like(w)
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        can = [e for e in range(E) if live[t, e]]
        k = key[t].tolist()
        if G > 1:
            per, best = E // G, []
            for g in range(G):
                two = sorted((k[e] for e in can if e // per == g), reverse=True)[:2]
                if two:
                    best.append((-sum(two), g))
            kept = {g for _, g in sorted(best)[:top]}
            can = [e for e in can if e // per in kept]
        order = l[t].tolist() if bias is None else k
        can = sorted(can, key=lambda e: (-order[e], e))[:K]
        n = len(can)
        if n == 0:
            continue
        at = torch.tensor(can)
        idx[t, :n] = at
        if normalize:
            v = shares(l[t:t + 1, at], scoring)[0]
        else:
            v = s[t, at]
        w[t, :n] = scale * v
        # the exponents', sums over 512 experts or K entries (14 roundings), the
        # quotients and the scale
        tol[t, :n] = (2 * (4 + float(spread(l[t:t + 1]))) + 14 + 6) * U * w[t, :n].abs() \
            + abs(scale) * TINY
    return idx, w, tol


def balance(l, idx, scoring, off=None):
    """(loss, counts, probs, num_tokens) and the relative bound of the shares."""
    l = l.double()
    T, E = l.shape
    K = idx.shape[1]
    off = [0, T] if off is None else [int(v) for v in off]
    S = len(off) - 1
    p = shares(l, scoring)
    counts = torch.zeros((S, E), dtype=torch.int32)
    probs = torch.zeros((S, E), dtype=torch.float64)
    seen, losses = [], []
    for s in range(S):
        n = 0
        for t in range(off[s], off[s + 1]):
            named = [int(e) for e in idx[t] if 0 <= e < E]
            for e in named:
                counts[s, e] += 1
            if named:
                n += 1
                probs[s] += p[t]
        if n:
            probs[s] /= n
            losses.append(float((counts[s].double() * probs[s]).sum()) * E / (K * n))
        seen.append(n)
    loss = sum(losses) / len(losses) if losses else 0.0
    # a block adds a run's tokens (64 at most), the last launch the runs (of 32
    # tokens at least), in any order
    adds = 64 + -(-T // 32)
    rel = (adds + 2 * (4 + float(spread(l).max() if T else 0.0)) + 14 + 6) * U
    return loss, counts, probs, torch.tensor(seen + [len(losses)], dtype=torch.int32), rel


def route_backward(l, idx, scoring, normalize, scale, d=None, counts=None, num_tokens=None,
                   dloss=0.0, off=None):
    """(dlogits, bound) by the formulas."""
    l = l.double()
    T, E = l.shape
    K = idx.shape[1]
    s, p = scores(l, scoring), shares(l, scoring)
    slope = 1.0 - s if scoring == "sigmoid" else torch.ones_like(s)
    if scoring == "sigmoid":
        slope = torch.sigmoid(-l)
    out, mag = torch.zeros_like(l), torch.zeros_like(l)
    off = [0, T] if off is None else [int(v) for v in off]
    for t in range(T):
        ks = [k for k in range(K) if 0 <= idx[t, k] < E]
        if not ks:
            continue
        es = idx[t, ks]
        if d is not None:
            dk = d[t, ks].double() * scale
            if normalize:
                q = shares(l[t:t + 1, es], scoring)[0]
                g = q * slope[t, es] * (dk - (q * dk).sum())
                m = q * slope[t, es] * (dk.abs() + (q * dk.abs()).sum())
                out[t].index_add_(0, es, g)
                mag[t].index_add_(0, es, m)
            elif scoring == "sigmoid":
                g = dk * s[t, es] * slope[t, es]
                out[t].index_add_(0, es, g)
                mag[t].index_add_(0, es, g.abs())
            else:
                D = torch.zeros(E, dtype=torch.float64).index_add_(0, es, dk)
                A = torch.zeros(E, dtype=torch.float64).index_add_(0, es, dk.abs())
                out[t] += s[t] * (D - (s[t] * D).sum())
                mag[t] += s[t] * (A + (s[t] * A).sum())
        if counts is not None:
            for q in range(len(off) - 1):
                if off[q] <= t < off[q + 1]:
                    n = int(num_tokens[q])
                    a = counts[q].double() * (dloss * E / (K * n * n * int(num_tokens[-1])))
                    out[t] += p[t] * slope[t] * (a - (a * p[t]).sum())
                    mag[t] += p[t] * slope[t] * (a + (a * p[t]).sum())
    # exponents of scores, sums over the experts, slope, quotients, products
    return out, (3 * (4 + spread(l)) + 2 * 14 + K + 12) * U * mag + TINY


def combine_backward(dout, y, pos, w):
    """(dy for the named rows and the mask of those, bit for bit; dw and its bound)."""
    T, K = pos.shape
    dy = torch.zeros_like(y)
    named = torch.zeros(y.shape[0], dtype=torch.bool)
    dw, mag = torch.zeros((T, K), dtype=torch.float64), torch.zeros((T, K), dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(pos[t, k])
            if 0 <= r < y.shape[0]:
                dy[r] = (w[t, k] * dout[t].float()).to(torch.bfloat16)
                named[r] = True
                x = dout[t].double() * y[r].double()
                dw[t, k], mag[t, k] = x.sum(), x.abs().sum()
    # products of bf16 are exact; a lane adds a 64th of the channels, in whole
    # vectors of 8, a wave six times more
    return dy, named, dw, (dout.shape[1] / 64 + 8 + 6) * U * mag
