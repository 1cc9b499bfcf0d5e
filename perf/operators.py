"""The experts' arithmetic between dispatch and combine, as calls that can be measured.

Four operators: the block quantiser of expert weights (``quantize``), the grouped
product over expert-major rows or low-latency regions (``gemm``, ``ll_gemm``), the same
product with the gated activation as its epilogue (``swiglu``, ``ll_swiglu``), and the
whole layer for a few tokens (``decode``). ``run`` computes each in plain torch operations
in 32 bits, or, with ``own`` set, through this repository's package.

Formats are the dispatch's: FP8 rows are e4m3 codes with fp32 scales per 128 channels in
rows of whole 128-byte lines; FP8 weights have one fp32 scale per 128 x 128 block.
"""
import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0
AMAX_FLOOR = 1e-4


# ----------------------------------------------------------------- cases

def listed():
    return [
        # A small bank of weights quantised at load: launch latency.
        dict(name="quantize small", op="quantize", experts=4, n=264, k=1024),
        # A rank's share of a large bank, as after a weight update: the memory's rate.
        dict(name="quantize bank", op="quantize", experts=32, n=4096, k=7168),
        # The tiny workload's down product: 64 tokens, top-2 of 8 experts. Latency.
        dict(name="gemm tiny bf16", op="gemm", dtype="bf16", tokens=64, topk=2, experts=8, n=128,
             k=128, zipf=False),
        # The skewed workload's down product, a few experts with most rows.
        dict(name="gemm skew fp8", op="gemm", dtype="fp8", tokens=8192, topk=6, experts=64, n=4096,
             k=2048, zipf=True),
        # A receiver's eight experts after its permute, bf16 rows, an odd number of them.
        dict(name="gemm receive bf16", op="gemm", dtype="bf16", tokens=29811, topk=1, experts=8,
             n=7168, k=2048, zipf=False),
        # A receiver's low-latency regions: eight experts, 32 sources of a few rows each.
        dict(name="ll gemm receive fp8", op="ll_gemm", dtype="fp8", tokens=1024, topk=1, experts=8,
             ranks=32, cap=128, n=7168, k=2048, zipf=False),
        # The prefill workload's first product with its activation, all 256 experts.
        dict(name="swiglu prefill fp8", op="swiglu", dtype="fp8", tokens=4096, topk=8, experts=256,
             f=2048, k=7168, zipf=False),
        # A medium ragged batch in bf16 with sizes that end inside tiles.
        dict(name="swiglu ragged bf16", op="swiglu", dtype="bf16", tokens=1003, topk=6, experts=64,
             f=1416, k=4096, zipf=True),
        # The decode workload's regions: 128 tokens over 256 experts, about four rows each.
        dict(name="ll swiglu decode fp8", op="ll_swiglu", dtype="fp8", tokens=128, topk=8,
             experts=256, ranks=1, cap=128, f=2048, k=7168, zipf=False),
        # One token through the whole layer: eight experts' weights.
        dict(name="decode 1 token fp8", op="decode", dtype="fp8", tokens=1, topk=8, experts=256,
             f=2048, h=7168),
        # A small serving batch in bf16 weights.
        dict(name="decode 8 tokens bf16", op="decode", dtype="bf16", tokens=8, topk=6, experts=64,
             f=1536, h=4096),
        # A larger serving batch: most experts are met, by a few tokens each.
        dict(name="decode 48 tokens fp8", op="decode", dtype="fp8", tokens=48, topk=8, experts=128,
             f=2048, h=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """One more case: any operator, sizes over their whole range. Drawn again while it costs
    more than the largest listed one or its weights take more than 8 GB."""
    top = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["quantize", "gemm", "gemm", "swiglu", "swiglu", "ll_gemm", "ll_swiglu",
                         "decode", "decode"])
        if op == "quantize":
            c = dict(op=op, experts=_log(rng, 1, 64), n=8 * _log(rng, 1, 1024),
                     k=128 * _log(rng, 1, 64))
            weights = c["experts"] * c["n"] * c["k"] * 2
        else:
            dtype = rng.choice(["fp8", "fp8", "bf16"])
            unit = 128 if dtype == "fp8" else 8
            experts = _log(rng, 1, 256)
            topk = rng.randint(1, min(8, experts))
            h = unit * _log(rng, 1, 8192 // unit)
            f = unit * _log(rng, 1, 4096 // unit)
            c = dict(op=op, dtype=dtype, topk=topk, experts=experts)
            if op == "decode":
                c.update(tokens=_log(rng, 1, 64), f=f, h=h)
            else:
                c.update(tokens=_log(rng, 1, 16384), zipf=rng.random() < 0.3)
                c.update(dict(f=f, k=h) if op.endswith("swiglu") else
                         dict(n=8 * _log(rng, 1, 1024), k=f))
                if op.startswith("ll_"):
                    c["ranks"] = rng.choice([1, 4, 8, 32])
                    c["topk"] = topk if c["ranks"] == 1 else 1
                    c["tokens"] = min(c["tokens"], 16 * experts * c["ranks"], 4096)
                    c["cap"] = rng.choice([64, 100, 128]) if c["ranks"] > 1 else c["tokens"]
                    if experts * c["ranks"] * c["cap"] > 65536:
                        continue
            wide = 3 * f * h if op == "decode" else c.get("n", 2 * f) * c["k"]
            weights = experts * wide * (1 if dtype == "fp8" else 2)
        if weights <= 8e9 and _cost(c) <= top:
            return c


def _expected_active(case):
    """How many experts the rows are expected to meet (the routing is drawn with the inputs)."""
    E, n = case["experts"], case["tokens"]
    return E * (1.0 - (1.0 - case["topk"] / E) ** n)


def work(case):
    op = case["op"]
    if op == "quantize":
        E, N, K = case["experts"], case["n"], case["k"]
        return dict(bytes=3.0 * E * N * K + 4.0 * E * -(-N // 128) * (K // 128), flops=3.0 * E * N * K)
    fp8 = case["dtype"] == "fp8"
    size = 1 if fp8 else 2
    if op == "decode":
        T, f, h = case["tokens"], case["f"], case["h"]
        scales = 3 * (f // 128) * (h // 128) * 4 if fp8 else 0
        return dict(bytes=_expected_active(case) * (3.0 * f * h * size + scales) + 4.0 * T * h
                    + 12.0 * T * case["topk"], flops=6.0 * T * case["topk"] * f * h)
    rows, K = case["tokens"] * case["topk"], case["k"]
    gated = op.endswith("swiglu")
    N = 2 * case["f"] if gated else case["n"]
    scales = lambda n, m: 4.0 * n * m / 128 if fp8 else 0.0  # noqa: E731
    b = rows * K * size + scales(rows, K)
    b += _expected_active(case) * (N * K * size + (scales(-(-N // 128), K) if fp8 else 0.0))
    if gated:
        b += rows * case["f"] * size + scales(rows, case["f"])
    else:
        b += rows * N * 2
    return dict(bytes=float(b), flops=2.0 * rows * N * K)


# ---------------------------------------------------------------- inputs

def _stride(k):
    return (k // 128 + 31) // 32 * 32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(g, shape):
    """e4m3 codes (uint8) of normal values whose group maximum sits near 448, as quantised
    normal data has it; made slice by slice."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for part in out.view(-1).split(1 << 28):
        v = torch.randn(part.shape, generator=g, device="cuda").mul_(110.0).clamp_(-448.0, 448.0)
        part.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _bf16(g, shape, scale):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(scale))
    return out


def _scales(g, shape, level):
    """fp32 scales spread over a factor of about three around ``level`` / 110."""
    return torch.empty(shape, device="cuda").uniform_(0.5, 1.5, generator=g).mul_(level / 110.0)


def _weights(g, E, N, K, fp8):
    """Weights whose products with unit rows are near one: (w, scales or None)."""
    if not fp8:
        return _bf16(g, (E, N, K), K ** -0.5), None
    return _codes(g, (E, N, K)), _scales(g, (E, -(-N // 128), K // 128), K ** -0.5)


def _routing(case, seed):
    """Distinct experts per token by the largest of noisy logits (skewed with ``zipf``)."""
    rng = np.random.default_rng(seed)
    T, E, k = case["tokens"], case["experts"], case["topk"]
    logits = rng.gumbel(size=(T, E)).astype(np.float32)
    if case.get("zipf"):
        logits += (-1.2 * np.log(rng.permutation(E) + 1.0)).astype(np.float32)
    return np.argsort(-logits, axis=1, kind="stable")[:, :k]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        w = _bf16(g, (case["experts"], case["n"], case["k"]), case["k"] ** -0.5)
        return dict(op=op, w=w)
    fp8 = case["dtype"] == "fp8"
    E = case["experts"]
    if op == "decode":
        T, f, h, k = case["tokens"], case["f"], case["h"], case["topk"]
        w13, s13 = _weights(g, E, 2 * f, h, fp8)
        w2, s2 = _weights(g, E, h, f, fp8)
        top = torch.rand((T, k), generator=g, device="cuda").add_(0.1)
        return dict(op=op, x=_bf16(g, (T, h), 1.0), w13=w13, s13=s13, w2=w2, s2=s2,
                    topk_idx=torch.from_numpy(_routing(case, seed)).cuda(),
                    topk_w=top / top.sum(1, keepdim=True))
    K = case["k"]
    gated = op.endswith("swiglu")
    N = 2 * case["f"] if gated else case["n"]
    counts = np.bincount(_routing(case, seed).ravel(), minlength=E)
    state = dict(op=op, cap=0)
    if op.startswith("ll_"):
        # region e * ranks + s holds the rows source s sent to expert e, in its first places
        R, cap = case["ranks"], case["cap"]
        rng = np.random.default_rng(seed + 1)
        per = np.stack([rng.multinomial(c, np.full(R, 1.0 / R)) for c in counts]).reshape(-1)
        per = np.minimum(per, cap)
        state.update(cap=cap, counts=torch.from_numpy(per.astype(np.int32)).cuda(),
                     segments=[[(r * cap, r * cap + int(per[r]))
                                for r in range(e * R, (e + 1) * R) if per[r]] for e in range(E)])
        rows = E * R * cap
    else:
        off = np.concatenate([[0], np.cumsum(counts)])
        rows = int(off[-1])
        state.update(exp_off=torch.from_numpy(off.astype(np.int32)).cuda(),
                     segments=[[(int(a), int(b))] if b > a else []
                               for a, b in zip(off[:-1], off[1:])])
    w, ws = _weights(g, E, N, K, fp8)
    state.update(w=w, ws=ws)
    if fp8:
        state["x"] = _codes(g, (rows, K))
        state["xs"] = torch.zeros((rows, _stride(K)), device="cuda")
        state["xs"][:, :K // 128] = _scales(g, (rows, K // 128), 1.0)
    else:
        state["x"], state["xs"] = _bf16(g, (rows, K), 1.0), None
    if gated and fp8:
        state["out"] = torch.zeros((rows, case["f"]), dtype=torch.uint8, device="cuda")
        state["out_scales"] = torch.zeros((rows, _stride(case["f"])), device="cuda")
    else:
        state["out"] = torch.zeros((rows, case["f"] if gated else N), dtype=torch.bfloat16,
                                   device="cuda")
        state["out_scales"] = None
    return state


# ------------------------------------------------------------ plain form

def _wide(s, n):
    """Group scales repeated over their 128 channels (or rows), cut to n."""
    return s.repeat_interleave(128, dim=-1)[..., :n]


def _rows32(x, xs):
    if xs is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _wide(xs, x.shape[-1])


def _weights32(w, ws):
    if ws is None:
        return w.float()
    s = _wide(_wide(ws, w.shape[-1]).transpose(-1, -2), w.shape[-2]).transpose(-1, -2)
    return w.view(torch.float8_e4m3fn).float() * s


def _silu_mul(y):
    g, u = y.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _quantized(v):
    """Groups of the last axis: fp32 scales max(amax, 1e-4) / 448 and e4m3 of the quotients."""
    s = v.abs().amax(-1).clamp_min(AMAX_FLOOR) / FP8_MAX
    return (v / s[..., None]).to(torch.float8_e4m3fn), s


def _plain_quantize(w):
    E, N, K = w.shape
    up = -(-N // 128) * 128
    v = torch.nn.functional.pad(w.float(), (0, 0, 0, up - N))
    v = v.view(E, up // 128, 128, K // 128, 128).permute(0, 1, 3, 2, 4).reshape(E, up // 128, K // 128, -1)
    q, s = _quantized(v)
    q = q.view(torch.uint8).view(E, up // 128, K // 128, 128, 128).permute(0, 1, 3, 2, 4)
    return q.reshape(E, up, K)[:, :N].contiguous().view(torch.float8_e4m3fn), s


def _plain_grouped(st):
    gated = st["op"].endswith("swiglu")
    for e, segments in enumerate(st["segments"]):
        if not segments:
            continue
        x = torch.cat([st["x"][a:b] for a, b in segments])
        xs = None if st["xs"] is None else torch.cat([st["xs"][a:b] for a, b in segments])
        y = _rows32(x, xs) @ _weights32(st["w"][e], None if st["ws"] is None else st["ws"][e]).T
        if gated:
            y = _silu_mul(y)
        s = None
        if st["out_scales"] is not None:
            q, s = _quantized(y.view(y.shape[0], -1, 128))
            y = q.view(torch.uint8).view(y.shape)
        at = 0
        for a, b in segments:
            st["out"][a:b] = y[at:at + b - a]
            if s is not None:
                st["out_scales"][a:b, :s.shape[1]] = s[at:at + b - a]
            at += b - a
    return _grouped_outputs(st)


def _plain_decode(st):
    T = st["x"].shape[0]
    out = []
    for t in range(T):
        e = st["topk_idx"][t]
        w13 = _weights32(st["w13"][e], None if st["s13"] is None else st["s13"][e])
        a = _silu_mul(w13 @ st["x"][t].float())
        w2 = _weights32(st["w2"][e], None if st["s2"] is None else st["s2"][e])
        y = torch.matmul(w2, a[:, :, None])[:, :, 0]
        out.append((st["topk_w"][t][:, None] * y).sum(0))
    return torch.stack(out).to(torch.bfloat16)


def _grouped_outputs(st):
    if st["out_scales"] is None:
        return st["out"]
    return st["out"].view(torch.float8_e4m3fn), st["out_scales"]


# ------------------------------------------------------------------- run

def run(state):
    st, op = state, state["op"]
    if own:
        import combine_get_dispatch_counts_amd as epx

        if op == "quantize":
            q, s = epx.quantize_weights(st["w"])
            return q.view(torch.float8_e4m3fn), s
        if op == "decode":
            return epx.moe_decode(st["x"], st["topk_idx"], st["topk_w"], st["w13"], st["w2"],
                                  w13_scales=st["s13"], w2_scales=st["s2"])
        more = dict(x_scales=st["xs"], w_scales=st["ws"], out=st["out"])
        if op.endswith("swiglu"):
            more["out_scales"] = st["out_scales"]
        if op.startswith("ll_"):
            call = epx.ll_grouped_swiglu if op == "ll_swiglu" else epx.ll_grouped_gemm
            call(st["x"], st["w"], st["counts"], st["cap"], **more)
        else:
            call = epx.grouped_swiglu if op == "swiglu" else epx.grouped_gemm
            call(st["x"], st["w"], st["exp_off"], **more)
        return _grouped_outputs(st)
    if op == "quantize":
        return _plain_quantize(st["w"])
    if op == "decode":
        return _plain_decode(st)
    return _plain_grouped(st)


# ----------------------------------------------------------------- exact

def _e4m3_64(v):
    """v rounded to the nearest e4m3 value, ties to even, saturating, in 64 bits: three
    mantissa bits from 2^-6 up, steps of 2^-9 below."""
    m, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _value64(w, s, dims):
    """The 64-bit values of a code tensor with scales over 128-long groups of ``dims``."""
    if s is None:
        return w.double()
    s = s.double()
    for d in dims:
        at = torch.arange(w.shape[d], device=w.device) // 128
        s = s.index_select(d, at)
    return w.view(torch.float8_e4m3fn).double() * s


def _quantize64(w):
    codes, scales = torch.empty(w.shape, dtype=torch.float64, device=w.device), []
    E, N, K = w.shape
    for n in range(0, N, 128):
        b = w[:, n:n + 128].double().reshape(E, -1, K // 128, 128)
        s = b.abs().amax(dim=(1, 3)).clamp(min=AMAX_FLOOR) / FP8_MAX
        codes[:, n:n + 128] = _e4m3_64(b / s[:, None, :, None]).reshape(E, -1, K)
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _swiglu64(y):
    f = y.shape[-1] // 2
    return y[..., :f] * torch.sigmoid(y[..., :f]) * y[..., f:]


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        return _quantize64(st["w"])
    if op == "decode":
        x, idx, top = st["x"].double(), st["topk_idx"], st["topk_w"].double()
        out = torch.zeros_like(x)
        for e in torch.unique(idx).tolist():
            t, k = torch.nonzero(idx == e, as_tuple=True)
            w13 = _value64(st["w13"][e], None if st["s13"] is None else st["s13"][e], (0, 1))
            w2 = _value64(st["w2"][e], None if st["s2"] is None else st["s2"][e], (0, 1))
            out.index_add_(0, t, top[t, k][:, None] * (_swiglu64(x[t] @ w13.T) @ w2.T))
        return out
    gated = op.endswith("swiglu")
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    scales = None if st["out_scales"] is None else torch.zeros(st["out_scales"].shape,
                                                               dtype=torch.float64, device="cuda")
    for e, segments in enumerate(st["segments"]):
        w = _value64(st["w"][e], None if st["ws"] is None else st["ws"][e], (0, 1))
        rows = [torch.arange(a, b, device="cuda") for a, b in segments]
        if not rows:
            continue
        r = torch.cat(rows)
        y = _value64(st["x"][r], None if st["xs"] is None else st["xs"][r], (1,)) @ w.T
        if gated:
            y = _swiglu64(y)
        if scales is not None:
            v = y.view(y.shape[0], -1, 128)
            s = v.abs().amax(-1).clamp(min=AMAX_FLOOR) / FP8_MAX
            scales[r, :s.shape[1]] = s
            y = _e4m3_64(v / s[..., None]).view(y.shape)
        out[r] = y
    return out if scales is None else (out, scales)
