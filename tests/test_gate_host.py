"""What the norm's, the router's and the gradients' calls refuse before any GPU
work, and the 64-bit forms that the GPU tests compare with, checked against
hand-worked values and, for gradients, against differences (CPU)."""
import ctypes

import pytest
import torch

import _gate as G


@pytest.fixture(scope="module")
def lib():
    from combine_get_dispatch_counts_amd import _lib

    return _lib.load()


def test_calls_need_a_context(lib):
    p = ctypes.c_void_p(256)
    assert lib.epx_rms_norm(None, p, None, p, 0, 1, 8, 1e-6, None, p, None, None, None) == -1
    assert lib.epx_rms_norm_backward(None, p, p, p, 0, None, 1, 8, 1e-6, p, 64, p, p, None) == -1
    assert lib.epx_route(None, p, None, None, 1, 8, 2, 0, 1, 1, 1, 1.0, p, p, None) == -1
    assert lib.epx_balance_loss(None, p, p, None, 1, 8, 2, 1, 0, p, p, p, p, p, 1 << 20,
                                None) == -1
    assert lib.epx_route_backward(None, p, p, 1, 8, 2, 0, 1, 1.0, p, None, None, None, None, 1, p,
                                  None) == -1
    assert lib.epx_combine_backward(None, p, p, 1, 8, p, p, 1, 1, p, p, None) == -1


def test_workspaces(lib):
    for T, h in ((1, 8), (7, 7168), (4096, 7168), (1 << 20, 32768)):
        n = lib.epx_rms_norm_backward_workspace(T, h)
        assert n % (4 * h) == 0 and 1 <= n // (4 * h) <= min(T, 1024)
    for bad in ((0, 8), (-1, 8), (4, 12), (4, 0), (4, 32768 + 8)):
        assert lib.epx_rms_norm_backward_workspace(*bad) == 0
    for T, E, S in ((0, 8, 1), (1, 1, 1), (64, 256, 9), (32, 512, 1)):   # one launch
        assert lib.epx_balance_workspace(T, E, S) == 0
    assert lib.epx_balance_workspace(65, 8, 1) > 2 * 8 * 8
    assert 512 * 256 * 8 < lib.epx_balance_workspace(16384, 256, 24) < 600 * 256 * 8
    for bad in ((-1, 8, 1), (4, 0, 1), (4, 513, 1), (4, 8, 0)):
        assert lib.epx_balance_workspace(*bad) == 0


def test_binding_refuses_host_tensors():
    import combine_get_dispatch_counts_amd as epx

    x, w = torch.zeros((2, 8), dtype=torch.bfloat16), torch.ones(8)
    l, idx = torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int64)
    top, pos = torch.zeros((2, 2)), torch.zeros((2, 2), dtype=torch.int32)
    for call in (lambda: epx.rms_norm(x, w), lambda: epx.rms_norm(None, w),
                 lambda: epx.rms_norm_backward(x, x, w), lambda: epx.route(l, 2),
                 lambda: epx.balance_loss(l, idx),
                 lambda: epx.route_backward(l, idx, dtopk_weights=top),
                 lambda: epx.combine_backward(x, x, pos, top)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------- the 64-bit forms themselves

def test_reference_norm():
    v = torch.tensor([[3.0, 4.0, 0.0, 0.0]], dtype=torch.float64)
    y, inv = G.norm(v, torch.tensor([1.0, 2.0, 1.0, 1.0], dtype=torch.float64), 0.0)
    assert abs(float(inv) - 0.4) < 1e-15                          # sqrt(4 / 25)
    assert torch.allclose(y, torch.tensor([[1.2, 3.2, 0.0, 0.0]], dtype=torch.float64))


def _difference(f, x, step=1e-6):
    """The derivative of the number f(x) by central differences."""
    d = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = step
        e = e.view(x.shape)
        d.view(-1)[i] = (f(x + e) - f(x - e)) / (2 * step)
    return d


def test_reference_norm_backward_against_differences():
    g = G.gen(1)
    v, w, dout, dres = (torch.randn(s, generator=g, dtype=torch.float64)
                        for s in ((3, 6), (6,), (3, 6), (3, 6)))
    dx, _, dw, _ = G.norm_backward(dout, v, w, 1e-3, dres)
    f = lambda v, w: float((G.norm(v, w, 1e-3)[0] * dout).sum() + (v * dres).sum())  # noqa: E731
    assert torch.allclose(dx, _difference(lambda a: f(a, w), v), atol=1e-8)
    assert torch.allclose(dw, _difference(lambda a: f(v, a), w), atol=1e-8)


def test_reference_route():
    l = torch.log(torch.tensor([[4.0, 1.0, 3.0, 2.0]], dtype=torch.float64))
    idx, w, _ = G.route(l, 2, "softmax", normalize=False)
    assert idx.tolist() == [[0, 2]] and torch.allclose(w, torch.tensor([[0.4, 0.3]]).double())
    idx, w, _ = G.route(l, 2, "softmax", scale=7.0)
    assert torch.allclose(w, torch.tensor([[4.0, 3.0]]).double())
    # a bias moves the choice, not the weights
    idx, w, _ = G.route(l, 2, "softmax", bias=torch.tensor([0.0, 1.0, 0.0, 0.0]), normalize=False)
    assert idx.tolist() == [[1, 0]] and torch.allclose(w, torch.tensor([[0.1, 0.4]]).double())
    # groups {0, 1} (0.5) and {2, 3} (0.5) tie: the lower stays
    idx, _, _ = G.route(l, 3, "softmax", G=2, top=1)
    assert idx.tolist() == [[0, 1, -1]]
    # ties to the lower expert; -inf is never chosen
    l = torch.tensor([[1.0, 2.0, 2.0, -torch.inf]])
    idx, w, _ = G.route(l, 4, "sigmoid", normalize=False)
    assert idx.tolist() == [[1, 2, 0, -1]]
    assert abs(float(w[0, 0]) - 1 / (1 + 2.718281828459045 ** -2)) < 1e-15 and w[0, 3] == 0
    idx, w, _ = G.route(l, 2, "softmax", mask=torch.tensor([False]))
    assert idx.tolist() == [[-1, -1]] and not w.any()


def test_reference_balance():
    l = torch.zeros((4, 2), dtype=torch.float64)
    idx = torch.tensor([[0], [0], [1], [-1]])
    loss, counts, probs, n, _ = G.balance(l, idx, "softmax")
    assert counts.tolist() == [[2, 1]] and probs.tolist() == [[0.5, 0.5]]
    assert n.tolist() == [3, 1] and abs(loss - 1.0) < 1e-15       # 2 / 3 (2 / 2 + 1 / 2)
    loss, counts, _, n, _ = G.balance(l, idx, "sigmoid", [0, 1, 1, 3])
    assert counts.tolist() == [[1, 0], [0, 0], [1, 1]] and n.tolist() == [1, 0, 2, 2]
    # one token's loss is 2 (1 / 2), two sequences with tokens
    assert abs(loss - 1.0) < 1e-15


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_reference_route_backward_against_differences(scoring, normalize):
    g = G.gen(2)
    l = torch.randn((5, 6), generator=g, dtype=torch.float64)
    idx = torch.stack([torch.randperm(6, generator=g)[:3] for _ in range(5)])
    idx[1] = -1
    idx[2, 2] = -1
    d = torch.randn((5, 3), generator=g, dtype=torch.float64)
    off = [0, 2, 2, 4]
    _, counts, _, n, _ = G.balance(l, idx, scoring, off)

    def total(l):
        v = 0.0
        s, p = G.scores(l, scoring), G.shares(l, scoring)
        for t in range(5):
            ks = [k for k in range(3) if idx[t, k] >= 0]
            if ks:
                w = s[t, idx[t, ks]]
                v += float((d[t, ks] * (w / w.sum() if normalize else w)).sum()) * 2.5
        for q in range(3):                       # counts held constant
            for t in range(off[q], off[q + 1]):
                if int(n[q]) and (idx[t] >= 0).any():
                    v += 0.3 * float((counts[q] * p[t]).sum()) * 6 / (3 * int(n[q]) ** 2) / int(n[-1])
        return v

    got, _ = G.route_backward(l, idx, scoring, normalize, 2.5, d, counts, n, 0.3, off)
    assert torch.allclose(got, _difference(total, l), atol=1e-8)


def test_reference_combine_backward_against_differences():
    g = G.gen(3)
    dout, y = G.rows((2, 4), 4), G.rows((3, 4), 5)
    pos, w = torch.tensor([[2, 0], [-1, 1]]), torch.rand((2, 2), generator=g)
    dy, named, dw, _ = G.combine_backward(dout, y, pos, w)

    def total(y, w):
        out = torch.zeros((2, 4), dtype=torch.float64)
        for t in range(2):
            for k in range(2):
                if pos[t, k] >= 0:
                    out[t] += w[t, k] * y[pos[t, k]]
        return float((out * dout.double()).sum())

    assert named.all()
    assert torch.allclose(dw, _difference(lambda a: total(y.double(), a), w.double()), atol=1e-7)
    assert torch.allclose(dy.double(), _difference(lambda a: total(a, w.double()), y.double()),
                          rtol=G.BF16, atol=1e-7)
