"""That the exact comparisons of long sums reject what they are there for:
mistakes planted into the expected results (CPU)."""
import pytest
import torch

import _experts as X
import _experts_exact as XE

STEP = 128   # bytes of a row that a kernel takes at a time


def _planted(fp8, K, unit, rows_w, seed):
    """Operands of one expert, and its sums with one step treated wrongly."""
    x, xs, w, ws = XE.operands(fp8, 24, 1, rows_w, K, seed, unit)
    v = X.rows64(x, xs)
    m = X.weights64(w[0], None if ws is None else ws[0])
    step, steps = STEP // (1 if fp8 else 2), K * (1 if fp8 else 2) // STEP
    wrong = {}
    for at in (0, steps // 2, steps - 1):
        part = v[:, at * step:(at + 1) * step] @ m[:, at * step:(at + 1) * step].T
        wrong[f"without step {at}"] = v @ m.T - part
        wrong[f"step {at} twice"] = v @ m.T + part
        wrong[f"half of step {at}"] = v @ m.T - part / 2
    wrong["zeros"] = torch.zeros_like(v @ m.T)
    return v @ m.T, wrong


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K", [256, 20608, 65536])
def test_sums_reject_planted_mistakes(K, fp8):
    y, wrong = _planted(fp8, K, 0, 64, 5)
    assert (y.float().double() == y).all()
    XE.assert_sums(y.float().to(torch.bfloat16), y, "right")
    for what, bad in wrong.items():
        with pytest.raises(AssertionError):
            XE.assert_sums(bad.float().to(torch.bfloat16), y, what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K", [20608, 65536])
def test_activations_reject_planted_mistakes(K, fp8):
    y, wrong = _planted(fp8, K, XE.UNIT, 256, 6)
    assert (y.float().double() == y).all()

    def result(y):
        a, _ = XE.activation(y)
        if not fp8:
            return a.float().to(torch.bfloat16), None
        q, s = XE.quantized_rows(a.float())
        pad = torch.zeros((q.shape[0], X.stride(q.shape[1])))
        pad[:, :s.shape[1]] = s
        return q, pad

    XE.assert_activation(*result(y), y, "right")
    for what, bad in wrong.items():
        with pytest.raises(AssertionError):
            XE.assert_activation(*result(bad), y, what)


def test_bounds_from_magnitudes_do_not():
    """Why these exist: over 65536 channels of random values the bound of
    sums in any order is wider than the results, so zeros pass it."""
    x, w = X.randn((4, 65536), 45), X.randn((32, 65536), 46, 65536 ** -0.5)
    a, tol = X.gated(x.double(), w.double())
    X.assert_close(torch.zeros_like(a), a, tol, "zeros")
