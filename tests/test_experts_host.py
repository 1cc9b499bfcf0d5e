"""What the experts' calls refuse before any GPU work, and the 64-bit forms
the GPU tests compare with, checked against hand-worked values (CPU)."""
import ctypes

import pytest
import torch

import _experts as X


@pytest.fixture(scope="module")
def lib():
    from combine_get_dispatch_counts_amd import _lib

    return _lib.load()


def test_decode_workspace(lib):
    assert lib.epx_moe_decode_workspace(1, 8, 2048) == 8 * 2048 * 2
    assert lib.epx_moe_decode_workspace(64, 32, 8) == 64 * 32 * 8 * 2
    for bad in ((0, 8, 64), (65, 8, 64), (-1, 8, 64), (1, 0, 64), (1, 33, 64), (1, 8, 4),
                (1, 8, 65536 + 8)):
        assert lib.epx_moe_decode_workspace(*bad) == 0


def test_calls_need_a_context(lib):
    p = ctypes.c_void_p(256)
    assert lib.epx_quantize_weights(None, p, 1, 8, 128, p, p, None) == -1
    assert lib.epx_grouped_gemm(None, p, None, 1, 8, p, None, 1, 8, 0, p, p, None) == -1
    assert lib.epx_grouped_swiglu(None, p, None, 1, 8, p, None, 1, 8, 0, p, p, None, None) == -1
    assert lib.epx_ll_grouped_gemm(None, p, None, 8, p, None, 1, 8, 0, p, 1, 1, p, None) == -1
    assert lib.epx_ll_grouped_swiglu(None, p, None, 8, p, None, 1, 8, 0, p, 1, 1, p, None,
                                     None) == -1
    assert lib.epx_moe_decode(None, p, 8, p, p, 1, 1, 1, p, None, p, None, 8, 0, p, 16, p,
                              None) == -1


def test_binding_refuses_host_tensors():
    import combine_get_dispatch_counts_amd as epx

    x, w = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros((1, 16, 8), dtype=torch.bfloat16)
    off = torch.tensor([0, 2], dtype=torch.int32)
    for call in (epx.grouped_gemm, epx.grouped_swiglu):
        with pytest.raises(ValueError):
            call(x, w, off)
        with pytest.raises(ValueError):
            call(None, w, off)
    with pytest.raises(ValueError):
        epx.ll_grouped_gemm(x, w, off[:1], 2)
    with pytest.raises(ValueError):
        epx.quantize_weights(torch.zeros((1, 8, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        epx.moe_decode(x, torch.zeros((2, 1), dtype=torch.int64), torch.ones((2, 1)), w,
                       torch.zeros((1, 8, 8), dtype=torch.bfloat16))


def test_reference_products():
    x = torch.tensor([[1.0, 2.0], [0.0, -1.0]], dtype=torch.float64)
    w = torch.tensor([[3.0, 4.0], [5.0, -6.0]], dtype=torch.float64)
    y, tol = X.product(x, w)
    assert y.tolist() == [[11.0, -7.0], [-4.0, 6.0]]
    assert tol.tolist() == [[11.0 * 10 * X.U32, 17.0 * 10 * X.U32], [4.0 * 10 * X.U32, 6.0 * 10 * X.U32]]
    a, _ = X.gated(x, w)                      # gate: row 0 of w, up: row 1
    g = 11.0 / (1.0 + 2.718281828459045 ** -11.0)
    assert abs(float(a[0, 0]) - g * -7.0) < 1e-12


def test_reference_scales():
    x = torch.full((1, 256), 0x38, dtype=torch.uint8)            # e4m3 of 1
    s = torch.zeros((1, X.stride(256)))
    s[0, 0], s[0, 1] = 2.0, 3.0
    v = X.rows64(x, s)
    assert (v[0, :128] == 2).all() and (v[0, 128:] == 3).all()
    w = torch.full((130, 128), 0x38, dtype=torch.uint8)
    v = X.weights64(w, torch.tensor([[0.5], [0.25]]))
    assert (v[:128] == 0.5).all() and (v[128:] == 0.25).all()
    with pytest.raises(AssertionError):       # a wrong value is found
        X.assert_close(torch.tensor([1.0]), torch.tensor([1.1]), torch.tensor([0.05]), "planted")


def test_reference_cut():
    """256 * 256 beside a product of 8: 8 is the last bit kept (2^16 / 2^13)."""
    one = torch.zeros((4, 128), dtype=torch.float8_e4m3fn)
    x, w = one.clone(), one.clone()
    x[:, 0] = w[:, 0] = 256.0
    x[:, 1], w[:, 1] = 2.0, torch.tensor([4.0, 7.5, -7.5, 3.5]).to(torch.float8_e4m3fn)
    x[:, 8], w[:, 8] = 1.0, 0.5                     # another eight: whole
    y, mag = X.cut_product(x.view(torch.uint8), w.view(torch.uint8))
    assert y.tolist() == [65544.5, 65544.5, 65528.5, 65536.5]
    assert mag[1] == 65551.5
    c = X.cut(x.view(torch.uint8), torch.full((4, X.stride(128)), 2.0), w.view(torch.uint8),
              torch.full((1, 1), 3.0))
    # the first eight, the second (1 * 0.5), fourteen of zeros (2^-6 each)
    assert abs(float(c[0, 0]) - 6 * 7 * 2.0 ** -13 * (65536 + 0.5 + 14 * 2.0 ** -12)) < 1e-9
