"""CPU-only checks of the products in 8-bit integers: refusals of the C calls
(made before any HIP call) and of the binding."""
import ctypes

import pytest
import torch

from combine_get_dispatch_layout_amd import ep, moe

PTR = 0x10000          # aligned, never dereferenced: the calls under test fail before
GOOD_W = dict(format=moe.EP_WEIGHT_INT8, group=0, num_experts=1, rows=64, cols=128, reserved=0, d_data=PTR,
              d_scales=PTR, d_zeros=None)


def _w(**kw):
    return moe.ep_weights(*{**GOOD_W, **kw}.values())


def _message():
    return ep.lib().ep_last_error_message().decode()


def _matmul(w, x=PTR, xs=PTR, n=1, act=0, y=PTR):
    return moe._lib().ep_matmul(None if w is None else ctypes.byref(w), x, xs, n, act, y, None)


@pytest.mark.parametrize("bad", [
    dict(format=4), dict(format=-1), dict(format=moe.EP_WEIGHT_INT4, group=32), dict(format=moe.EP_WEIGHT_BF16),
    dict(group=32), dict(group=128), dict(num_experts=0), dict(num_experts=1025), dict(num_experts=2), dict(rows=0),
    dict(rows=(1 << 24) + 1), dict(cols=0), dict(cols=-16), dict(cols=8), dict(cols=120), dict(cols=1 << 17),
    dict(cols=1 << 24), dict(reserved=1), dict(d_data=None), dict(d_data=PTR + 8), dict(d_scales=None),
    dict(d_scales=PTR + 2), dict(d_zeros=PTR),
])
def test_weight_refusals(bad):
    assert _matmul(_w(**bad)) == ep.EP_ERR_INVALID_ARG
    assert "moe_api.cpp:" in _message()


def test_int8_weights_are_for_these_calls_alone():
    w = _w()
    assert moe._lib().ep_matvec(ctypes.byref(w), PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG
    assert "INT8" in _message()


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=PTR + 8), dict(xs=None), dict(xs=PTR + 2), dict(n=-1), dict(n=1 << 31), dict(act=2), dict(act=-1),
    dict(y=None), dict(y=PTR + 1),
])
def test_matmul_refusals(bad):
    assert _matmul(_w(), **bad) == ep.EP_ERR_INVALID_ARG
    assert _matmul(None) == ep.EP_ERR_INVALID_ARG
    assert _matmul(_w(rows=33), act=1) == ep.EP_ERR_INVALID_ARG
    assert _matmul(_w(rows=1 << 24), n=1 << 11) == ep.EP_ERR_INVALID_ARG        # 2^35 outputs
    assert _matmul(_w(), x=None, xs=None, n=0, y=None) == ep.EP_OK               # no rows
    w = _w(num_experts=4)
    assert moe._lib().ep_expert_matmul(None, ctypes.byref(w), PTR, PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG


def test_binding_weights():
    z = torch.zeros
    i8 = torch.int8
    for args in ((z((4, 16), dtype=torch.uint8), z(4)), (z((4, 16), dtype=i8),), (z((4, 16), dtype=i8), z(5)),
                 (z((4, 16), dtype=i8), z((4, 1))), (z((4, 16), dtype=i8), z(4, dtype=torch.bfloat16)),
                 (z((2, 4, 16), dtype=i8), z(4)), (z((4, 16), dtype=i8), z(4), z(4)), (z(16, dtype=i8), z(16)),
                 (z((4, 16), dtype=i8), z(4), None, 32)):
        with pytest.raises(ValueError):
            moe.Weights(moe.EP_WEIGHT_INT8, *args)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.Weights(moe.EP_WEIGHT_INT8, z((4, 16), dtype=i8), z(4))


class _FakeWeights(moe.Weights):
    """A descriptor without GPU tensors, for the checks that come before."""

    def __init__(self, E, rows, cols):
        self.num_experts, self.rows, self.cols = E, rows, cols
        self.device = torch.device("cpu")
        self._ref = None


def test_binding_products():
    w, odd = _FakeWeights(4, 32, 64), _FakeWeights(4, 33, 64)
    x, s = torch.zeros((6, 64), dtype=torch.int8), torch.zeros(6)
    h = ep.Handle.__new__(ep.Handle)
    h.cfg, h.max_tokens, h.workspace = ep.Config(64, 2, 4, 1), 8, torch.empty(0, dtype=torch.uint8)
    h._device, h._ptr = torch.device("cpu"), ctypes.c_void_p()
    for call in (moe.ep_matmul, lambda *a, **k: moe.ep_expert_matmul(h, *a, **k)):
        for bad in (x.float(), x.to(torch.uint8), x[:, :32], x[0]):
            with pytest.raises(ValueError, match="x must be"):
                call(w, bad, s)
        for bad in (s[:5], s.double(), s[None], s[:, None].expand(6, 2), s.reshape(6, 1, 1)):
            with pytest.raises(ValueError, match="x_scales must be"):
                call(w, x, bad)
        with pytest.raises(ValueError, match="activation"):
            call(w, x, s, activation=3)
        with pytest.raises(ValueError, match="even"):
            call(odd, x, s, activation=moe.EP_ACT_SWIGLU)
        with pytest.raises(ValueError, match="y must be"):
            call(w, x, s, torch.zeros((6, 31), dtype=torch.bfloat16))
