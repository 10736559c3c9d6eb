"""CPU-only checks of include/ep_moe.h: declarations, exports, the refusals of
the C calls (made before any HIP call) and of the binding, and the reference
gradient of moe_reference against differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import moe_reference as R
from combine_get_dispatch_layout_amd import ep, moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD_GATE = dict(num_experts=64, num_topk=8)
PTR = 0x10000          # aligned, never dereferenced: the calls under test fail before


def test_header_binding_and_exports_agree():
    with open(os.path.join(ROOT, "include", "ep_moe.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_[a-z_]+)\s*\(", text)))
    assert names == sorted(moe.SYMBOLS)
    L = moe._lib()
    for n in names:
        assert hasattr(L, n), n


def _gate(n=4, logits=PTR, bias=None, idx=PTR, w=PTR, dtype=torch.float32, **kw):
    cfg = moe.GateConfig(**{**GOOD_GATE, **kw})
    return moe._lib().ep_gate(cfg.c(dtype), logits, bias, None, n, idx, w, None)


def _message():
    return ep.lib().ep_last_error_message().decode()


@pytest.mark.parametrize("bad", [
    dict(num_experts=0), dict(num_experts=1025), dict(num_topk=0), dict(num_topk=17),
    dict(num_topk=9, num_experts=8), dict(scoring=2), dict(scoring=-1), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(num_groups=-1), dict(num_groups=65, num_experts=650),
    dict(num_groups=7, topk_groups=2, group_top=1), dict(num_groups=8, topk_groups=0, group_top=1),
    dict(num_groups=8, topk_groups=9, group_top=1), dict(num_groups=8, topk_groups=2, group_top=0),
    dict(num_groups=8, topk_groups=2, group_top=9),
    dict(num_groups=8, topk_groups=3, group_top=2, group_limit=True),     # holds 6 of 8
    dict(num_groups=32, topk_groups=3, group_top=2),                      # holds 6 of 8
    dict(n=-1), dict(n=1 << 31), dict(logits=None), dict(idx=None), dict(w=None),
    dict(logits=PTR + 2), dict(idx=PTR + 1), dict(w=PTR + 2), dict(bias=PTR + 1),
    dict(logits=PTR + 1, dtype=torch.bfloat16),
])
def test_gate_refusals(bad):
    assert _gate(**bad) == ep.EP_ERR_INVALID_ARG
    assert "moe_api.cpp:" in _message()
    names = ("n", "logits", "bias", "idx", "w", "dtype")
    cfg = moe.GateConfig(**{**GOOD_GATE, **{k: v for k, v in bad.items() if k not in names}})
    if "bias" not in bad:
        st = moe._lib().ep_gate_backward(cfg.c(bad.get("dtype", torch.float32)), bad.get("logits", PTR),
                                         bad.get("idx", PTR), bad.get("w", PTR), bad.get("n", 4), PTR, None)
        assert st == ep.EP_ERR_INVALID_ARG


def test_gate_without_tokens_needs_no_pointers():
    assert _gate(n=0, logits=None, idx=None, w=None) == ep.EP_OK
    assert moe._lib().ep_gate(None, PTR, None, None, 1, PTR, PTR, None) == ep.EP_ERR_INVALID_ARG
    assert moe._lib().ep_gate_backward(moe.GateConfig(**GOOD_GATE).c(torch.float32), PTR, PTR, PTR, 4,
                                       None, None) == ep.EP_ERR_INVALID_ARG


GOOD_W = dict(format=moe.EP_WEIGHT_INT4, group=32, num_experts=1, rows=64, cols=128, reserved=0,
              d_data=PTR, d_scales=PTR, d_zeros=None)


def _w(**kw):
    return moe.ep_weights(*{**GOOD_W, **kw}.values())


BAD_WEIGHTS = [
    dict(format=3), dict(format=-1), dict(num_experts=0), dict(num_experts=1025), dict(rows=0),
    dict(rows=(1 << 24) + 1), dict(cols=0), dict(cols=(1 << 24) + 32), dict(reserved=1), dict(group=16),
    dict(group=256), dict(group=0), dict(cols=144), dict(group=128, cols=192), dict(d_data=None),
    dict(d_data=PTR + 8), dict(d_scales=None), dict(d_scales=PTR + 8), dict(d_zeros=PTR + 4),
    dict(format=moe.EP_WEIGHT_MXFP4, group=64), dict(format=moe.EP_WEIGHT_MXFP4, d_zeros=PTR),
    dict(format=moe.EP_WEIGHT_BF16), dict(format=moe.EP_WEIGHT_BF16, group=0),          # scales
    dict(format=moe.EP_WEIGHT_BF16, group=0, d_scales=None, cols=100),
    dict(format=moe.EP_WEIGHT_BF16, group=0, d_scales=None, d_zeros=PTR),
]


@pytest.mark.parametrize("bad", BAD_WEIGHTS)
def test_weight_refusals(bad):
    w = _w(**bad)
    assert moe._lib().ep_matvec(ctypes.byref(w), PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG
    assert "moe_api.cpp:" in _message()


@pytest.mark.parametrize("args", [
    (None, 1, 0, PTR), (PTR, -1, 0, PTR), (PTR, 1 << 31, 0, PTR), (PTR, 1, 2, PTR), (PTR, 1, -1, PTR),
    (PTR, 1, 0, None), (PTR + 8, 1, 0, PTR), (PTR, 1, 0, PTR + 1),
])
def test_matvec_refusals(args):
    w = _w()
    assert moe._lib().ep_matvec(ctypes.byref(w), *args, None) == ep.EP_ERR_INVALID_ARG
    assert moe._lib().ep_matvec(None, PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG
    odd = _w(rows=33)
    assert moe._lib().ep_matvec(ctypes.byref(odd), PTR, 1, 1, PTR, None) == ep.EP_ERR_INVALID_ARG
    two = _w(num_experts=2)
    assert moe._lib().ep_matvec(ctypes.byref(two), PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG
    assert moe._lib().ep_matvec(ctypes.byref(w), None, 0, 0, None, None) == ep.EP_OK      # no rows


def test_handle_calls_refuse_null():
    w = _w()
    r = ctypes.byref(w)
    out = ctypes.c_int64()
    L = moe._lib()
    assert L.ep_expert_matvec(None, r, PTR, 1, 0, PTR, None) == ep.EP_ERR_INVALID_ARG
    assert L.ep_moe_workspace_size(None, r, r, 1, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert L.ep_moe_layer(None, r, r, PTR, PTR, PTR, 1, PTR, PTR, 1 << 20, None) == ep.EP_ERR_INVALID_ARG


# ---- the binding ---------------------------------------------------------------


def test_binding_gate_checks():
    cfg = moe.GateConfig(**GOOD_GATE)
    z = torch.zeros
    for bad in (z((4, 63)), z((4, 64), dtype=torch.float16), z(64)):
        with pytest.raises(ValueError, match="logits"):
            moe.ep_gate(cfg, bad)
        with pytest.raises(ValueError, match="logits"):
            moe.ep_gate_backward(cfg, bad, z((4, 8), dtype=torch.int32), z((4, 8)))
    lg = z((4, 64))
    for kw in (dict(bias=z(63)), dict(bias=z(64, dtype=torch.bfloat16)), dict(token_mask=z(5, dtype=torch.bool)),
               dict(token_mask=z(4)), dict(topk_idx=z((4, 8), dtype=torch.int64)), dict(topk_weights=z((3, 8)))):
        with pytest.raises(ValueError, match="must be"):
            moe.ep_gate(cfg, lg, **kw)
    for args in ((z((4, 8)), z((4, 8))), (z((4, 7), dtype=torch.int32), z((4, 8))),
                 (z((4, 8), dtype=torch.int32), z((4, 8), dtype=torch.float64)),
                 (z((4, 8), dtype=torch.int32), z((4, 8)), z((4, 64), dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="must be"):
            moe.ep_gate_backward(cfg, lg, *args)


def test_binding_gate_with_a_gradient():
    """The checks are those without one."""
    cfg = moe.GateConfig(**GOOD_GATE)
    lg = torch.zeros((4, 64), requires_grad=True)
    for kw in (dict(bias=torch.zeros(63)), dict(topk_idx=torch.zeros((4, 8), dtype=torch.int64)),
               dict(topk_weights=torch.zeros((3, 8)))):
        with pytest.raises(ValueError, match="must be"):
            moe.ep_gate(cfg, lg, **kw)
    for grad in (True, False):
        with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="on the GPU"):
            moe.ep_gate(cfg, lg)


def test_binding_weights_checks():
    z = torch.zeros
    u8, bf = torch.uint8, torch.bfloat16
    for args in ((9, z((4, 8), dtype=bf)), (moe.EP_WEIGHT_BF16, z((4, 8))), (moe.EP_WEIGHT_BF16, z(8, dtype=bf)),
                 (moe.EP_WEIGHT_BF16, z((4, 8), dtype=bf), z((4, 1))), (moe.EP_WEIGHT_MXFP4, z((4, 16), dtype=u8)),
                 (moe.EP_WEIGHT_MXFP4, z((4, 16), dtype=u8), z((4, 1))),
                 (moe.EP_WEIGHT_MXFP4, z((4, 16), dtype=u8), z((4, 2), dtype=u8)),
                 (moe.EP_WEIGHT_MXFP4, z((4, 16), dtype=u8), z((4, 1), dtype=u8), z((4, 1), dtype=u8)),
                 (moe.EP_WEIGHT_INT4, z((4, 16), dtype=u8), z((4, 1), dtype=bf)),          # no group
                 (moe.EP_WEIGHT_INT4, z((4, 16), dtype=u8), z((4, 1), dtype=bf), None, 64),
                 (moe.EP_WEIGHT_INT4, z((4, 16), dtype=u8), z((4, 1), dtype=bf), z((4, 1)), 32)):
        with pytest.raises(ValueError):
            moe.Weights(*args)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.Weights(moe.EP_WEIGHT_BF16, z((4, 8), dtype=bf))


class _FakeWeights(moe.Weights):
    """A descriptor without GPU tensors, for the checks that come before."""

    def __init__(self, E, rows, cols):
        self.num_experts, self.rows, self.cols = E, rows, cols
        self.device = torch.device("cpu")
        self._ref = None


def _fake_handle():
    h = ep.Handle.__new__(ep.Handle)
    h.cfg = ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=1)
    h.max_tokens, h.workspace, h._device = 8, torch.empty(0, dtype=torch.uint8), torch.device("cpu")
    h._ptr = ctypes.c_void_p()
    return h


def test_binding_product_and_layer_checks():
    bf = torch.bfloat16
    w, odd = _FakeWeights(4, 32, 64), _FakeWeights(4, 33, 64)
    x = torch.zeros((6, 64), dtype=bf)
    for bad in (x.float(), x[:, :32], x[0]):
        with pytest.raises(ValueError, match="x must be"):
            moe.ep_matvec(w, bad)
    with pytest.raises(ValueError, match="activation"):
        moe.ep_matvec(w, x, activation=3)
    with pytest.raises(ValueError, match="even"):
        moe.ep_matvec(odd, x, activation=moe.EP_ACT_SWIGLU)
    with pytest.raises(ValueError, match="y must be"):
        moe.ep_expert_matvec(_fake_handle(), w, x, torch.zeros((6, 31), dtype=bf))
    h, up, down = _fake_handle(), _FakeWeights(4, 32, 64), _FakeWeights(4, 64, 16)
    idx, wt = torch.zeros((6, 2), dtype=torch.int32), torch.zeros((6, 2))
    for args in ((x.float(), idx, wt), (x[:, :32], idx, wt), (x, idx.long(), wt), (x, idx[:5], wt),
                 (x, idx, wt.double()), (x, idx, wt, x.float()), (x, idx, wt, x[:5])):
        with pytest.raises(ValueError, match="must be"):
            moe.ep_moe_layer(h, up, down, *args)


# ---- the reference itself --------------------------------------------------------


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((5, 12))
    idx = np.argsort(-z, axis=1)[:, :4].astype(np.int32)
    idx[1, 2], idx[2] = -1, -1
    idx[3, 1] = idx[3, 0]
    g = rng.standard_normal((5, 4))
    got = R.gate_grad(z, idx, g, score, renorm, 1.5)
    step = 1e-5
    for t in range(5):
        for e in range(12):
            zp, zm = z.copy(), z.copy()
            zp[t, e] += step
            zm[t, e] -= step
            d = ((R.gate_weights(zp, idx, score, renorm, 1.5) -
                  R.gate_weights(zm, idx, score, renorm, 1.5)) * g).sum() / (2 * step)
            # central differences: step^2 times a third derivative below 10,
            # and 2^-53 / step of rounding
            assert abs(d - got[t, e]) <= 10 * step ** 2 + 1e-10


def test_reference_gate_by_hand():
    lg = np.array([[1.0, 3.0, 2.0, 0.0, 3.0, -1.0, 0.5, 2.5]], np.float32)
    idx, w = R.gate(lg, 3)
    assert idx.tolist() == [[1, 4, 7]] and abs(w.sum() - 1) < 1e-12
    idx, _ = R.gate(lg, 2, groups=4, topk_groups=1, group_top=2)
    assert idx.tolist() == [[1, 0]]             # groups {0,1} and {2,3} ... by summed softmax
    idx, _ = R.gate(lg, 2, groups=4, topk_groups=2, group_top=1, limit=True)
    assert idx.tolist() == [[1, 4]]


def grad_case(N, E, K, seed=0):
    """Logits, a choice with masked, foreign and repeated entries, gradients."""
    rng = np.random.default_rng(seed + N + E)
    z = (2 * rng.standard_normal((N, E))).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K].astype(np.int32)
    idx[rng.random(idx.shape) < 0.1] = -1
    if N > 4:
        idx[2] = -1
        idx[3, 0], idx[3, K - 1] = E, -5
        idx[4] = idx[4, 0]
    return z, idx, rng.standard_normal((N, K)).astype(np.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,E,K", [(1, 256, 8), (33, 7, 3), (70, 128, 8), (5, 1024, 16), (6, 300, 2)])
@pytest.mark.parametrize("half", [R.F32_HALF, R.BF16_HALF])
def test_gradient_bound_sees_what_it_should(half, N, E, K, renorm, score):
    """The bound holds the definition and tells left-out terms from it."""
    z, idx, g = grad_case(N, E, K)
    g = g.astype(np.float64)
    want, tol = R.gate_grad_bound(z, idx, g, score, renorm, 2.5, half)
    np.testing.assert_allclose(want, R.gate_grad(z, idx, g, score, renorm, 2.5), rtol=1e-9, atol=1e-12)
    ok = (idx >= 0) & (idx < E)
    chosen = np.zeros(z.shape, bool)
    t, k = ok.nonzero()
    chosen[t, idx[t, k]] = True
    live = chosen.any(1)
    if renorm:      # without the common term
        p = np.where(ok, R.gate_weights(z.astype(np.float64), idx, score, True, 1.0), 0)
        q = 1 / (1 + np.exp(z[np.arange(N)[:, None], np.where(ok, idx, 0)])) if score == "sigmoid" else 1.0
        wrong = np.zeros(z.shape)
        np.add.at(wrong, (t, idx[t, k]), (2.5 * p * q * g)[t, k])
        several = (ok.sum(1) > 1)[:, None] & chosen
        assert (np.abs(wrong - want) > tol)[several].mean() > 0.9
    if score == "softmax" and not renorm:
        rest = ~chosen & live[:, None]
        assert (np.abs(want) > 10 * tol)[rest].mean() > 0.9 if half == R.F32_HALF else \
            (np.abs(want) > tol)[rest].all()
        s = np.exp(z - z.max(1, keepdims=True).astype(np.float64))
        s /= s.sum(1, keepdims=True)
        gs = np.zeros(z.shape)
        np.add.at(gs, (t, idx[t, k]), 2.5 * g[t, k])
        assert (np.abs(s * gs - want) > tol)[live].mean() > 0.9       # no dot term
    # one bf16 step is outside an fp32 bound
    if half == R.F32_HALF:
        big = np.abs(want) > 1e-6
        assert (np.abs(want * 2.0 ** -9) > tol)[big].mean() > 0.9
