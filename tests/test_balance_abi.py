"""CPU-only checks of the balance loss: refusals of the C calls (made before
any HIP call) and of the binding, and the reference gradient against
differences."""
import ctypes

import numpy as np
import pytest
import torch

import balance_reference as B
from combine_get_dispatch_layout_amd import ep, moe

GOOD = dict(num_experts=64, num_topk=8)
PTR = 0x10000          # aligned, never dereferenced: the calls under test fail before
CALL = dict(logits=PTR, idx=PTR, mask=None, n=4, start=None, q=1, loss=PTR, counts=PTR, tokens=PTR, sums=PTR,
            ws=PTR, size=1 << 30)


def _message():
    return ep.lib().ep_last_error_message().decode()


def _split(kw):
    call = {**CALL, **{k: v for k, v in kw.items() if k in CALL}}
    cfg = moe.BalanceConfig(**{**GOOD, **{k: v for k, v in kw.items() if k not in CALL and k != "dtype"}})
    return cfg.c(kw.get("dtype", torch.float32)), call


def _forward(**kw):
    cfg, c = _split(kw)
    return moe._lib().ep_balance_loss(cfg, c["logits"], c["idx"], c["mask"], c["n"], c["start"], c["q"], c["loss"],
                                      c["counts"], c["tokens"], c["sums"], c["ws"], c["size"], None)


def _backward(**kw):
    cfg, c = _split(kw)
    return moe._lib().ep_balance_loss_backward(cfg, c["logits"], c["mask"], c["n"], c["start"], c["q"], c["counts"],
                                               c["tokens"], c["loss"], c["sums"], None)


BAD = [
    dict(num_experts=0), dict(num_experts=1025), dict(num_topk=0), dict(num_topk=17), dict(num_topk=9, num_experts=8),
    dict(scoring=2), dict(scoring=-1), dict(coefficient=float("inf")), dict(coefficient=float("nan")), dict(n=-1),
    dict(n=1 << 31), dict(n=1 << 28), dict(n=1 << 62), dict(q=0), dict(q=-1), dict(q=2),
    dict(q=(1 << 18) + 1, start=PTR), dict(start=PTR + 2), dict(logits=None), dict(logits=PTR + 2),
    dict(logits=PTR + 1, dtype=torch.bfloat16), dict(counts=None), dict(counts=PTR + 2), dict(tokens=None),
    dict(tokens=PTR + 1), dict(loss=None), dict(loss=PTR + 2), dict(sums=None), dict(sums=PTR + 1),
]


@pytest.mark.parametrize("bad", BAD + [dict(idx=None), dict(idx=PTR + 1)])
def test_forward_refusals(bad):
    assert _forward(**bad) == ep.EP_ERR_INVALID_ARG
    assert "moe_api.cpp:" in _message()


@pytest.mark.parametrize("bad", BAD)
def test_backward_refusals(bad):
    assert _backward(**bad) == ep.EP_ERR_INVALID_ARG
    assert "moe_api.cpp:" in _message()


def test_normalize_and_type_must_be_known():
    L = moe._lib()
    for fields in ((64, 8, 1, 2, 0, 1.0), (64, 8, 0, -1, 0, 1.0), (64, 8, 0, 1, 2, 1.0)):
        c = moe.ep_balance_config(*fields)
        out = ctypes.c_int64()
        assert L.ep_balance_workspace_size(ctypes.byref(c), 4, 1, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert L.ep_balance_workspace_size(None, 4, 1, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert L.ep_balance_loss_backward(moe.BalanceConfig(**GOOD).c(torch.float32), None, None, 0, None, 1, None, None,
                                      None, None, None) == ep.EP_OK      # no tokens


def test_workspace():
    cfg = moe.BalanceConfig(**GOOD)
    sizes = [moe.ep_balance_workspace_size(cfg, n, q) for n, q in ((0, 1), (1, 1), (4096, 1), (4096, 1000), (1 << 27, 1))]
    assert all(s > 0 for s in sizes) and sizes[2] < sizes[3]
    assert sizes[4] < (1 << 27) * 64 * 4 // 64         # a small share of the logits
    need = moe.ep_balance_workspace_size(cfg, 4, 1)
    assert _forward(size=need - 1) == ep.EP_ERR_WORKSPACE and str(need) in _message()
    assert _forward(ws=None) == ep.EP_ERR_WORKSPACE
    assert _forward(ws=PTR + 128) == ep.EP_ERR_WORKSPACE
    with pytest.raises(ep.EpError):
        moe.ep_balance_workspace_size(cfg, 4, 0)


def test_binding_checks():
    cfg = moe.BalanceConfig(**GOOD)
    z, i32 = torch.zeros, torch.int32
    lg, idx = z((4, 64)), z((4, 8), dtype=i32)
    for bad in (z((4, 63)), z((4, 64), dtype=torch.float16), z(64)):
        with pytest.raises(ValueError, match="logits"):
            moe.ep_balance_loss(cfg, bad, idx)
        with pytest.raises(ValueError, match="logits"):
            moe.ep_balance_loss_backward(cfg, bad, z((1, 64), dtype=i32), z(1, dtype=i32), z(()))
    for kw in (dict(token_mask=z(4)), dict(token_mask=z(3, dtype=torch.bool)), dict(seq_start=z(3)),
               dict(seq_start=z(1, dtype=i32)), dict(seq_start=z((2, 2), dtype=i32)), dict(loss=z(1)),
               dict(counts=z((1, 64))), dict(counts=z((2, 64), dtype=i32)), dict(seq_tokens=z(2, dtype=i32)),
               dict(score_sums=z((1, 63)))):
        for grad in (True, False):
            with pytest.raises(ValueError, match="must be"):
                moe.ep_balance_loss(cfg, lg.clone().requires_grad_(grad), idx, **kw)
    for bad in (idx.long(), z((4, 7), dtype=i32), z((5, 8), dtype=i32)):
        with pytest.raises(ValueError, match="topk_idx"):
            moe.ep_balance_loss(cfg, lg, bad)
    good = dict(counts=z((1, 64), dtype=i32), seq_tokens=z(1, dtype=i32), grad_loss=z(()))
    for kw in (dict(counts=z((2, 64), dtype=i32)), dict(seq_tokens=z(1)), dict(grad_loss=z(1)),
               dict(grad_loss=z((), dtype=torch.float64)), dict(token_mask=z(4)), dict(grad_logits=z((4, 63))),
               dict(grad_logits=z((4, 64), dtype=torch.bfloat16)), dict(seq_start=z(2))):
        with pytest.raises(ValueError, match="must be"):
            moe.ep_balance_loss_backward(cfg, lg, **{**good, **kw})
    with pytest.raises(ValueError, match="on the GPU"):
        moe.ep_balance_loss(cfg, lg, idx)


# ---- the reference itself --------------------------------------------------------

START = [0, 3, 3, 7, 9]


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("sigmoid", True), ("sigmoid", False)])
def test_reference_gradient_against_differences(score, normalize):
    rng = np.random.default_rng(4)
    z = rng.standard_normal((10, 6))
    idx = np.argsort(-z, axis=1)[:, :2].astype(np.int32)
    idx[1, 1] = -1
    mask = np.ones(10, bool)
    mask[4] = False
    kw = dict(score=score, normalize=normalize, coefficient=0.5, start=START, mask=mask)
    n, T = B.counts(idx, 6, START, mask), np.array([len(t) for t in B.tokens_of(START, mask, 10)])
    got, _ = B.gradient(z, n, T, 2, g=1.5, **kw)
    step = 1e-5
    for t in range(10):
        for e in range(6):
            zp, zm = z.copy(), z.copy()
            zp[t, e] += step
            zm[t, e] -= step
            d = 1.5 * (B.balance(zp, idx, **kw)[0] - B.balance(zm, idx, **kw)[0]) / (2 * step)
            # step^2 times a third derivative below 10, and 2^-53 / step of rounding
            assert abs(d - got[t, e]) <= 10 * step ** 2 + 1e-10
    assert (got[[4, 9]] == 0).all() and got[0].any()


def test_reference_loss_by_hand():
    """Even use of the experts costs the coefficient, all tokens on one expert
    with all score there E times as much."""
    z = np.zeros((8, 4))
    idx = np.stack([np.arange(8) % 4, (np.arange(8) + 1) % 4], axis=1).astype(np.int32)
    assert abs(B.balance(z, idx, coefficient=0.25)[0] - 0.25) < 1e-12
    z[:, 2] = 100
    assert abs(B.balance(z, np.full((8, 1), 2, np.int32))[0] - 4) < 1e-12
    loss, n, T, S, *_ = B.balance(np.zeros((4, 2)), np.array([[0], [0], [1], [5]], np.int32), start=[0, 2, 4])
    assert n.tolist() == [[2, 0], [0, 1]] and T.tolist() == [2, 2] and S.tolist() == [[1, 1], [1, 1]]
    assert abs(loss - (2 / 4 * 2 + 2 / 4 * 1) / 2) < 1e-12


def test_gradient_bound_sees_what_it_should():
    """The bound is far below the gradient's terms: with f the counts less the
    even share, each is at most p F of 2 max |f|, and the errors sum to fewer than
    (|a| < 16) + 40 + 24 of the dot, 2 and (|a| + 56) of the rest: 160 u < 2^-16
    of it.  And it tells a left-out common term."""
    rng = np.random.default_rng(6)
    z = rng.standard_normal((60, 32)).astype(np.float32) + rng.standard_normal(32).astype(np.float32)
    idx = np.argsort(-z, axis=1)[:, :4].astype(np.int32)
    n, T = B.counts(idx, 32), np.array([60])
    for score, normalize in (("softmax", True), ("sigmoid", True), ("sigmoid", False)):
        got, err = B.gradient(z, n, T, 4, score, normalize)
        p, rest, _ = B.scores(z, score, normalize)
        f = n[0] - (4 * 60 // 32 if score == "softmax" or normalize else 0)
        assert (err <= 2.0 ** -16 * p * 32 / (4 * 60.0 ** 2) * 2 * np.abs(f).max() + 1e-30).all()
        wrong = p * (rest if score == "sigmoid" else 1) * 32 / (4 * 60.0 ** 2) * n[0]     # no common term
        if score == "softmax" or normalize:
            assert (np.abs(wrong - got) > err).mean() > 0.99
        else:
            np.testing.assert_allclose(wrong, got, rtol=1e-12)
