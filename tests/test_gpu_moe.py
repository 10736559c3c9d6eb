"""GPU tests of the router, the products with expert weights and the whole
expert layer against their plain 64-bit definitions (moe_reference)."""
import ctypes

import numpy as np
import pytest
import torch

import moe_reference as R
from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu

FMT = dict(bf16=moe.EP_WEIGHT_BF16, mxfp4=moe.EP_WEIGHT_MXFP4, int4=moe.EP_WEIGHT_INT4)
SCORE = dict(softmax=moe.EP_SCORE_SOFTMAX, sigmoid=moe.EP_SCORE_SIGMOID)


def say(*a):
    print(*a, flush=True)


# ---- router ------------------------------------------------------------------

def run_gate(logits, K, bias=None, mask=None, dtype=torch.float32, score="softmax", renorm=True,
             groups=0, topk_groups=0, group_top=0, limit=False, scale=1.0):
    cfg = moe.GateConfig(logits.shape[1], K, SCORE[score], renorm, groups, topk_groups, group_top,
                         limit, scale)
    lg = torch.from_numpy(logits).cuda().to(dtype)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    m = None if mask is None else torch.from_numpy(mask).cuda()
    idx, w = moe.ep_gate(cfg, lg, b, m)
    ridx, rw = R.gate(lg.float().cpu().numpy(), K, score, renorm, bias, groups, topk_groups,
                      group_top, limit, scale, mask)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    # fp64 up to the one rounding to fp32
    assert np.allclose(w.cpu().numpy(), rw, rtol=2 * R.F32_HALF, atol=1e-44)
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,E,K", [(1, 256, 8), (3, 1, 1), (37, 64, 6), (65, 100, 5), (130, 128, 8),
                                   (9, 1024, 16), (5, 16, 16), (2, 513, 7)])
def test_gate(N, E, K, score, renorm):
    say(f"[gate] {N} {E} {K} {score} {renorm}")
    rng = np.random.default_rng(N * E + K)
    lg = (2 * rng.standard_normal((N, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    mask = rng.random(N) < 0.8
    run_gate(lg, K, score=score, renorm=renorm, scale=2.5)
    run_gate(lg, K, bias=bias, score=score, renorm=renorm, mask=mask)
    run_gate(lg, K, dtype=torch.bfloat16, score=score, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("limit", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("E,groups,topk_groups,top,K", [
    (256, 32, 4, 2, 8), (256, 8, 4, 2, 8), (60, 12, 3, 1, 3), (64, 2, 1, 5, 5), (128, 64, 5, 2, 10),
    (1024, 4, 2, 8, 16), (36, 4, 4, 9, 16)])
def test_gate_groups(E, groups, topk_groups, top, K, bias, limit, score):
    say(f"[gate groups] {E} {groups} {topk_groups} {top} {K} {bias} {limit} {score}")
    rng = np.random.default_rng(E + groups)
    lg = rng.standard_normal((41, E)).astype(np.float32)
    b = (0.3 * rng.standard_normal(E)).astype(np.float32) if bias else None
    run_gate(lg, K, bias=b, score=score, groups=groups, topk_groups=topk_groups, group_top=top,
             limit=limit)
    run_gate(lg, K, bias=b, score=score, groups=groups, topk_groups=topk_groups, group_top=top,
             limit=limit, dtype=torch.bfloat16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [0, 8])
def test_gate_odd_logits(groups, score):
    """Ties, infinities, NaN, rows with fewer eligible experts than K, none at
    all, and logits far apart."""
    say(f"[gate odd] {groups} {score}")
    rng = np.random.default_rng(5)
    E, K = 64, 6
    lg = np.round(rng.standard_normal((40, E)) * 2).astype(np.float32) / 2      # many ties
    lg[1] = 0
    lg[2] = -np.inf
    lg[3] = np.nan
    lg[4, 3:] = -np.inf
    lg[5, ::2] = np.nan
    lg[6, 7] = np.inf
    lg[7, [9, 30]] = np.inf
    lg[8] = rng.permutation(E) * 40 - 2000
    lg[9] = np.float32(3.0e38)
    lg[10] = np.float32(-3.0e38)
    lg[11] = rng.standard_normal(E) - 200
    lg[12, 5] = -0.0
    kw = dict(groups=groups, topk_groups=3, group_top=2) if groups else {}
    for renorm in (True, False):
        run_gate(lg, K, score=score, renorm=renorm, **kw)
        if groups:
            run_gate(lg, K, score=score, renorm=renorm, limit=True, **kw)
    bias = rng.standard_normal(E).astype(np.float32)
    bias[3], bias[4] = -np.inf, np.nan
    run_gate(lg, K, bias=bias, score=score, **kw)


def test_gate_near_ties_with_bias():
    """Choices one fp32 rounding apart: only the exact order passes."""
    rng = np.random.default_rng(8)
    E = 128
    lg = np.zeros((64, E), np.float32)
    lg += rng.integers(0, 3, (64, E)).astype(np.float32) * np.float32(2.0 ** -22)
    bias = rng.integers(0, 3, E).astype(np.float32) * np.float32(2.0 ** -24)
    for score in ("softmax", "sigmoid"):
        run_gate(lg, 8, bias=bias, score=score)
        run_gate(lg, 8, bias=bias, score=score, groups=16, topk_groups=4, group_top=2)


def test_gate_large_and_empty():
    rng = np.random.default_rng(1)
    lg = rng.standard_normal((3001, 256)).astype(np.float32)
    run_gate(lg, 8, bias=(0.1 * rng.standard_normal(256)).astype(np.float32), score="sigmoid",
             groups=32, topk_groups=4, group_top=2, limit=True)
    cfg = moe.GateConfig(256, 8)
    idx, w = moe.ep_gate(cfg, torch.zeros((0, 256), device="cuda"))
    assert idx.shape == w.shape == (0, 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K", [(1, 256, 8), (33, 7, 3), (70, 128, 8), (5, 1024, 16), (6, 300, 1)])
def test_gate_backward(N, E, K, dtype, renorm, score):
    say(f"[gate grad] {N} {E} {K} {dtype} {renorm} {score}")
    rng = np.random.default_rng(N + E)
    lg = torch.from_numpy((2 * rng.standard_normal((N, E))).astype(np.float32)).to(dtype)
    z = lg.float().numpy()
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K].astype(np.int32)
    idx[rng.random(idx.shape) < 0.1] = -1
    if N > 4:
        idx[2] = -1
        idx[3, 0], idx[3, K - 1] = E, -5               # outside: masked
        idx[4] = idx[4, 0]                             # one expert listed K times
    g = rng.standard_normal((N, K)).astype(np.float32)
    cfg = moe.GateConfig(E, K, SCORE[score], renorm, scale=2.5)
    got = moe.ep_gate_backward(cfg, lg.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(g).cuda())
    assert got.dtype == dtype
    want = R.gate_grad(z, idx, g, score, renorm, 2.5)
    # fp32: p to 2^-19 (exp of arguments up to 20), the dot over E or K terms;
    # every term is at most p (|g| + |dot|) <= 2 p max|g| 2.5
    scale = 2.5 * np.abs(g).max(axis=1, keepdims=True) * K
    tol = (2.0 ** -19 + 32 * R.F32_HALF) * 2 * scale + \
        (R.BF16_HALF if dtype == torch.bfloat16 else R.F32_HALF) * np.abs(want)
    assert (np.abs(got.float().cpu().numpy() - want) <= tol).all()


def test_gate_backward_of_masked_logits():
    """A chosen expert with a logit of -infinity, and rows of nothing else."""
    lg = torch.randn((4, 32), generator=torch.Generator().manual_seed(3))
    lg[0, 5] = -float("inf")
    lg[1] = -float("inf")
    lg[2, 4:] = float("nan")
    idx = torch.tensor([[5, 6, 7]] * 2 + [[0, 1, 2]] * 2, dtype=torch.int32).cuda()
    for score in SCORE.values():
        for renorm in (True, False):
            cfg = moe.GateConfig(32, 3, score, renorm)
            got = moe.ep_gate_backward(cfg, lg.cuda(), idx, torch.ones((4, 3), device="cuda"))
            assert torch.isfinite(got).all()
            assert got[0, 5] == 0 and (got[1] == 0).all()


# ---- products ------------------------------------------------------------------

def stack(fmt, E, M, C, group=0, zeros=False, seed=0):
    """(package weights on the GPU, float64 weights, magnitudes, terms)"""
    d, s, z = R.make_weights(fmt, E, M, C, group, zeros, seed)
    w, mag = R.dequant(fmt, d, s, z, group)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    return moe.Weights(FMT[fmt], cu(d), cu(s), cu(z), group=group), w, mag, \
        R.terms(C, group if fmt == "int4" else 0)


def rand_x(rows, C, seed):
    return torch.randn((rows, C), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


KINDS = [("bf16", 0, False), ("mxfp4", 32, False), ("int4", 32, False), ("int4", 32, True),
         ("int4", 64, False), ("int4", 64, True), ("int4", 128, False), ("int4", 128, True)]


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("rows,M,C", [(1, 64, 512), (1, 1, 128), (2, 33, 256), (5, 100, 384), (16, 48, 1152),
                                      (17, 31, 640), (33, 70, 896), (64, 16, 128), (65, 18, 256),
                                      (200, 40, 384), (3, 130, 4096)])
def test_matvec(rows, M, C, fmt, group, zeros):
    say(f"[matvec] {rows} {M} {C} {fmt} {group} {zeros}")
    w, w64, mag, n = stack(fmt, 1, M, C, group, zeros, seed=M + C)
    x = rand_x(rows, C, rows)
    for act in ([moe.EP_ACT_NONE] if M % 2 else [moe.EP_ACT_NONE, moe.EP_ACT_SWIGLU]):
        y = torch.full((rows + 1, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_matvec(w, x.cuda(), y[:rows], activation=act)
        want, err = R.product(x.double().numpy(), w64[0], mag[0], n, act)
        R.assert_close(y[:rows], want, err, (fmt, act))
        assert (y[rows:] == 77).all()


@pytest.mark.parametrize("fmt,group,C", [("bf16", 0, 8), ("bf16", 0, 24), ("bf16", 0, 1000), ("mxfp4", 32, 32),
                                         ("mxfp4", 32, 96), ("mxfp4", 32, 1056), ("int4", 32, 32),
                                         ("int4", 32, 160), ("int4", 64, 64), ("int4", 64, 192),
                                         ("int4", 128, 128), ("int4", 32, 2080)])
def test_matvec_ragged_columns(fmt, group, C):
    """Columns that end inside a 64-byte span, with an infinity in x there."""
    say(f"[matvec columns] {fmt} {group} {C}")
    w, w64, mag, n = stack(fmt, 1, 37, C, group, False, seed=C)
    x = rand_x(6, C, C)
    want, err = R.product(x.double().numpy(), w64[0], mag[0], n, 0)
    R.assert_close(moe.ep_matvec(w, x.cuda()), want, err)
    x[2, -1] = float("inf")
    y = moe.ep_matvec(w, x.cuda()).float().cpu()
    assert not torch.isfinite(y[2]).all()
    keep = [0, 1, 3, 4, 5]                     # the other rows are as before
    R.assert_close(y[keep].to(torch.bfloat16), want[keep], err[keep])


def test_matvec_every_code_and_scale():
    """Each code and scale byte of the 4-bit formats, one weight at a time:
    x = 1 on one column picks it."""
    E, M, C = 1, 256, 128
    data = torch.zeros((M, C // 2), dtype=torch.uint8)
    data[:, 5] = torch.arange(256, dtype=torch.uint8)      # columns 10 and 11
    x = torch.zeros((2, C), dtype=torch.bfloat16)
    x[0, 10] = x[1, 11] = 1
    for byte in (0, 1, 2, 64, 126, 127, 128, 130, 200, 250):
        scales = torch.full((M, C // 32), byte, dtype=torch.uint8)
        y = moe.ep_matvec(moe.Weights(moe.EP_WEIGHT_MXFP4, data.cuda(), scales.cuda()), x.cuda())
        lo, hi = R.E2M1[data[:, 5].numpy() & 15], R.E2M1[data[:, 5].numpy() >> 4]
        want = np.stack([lo, hi]) * 2.0 ** (byte - 127)
        got = y.float().cpu().numpy().astype(np.float64)
        if byte >= 2:       # below, bf16's subnormals may round or flush
            assert np.array_equal(got, want), byte
        else:
            assert (np.abs(got - want) <= 2.0 ** -126).all()
    scales[:] = 255
    y = moe.ep_matvec(moe.Weights(moe.EP_WEIGHT_MXFP4, data.cuda(), scales.cuda()), x.cuda())
    assert torch.isnan(y).all()
    for group in (32, 64, 128):
        for zero in (None, 0, 5, 15):
            s = torch.full((M, C // group), 0.375, dtype=torch.bfloat16)
            z = None if zero is None else torch.full(s.shape, zero, dtype=torch.uint8).cuda()
            y = moe.ep_matvec(moe.Weights(moe.EP_WEIGHT_INT4, data.cuda(), s.cuda(), z, group=group),
                              x.cuda())
            q = np.stack([data[:, 5].numpy() & 15, data[:, 5].numpy() >> 4]).astype(np.float64)
            want = (q - (8 if zero is None else zero)) * 0.375
            assert np.array_equal(y.float().cpu().numpy(), want), (group, zero)


def routed(N, E, K, mask=0.0, seed=0, skew=False, dup=False):
    rng = np.random.default_rng(seed)
    if dup:
        idx = rng.integers(0, E, (N, K))
    else:
        p = rng.random((N, E)) + (np.linspace(1.5, 0, E) if skew else 0)
        idx = np.argsort(-p, axis=1)[:, :K]
    idx = idx.astype(np.int32)
    idx[rng.random(idx.shape) < mask] = -1
    return idx, rng.random((N, K)).astype(np.float32)


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("N,E,K,align,cap,mask,sources,skew", [
    (1, 16, 2, 1, 0, 0.0, 1, False),
    (40, 8, 3, 1, 0, 0.1, 1, False),
    (40, 8, 3, 16, 0, 0.1, 1, True),
    (30, 33, 4, 1, 9, 0.0, 1, True),       # fixed capacity, some pairs dropped
    (24, 16, 2, 5, 0, 0.3, 4, False),      # stacked sources
    (300, 4, 2, 1, 0, 0.0, 1, False),      # many rows per expert
])
def test_expert_matvec(N, E, K, align, cap, mask, sources, skew, fmt, group, zeros):
    say(f"[experts] {N} {E} {K} {align} {cap} {fmt} {group} {zeros}")
    cfg = ep.Config(hidden=256, num_topk=K, num_experts=E, num_ranks=1, expert_alignment=align,
                    expert_capacity=cap, num_sources=sources)
    idx, _ = routed(N, E, K, mask, seed=N, skew=skew)
    h = ep.ep_handle_init(cfg, N)
    ep.ep_get_layout(h, torch.from_numpy(idx).cuda())
    ep.ep_check_error(h)                   # a full segment's flag
    v = ep.ep_handle_view(h)
    first, count = v["psum_expert"].cpu().numpy(), v["num_unaligned"].cpu().numpy()
    if cap:
        count = np.minimum(count, cap)
    rows = ep.ep_recv_capacity(cfg, N)
    M, C = 50, 256
    w, w64, mag, n = stack(fmt, E, M, C, group, zeros, seed=E)
    x = rand_x(rows, C, 3)
    live = np.zeros(rows, bool)
    for e in range(E):
        live[first[e]:first[e] + count[e]] = True
    xg = x.clone()
    xg[torch.from_numpy(~live)] = float("nan")         # padding rows are not read
    for act in (moe.EP_ACT_NONE, moe.EP_ACT_SWIGLU):
        y = torch.full((rows, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_expert_matvec(h, w, xg.cuda(), y, activation=act)
        assert ep.ep_check_error(h) == (ep.EP_OK, 0)
        want, err = np.full(y.shape, 77.0), np.zeros(y.shape)
        for e in range(E):
            s = slice(first[e], first[e] + count[e])
            want[s], err[s] = R.product(x[s].double().numpy(), w64[e], mag[e], n, act)
        assert (y.float().cpu().numpy()[~live] == 77).all()
        R.assert_close(y[torch.from_numpy(live).cuda()], want[live], err[live])


def test_expert_matvec_short_buffer_is_flagged():
    cfg = ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=1)
    idx, _ = routed(20, 4, 2, seed=1)
    h = ep.ep_handle_init(cfg, 20)
    ep.ep_get_layout(h, torch.from_numpy(idx).cuda())
    w, w64, mag, n = stack("bf16", 4, 24, 64)
    first = ep.ep_handle_view(h)["psum_expert"].cpu().numpy()
    x = rand_x(40, 64, 2)
    y = torch.full((40, 24), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_expert_matvec(h, w, x[:23].contiguous().cuda(), y[:23])
    st, flags = ep.ep_check_error(h)
    assert st == ep.EP_ERR_CAPACITY and flags == ep.EP_FLAG_RECV_CAPACITY
    e_of = np.searchsorted(first, np.arange(23), side="right") - 1
    for r in range(23):
        want, err = R.product(x[r:r + 1].double().numpy(), w64[e_of[r]], mag[e_of[r]], n, 0)
        R.assert_close(y[r:r + 1], want, err)
    assert (y[23:] == 77).all()
    moe.ep_expert_matvec(h, w, x[:0].cuda(), y[:0])
    assert ep.ep_check_error(h)[1] == ep.EP_FLAG_RECV_CAPACITY


def test_expert_matvec_states():
    w, *_ = stack("bf16", 4, 24, 64)
    x = rand_x(8, 64, 2).cuda()
    h = ep.ep_handle_init(ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=1), 4)
    with pytest.raises(ep.EpError) as ei:
        moe.ep_expert_matvec(h, w, x)
    assert ei.value.status == ep.EP_ERR_STATE
    hn = ep.ep_handle_init(ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=2, non_expand=True), 4)
    ep.ep_get_layout(hn, torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ep.EpError) as ei:
        moe.ep_expert_matvec(hn, w, x)
    assert ei.value.status == ep.EP_ERR_INVALID_ARG
    ep.ep_get_layout(h, torch.full((4, 2), -1, dtype=torch.int32, device="cuda"))   # nothing to do
    y = torch.full((8, 24), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_expert_matvec(h, w, x, y)
    assert (y == 77).all() and ep.ep_check_error(h) == (ep.EP_OK, 0)


# ---- whole layer ---------------------------------------------------------------

def layer_case(N, E, K, H, I, fmt, group=0, zeros=False, mask=0.0, seed=0, dup=False, skew=False,
               wts=True):
    cfg = ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1)
    idx, w = routed(N, E, K, mask, seed, dup=dup, skew=skew)
    up, down = stack(fmt, E, 2 * I, H, group, zeros, seed=1), stack(fmt, E, H, I, group, zeros, seed=2)
    x = rand_x(N, H, seed)
    h = ep.ep_handle_init(cfg, 1)
    want, err = R.layer(x.double().numpy(), idx, w if wts else None, up[1:3], down[1:3], up[3], down[3])
    return dict(h=h, x=x.cuda(), idx=torch.from_numpy(idx).cuda(), up=up[0], down=down[0],
                w=torch.from_numpy(w).cuda() if wts else None, want=want, err=err)


def run_layer(c, **kw):
    return moe.ep_moe_layer(c["h"], c["up"], c["down"], c["x"], c["idx"], c["w"], **kw)


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("N,E,K,H,I,mask,dup,skew", [
    (1, 16, 2, 256, 128, 0.0, False, False),
    (1, 8, 8, 128, 384, 0.0, False, False),
    (2, 1, 1, 384, 128, 0.0, False, False),
    (7, 16, 4, 640, 256, 0.1, False, False),
    (16, 8, 3, 256, 384, 0.0, False, False),
    (17, 12, 5, 256, 128, 0.3, True, False),
    (40, 4, 2, 384, 256, 0.1, True, True),
    (70, 3, 2, 128, 128, 0.0, False, True),
])
def test_layer(N, E, K, H, I, mask, dup, skew, fmt, group, zeros):
    say(f"[layer] {N} {E} {K} {H} {I} {mask} {dup} {fmt} {group} {zeros}")
    c = layer_case(N, E, K, H, I, fmt, group, zeros, mask, seed=N + K, dup=dup, skew=skew)
    out = torch.full((N + 1, H), 77.0, dtype=torch.bfloat16, device="cuda")
    run_layer(c, out=out[:N])
    assert ep.ep_check_error(c["h"]) == (ep.EP_OK, 0)
    R.assert_close(out[:N], c["want"], c["err"])
    assert (out[N:] == 77).all()


@pytest.mark.parametrize("N,E,K,H,I,mask", [
    (4, 3, 4, 128, 128, 0.2),        # one expert several times in a row
    (3, 2, 16, 128, 128, 0.0),
    (16, 5, 4, 384, 128, 0.1),       # 16 tokens, 64 pairs: the most of a handful
    (13, 5, 5, 256, 128, 0.1),       # 65 pairs: one more
    (17, 5, 2, 256, 128, 0.0),       # 17 tokens
    (8, 4, 8, 128, 512, 0.0),        # activations past 64 KB
])
@pytest.mark.parametrize("fmt,group", [("bf16", 0), ("mxfp4", 32), ("int4", 128)])
def test_layer_handful(N, E, K, H, I, mask, fmt, group):
    """Around the limits of the batches that are summed inside the down
    projection, with ids listed more than once."""
    say(f"[layer handful] {N} {E} {K} {H} {I} {fmt}")
    c = layer_case(N, E, K, H, I, fmt, group, seed=N + K, mask=mask, dup=True)
    R.assert_close(run_layer(c), c["want"], c["err"])


@pytest.mark.parametrize("N", [5, 24])
def test_layer_keeps_nan_with_the_tokens_that_chose_it(N):
    """An expert of NaN weights (and a NaN row of x): the other tokens do not
    see them."""
    for fmt, group in (("bf16", 0), ("mxfp4", 32), ("int4", 64)):
        c = layer_case(N, 6, 2, 128, 64, fmt, group, seed=3)
        idx = c["idx"].cpu().numpy()
        idx[idx == 5] = 4
        idx[2] = [5, 1]
        c["idx"].copy_(torch.from_numpy(idx))
        want = run_layer(c).clone()
        assert torch.isfinite(want).all()
        for w in (c["up"], c["down"]):
            if fmt == "bf16":
                w.data[5] = float("nan")
            elif fmt == "mxfp4":
                w.scales[5] = 255
            else:
                w.scales[5] = float("inf")
        c["x"][N - 1] = float("nan")
        got = run_layer(c)
        keep = [t for t in range(N) if t not in (2, N - 1)]
        assert torch.equal(got[keep], want[keep]), fmt
        assert not torch.isfinite(got[2]).any() and torch.isnan(got[N - 1]).all()


@pytest.mark.parametrize("fmt,H,I", [("bf16", 72, 40), ("bf16", 8, 8), ("mxfp4", 96, 32), ("mxfp4", 32, 160)])
@pytest.mark.parametrize("N", [1, 5, 20])
def test_layer_odd_sizes(N, fmt, H, I):
    say(f"[layer odd] {N} {fmt} {H} {I}")
    c = layer_case(N, 9, 3, H, I, fmt, 32 if fmt == "mxfp4" else 0, seed=N)
    R.assert_close(run_layer(c), c["want"], c["err"])


@pytest.mark.parametrize("N", [1, 3, 18])
def test_layer_without_weights_or_experts(N):
    c = layer_case(N, 6, 2, 128, 64, "bf16", wts=False, seed=4)
    R.assert_close(run_layer(c), c["want"], c["err"])
    c["idx"].fill_(-1)
    out = torch.full((N, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    run_layer(c, out=out)
    assert (out.view(torch.int16) == 0).all()                # +0
    # masked entries' weights are not looked at, an expert of another row is
    c = layer_case(N, 6, 2, 128, 64, "bf16", seed=4)
    c["idx"][0, 0] = -1
    c["w"][0, 0] = float("nan")
    assert torch.isfinite(run_layer(c)).all()


@pytest.mark.parametrize("N", [2, 30])
def test_layer_bad_ids_are_flagged(N):
    c = layer_case(N, 6, 2, 128, 64, "mxfp4", 32, seed=4)
    idx = c["idx"].clone()
    c["idx"][1, 0] = -1
    want = run_layer(c).clone()
    for bad in (6, -2, 1 << 30, -(1 << 31)):
        c["idx"].copy_(idx)
        c["idx"][1, 0] = bad
        out = run_layer(c)
        st, flags = ep.ep_check_error(c["h"])
        assert st == ep.EP_ERR_DEVICE_INDEX and flags == ep.EP_FLAG_BAD_EXPERT_ID
        assert torch.equal(out, want)


def test_layer_largest_batch_of_one_expert():
    """256 tokens that all choose the same experts: row blocks past the first,
    and the batch limit."""
    N, H, I = 256, 128, 64
    c = layer_case(N, 2, 2, H, I, "bf16", seed=9)
    R.assert_close(run_layer(c), c["want"], c["err"])
    big = torch.zeros((257, H), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ep.EpError):
        moe.ep_moe_layer(c["h"], c["up"], c["down"], big,
                         torch.zeros((257, 2), dtype=torch.int32, device="cuda"))
    # sixteen entries a token, one expert
    c = layer_case(256, 1, 1, 64, 32, "bf16", seed=3)
    h = ep.ep_handle_init(ep.Config(hidden=64, num_topk=16, num_experts=1, num_ranks=1), 1)
    idx = torch.zeros((256, 16), dtype=torch.int32, device="cuda")
    w = torch.full((256, 16), 0.0625, device="cuda")
    w16 = moe.ep_moe_layer(h, c["up"], c["down"], c["x"], idx, w)
    c["w"].fill_(1.0)
    one = run_layer(c).double().cpu().numpy()
    # the same value, summed in sixteen equal parts
    assert (np.abs(w16.double().cpu().numpy() - one) <= 2 * R.BF16_HALF * np.abs(one) + 1e-6).all()


@pytest.mark.parametrize("N", [1, 8, 33])
def test_layer_in_place_and_guarded_workspace(N):
    c = layer_case(N, 8, 2, 256, 96, "mxfp4", 32, seed=6)
    want = run_layer(c).clone()
    size = moe.ep_moe_workspace_size(c["h"], c["up"], c["down"], N)
    ws = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    x = c["x"].clone()
    got = moe.ep_moe_layer(c["h"], c["up"], c["down"], x, c["idx"], c["w"], out=x, workspace=ws[:size])
    assert torch.equal(got, want) and (ws[size:] == 0xA5).all()
    with pytest.raises(ep.EpError) as ei:
        run_layer(c, workspace=ws[:size - 1])
    assert ei.value.status == ep.EP_ERR_WORKSPACE
    with pytest.raises(ep.EpError) as ei:
        run_layer(c, workspace=ws[16:])
    assert ei.value.status == ep.EP_ERR_WORKSPACE


@pytest.mark.parametrize("N,K", [(1, 4), (20, 4)])
def test_layer_keeps_the_handle(N, K):
    """The handle's layout is the same before and after."""
    c = layer_case(N, 16, K, 128, 64, "bf16", seed=6)
    h = ep.ep_handle_init(c["h"].cfg, 50)
    other, _ = routed(50, 16, K, seed=11)
    ep.ep_get_layout(h, torch.from_numpy(other).cuda())
    before = {k: v.clone() for k, v in ep.ep_handle_view(h).items() if torch.is_tensor(v)}
    c["h"] = h
    R.assert_close(run_layer(c), c["want"], c["err"])
    after = ep.ep_handle_view(h)
    assert after["num_tokens"] == 50
    for k, v in before.items():
        assert torch.equal(v, after[k]), k


@pytest.mark.parametrize("N", [1, 12, 40])
def test_layer_graph_replays(N):
    """A captured layer against the eager one, with new inputs and eager work
    between the replays."""
    c = layer_case(N, 8, 3, 256, 128, "int4", 64, True, seed=2)
    ws = torch.empty(moe.ep_moe_workspace_size(c["h"], c["up"], c["down"], N), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["x"])
    run_layer(c, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_layer(c, out=out, workspace=ws)
    for i in range(4):
        c["x"].copy_(rand_x(N, 256, 50 + i).cuda())
        idx, w = routed(N, 8, 3, 0.2, seed=60 + i)
        c["idx"].copy_(torch.from_numpy(idx))
        c["w"].copy_(torch.from_numpy(w))
        out.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_layer(c)), i
    assert ep.ep_check_error(c["h"]) == (ep.EP_OK, 0)


def test_calls_follow_the_current_stream():
    c = layer_case(3, 8, 2, 256, 128, "mxfp4", 32, seed=2)
    want = run_layer(c).clone()
    s = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x = torch.zeros_like(c["x"])
        for _ in range(10):
            big = big @ big * 1e-3
        x.copy_(c["x"])                       # queued behind the products above
        got = moe.ep_moe_layer(c["h"], c["up"], c["down"], x, c["idx"], c["w"])
    s.synchronize()
    assert torch.equal(got, want)


def test_large_offsets():
    """A stack past 4 GiB: its last expert's rows, and a row length whose tile
    is far from its base."""
    E, M, C = 300, 2048, 8192
    data = torch.zeros((E, M, C // 2), dtype=torch.uint8, device="cuda")      # 2.5 GB
    data[-1] = torch.randint(0, 256, (M, C // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, M, C // 32), 120, dtype=torch.uint8, device="cuda")
    d2 = torch.zeros((E, M, C), dtype=torch.bfloat16, device="cuda")          # 10 GB
    d2[-1].normal_(0, 0.01)
    x = torch.randn((1, C), device="cuda").to(torch.bfloat16)
    h = ep.ep_handle_init(ep.Config(hidden=C, num_topk=1, num_experts=E, num_ranks=1), 1)
    ep.ep_get_layout(h, torch.full((1, 1), E - 1, dtype=torch.int32, device="cuda"))
    for fmt, d, s in (("mxfp4", data, scales), ("bf16", d2, None)):
        w64, mag = R.dequant(fmt, d[-1:].cpu(), None if s is None else s[-1:].cpu(), None, 0)
        y = moe.ep_expert_matvec(h, moe.Weights(FMT[fmt], d, s), x)
        want, err = R.product(x.double().cpu().numpy(), w64[0], mag[0], R.terms(C, 0), 0)
        R.assert_close(y, want, err, fmt)


# ---- refusals that need a handle (the pointers are never used) -------------------

PTR = 0x10000


def _w(**kw):
    return moe.ep_weights(*{**dict(format=moe.EP_WEIGHT_INT4, group=32, num_experts=1, rows=64, cols=128,
                                   reserved=0, d_data=PTR, d_scales=PTR, d_zeros=None), **kw}.values())


@pytest.mark.parametrize("up,down,n,ok", [
    ({}, {}, 256, True), ({}, {}, 257, False), ({}, {}, -1, False),
    (dict(rows=96), {}, 4, False), (dict(cols=256), {}, 4, False), ({}, dict(rows=256), 4, False),
    (dict(num_experts=3), {}, 4, False), ({}, dict(num_experts=5), 4, False), (dict(rows=63), {}, 4, False),
])
def test_layer_sizes(up, down, n, ok):
    """The layer's stacks against the handle: refused before anything runs."""
    h = ep.ep_handle_init(ep.Config(hidden=128, num_topk=2, num_experts=4, num_ranks=1), 1)
    raw = h.ptr
    wu = _w(**{**dict(num_experts=4, rows=64, cols=128), **up})
    wd = _w(**{**dict(num_experts=4, rows=128, cols=32), **down})
    out = ctypes.c_int64(-1)
    st = moe._lib().ep_moe_workspace_size(raw, ctypes.byref(wu), ctypes.byref(wd), n, ctypes.byref(out))
    assert st == (ep.EP_OK if ok else ep.EP_ERR_INVALID_ARG)
    if ok:      # two terms of the activations and each pair's output
        assert out.value >= n * 2 * (4 * 32 + 4 * 128) and out.value % 256 == 0
    else:
        assert moe._lib().ep_moe_layer(raw, ctypes.byref(wu), ctypes.byref(wd), PTR, PTR, PTR, n, PTR, PTR,
                                       1 << 30, None) == ep.EP_ERR_INVALID_ARG


def test_layer_refuses_sizes_past_32_bits_and_bad_pointers():
    held = ep.ep_handle_init(ep.Config(hidden=1 << 24, num_topk=16, num_experts=4, num_ranks=1), 1)
    big = held.ptr
    wu = _w(num_experts=4, rows=64, cols=1 << 24)
    wd = _w(num_experts=4, rows=1 << 24, cols=32)
    L, out = moe._lib(), ctypes.c_int64()
    assert L.ep_moe_workspace_size(big, ctypes.byref(wu), ctypes.byref(wd), 256, ctypes.byref(out)) == \
        ep.EP_ERR_INVALID_ARG
    assert L.ep_moe_workspace_size(big, ctypes.byref(wu), ctypes.byref(wd), 64, ctypes.byref(out)) == ep.EP_OK
    small = ep.ep_handle_init(ep.Config(hidden=128, num_topk=2, num_experts=4, num_ranks=1), 1)
    h = small.ptr
    wu, wd = _w(num_experts=4, rows=64, cols=128), _w(num_experts=4, rows=128, cols=32)
    good = [PTR, PTR, PTR, 4, PTR, PTR, 1 << 30]
    for i, v in ((0, None), (0, PTR + 8), (1, None), (1, PTR + 2), (2, PTR + 2), (4, None), (4, PTR + 8)):
        a = list(good)
        a[i] = v
        assert L.ep_moe_layer(h, ctypes.byref(wu), ctypes.byref(wd), *a, None) == ep.EP_ERR_INVALID_ARG
    for i, v in ((5, None), (5, PTR + 128), (6, 1000)):
        a = list(good)
        a[i] = v
        assert L.ep_moe_layer(h, ctypes.byref(wu), ctypes.byref(wd), *a, None) == ep.EP_ERR_WORKSPACE
    assert L.ep_moe_layer(h, ctypes.byref(wu), ctypes.byref(wd), None, None, None, 0, None, None, 0, None) == ep.EP_OK


# ---- together -------------------------------------------------------------------

@pytest.mark.parametrize("fmt,group", [("bf16", 0), ("mxfp4", 32), ("int4", 64)])
@pytest.mark.parametrize("N", [1, 29])
def test_router_to_output_both_ways(N, fmt, group):
    """gate -> layout -> dispatch -> products -> combine, and gate -> layer."""
    E, K, H, I = 32, 4, 256, 128
    up, down = stack(fmt, E, 2 * I, H, group, seed=1), stack(fmt, E, H, I, group, seed=2)
    x = rand_x(N, H, 8)
    logits = np.random.default_rng(N).standard_normal((N, E)).astype(np.float32)
    gcfg = moe.GateConfig(E, K, moe.EP_SCORE_SIGMOID, num_groups=8, topk_groups=3, group_top=2)
    idx, w = moe.ep_gate(gcfg, torch.from_numpy(logits).cuda())
    ridx, rw = R.gate(logits, K, "sigmoid", groups=8, topk_groups=3, group_top=2)
    assert np.array_equal(idx.cpu().numpy(), ridx)

    cfg = ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=4, expert_alignment=4)
    h = ep.ep_handle_init(cfg, N)
    rows = ep.ep_recv_capacity(cfg, N)
    recv = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    ep.ep_layout_dispatch(h, idx, x.cuda(), recv)
    act = moe.ep_expert_matvec(h, up[0], recv, activation=moe.EP_ACT_SWIGLU)
    y = moe.ep_expert_matvec(h, down[0], act)
    out = torch.empty((N, H), dtype=torch.bfloat16, device="cuda")
    ep.ep_combine(h, y, w, out)
    assert ep.ep_check_error(h) == (ep.EP_OK, 0)

    layer = moe.ep_moe_layer(h, up[0], down[0], x.cuda(), idx, w)
    want, err = R.layer(x.double().numpy(), ridx, rw, up[1:3], down[1:3], up[3], down[3])
    R.assert_close(layer, want, err)
    # the shuffled path rounds a and each expert's output to bf16 as well
    extra = np.zeros_like(want)
    for t in range(N):
        for k in range(K):
            a = R.product(x[t:t + 1].double().numpy(), up[1][ridx[t, k]], up[2][ridx[t, k]], up[3], 1)[0]
            extra[t] += rw[t, k] * R.BF16_HALF * (
                np.abs(a) @ np.abs(down[1][ridx[t, k]]).T + np.abs(a @ down[1][ridx[t, k]].T))[0]
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 1.01 * (err + extra) + R.BF16_HALF * (np.abs(want) + err + extra)).all()
