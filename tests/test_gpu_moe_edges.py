"""GPU tests of the router, the products and the expert layer where results can
go wrong without a plain case showing it."""
import numpy as np
import pytest
import torch

import moe_reference as R
from test_moe_abi import grad_case
from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


# ---- INT4: what the codes' offset costs -----------------------------------------

def int4(codes, group, zero, scale):
    """An INT4 stack of one matrix with one scale and one zero (None: 8)."""
    M, C = codes.shape
    data = torch.from_numpy((codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)).cuda()
    s = torch.full((M, C // group), scale, dtype=torch.bfloat16, device="cuda")
    z = None if zero is None else torch.full((M, C // group), zero, dtype=torch.uint8, device="cuda")
    return moe.Weights(moe.EP_WEIGHT_INT4, data, s, z, group=group)


@pytest.mark.parametrize("rows", [1, 9, 20])
@pytest.mark.parametrize("zero", [None, 5, 0, 15])
@pytest.mark.parametrize("group,C", [(32, 512), (32, 160), (64, 512), (64, 192), (128, 512), (128, 384)])
def test_int4_large_columns_of_zero_weight(group, C, zero, rows):
    """Each group has a column of x = 2^17 whose weight is 0; the others are
    multiples of 1/4 up to 1.  With codes as 16 + q every partial sum is a
    multiple of 1/4 of at most 31 * 2^17 + 31 * 127 < 2^22 (exact in fp32), so
    y is the exact sum, rounded once."""
    say(f"[int4 offset] {group} {C} {zero} {rows}")
    rng = np.random.default_rng(C + rows)
    M, z = 37, 8 if zero is None else zero
    codes = rng.integers(0, 16, (M, C))
    x = rng.integers(-4, 5, (rows, C)) / 4
    big = np.arange(0, C, group) + rng.integers(0, group, C // group)
    codes[:, big] = z
    x[:, big] = 2.0 ** 17 * rng.choice([-1, 1], (rows, len(big)))
    y = moe.ep_matvec(int4(codes, group, zero, 1.0), torch.from_numpy(x).to(torch.bfloat16).cuda())
    want = torch.from_numpy(x @ (codes - z).T).float().to(torch.bfloat16)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_x_near_the_largest(group, rows):
    """One column of 2^121: (16 + q) x is at most 31 * 2^121 < 2^126, so the
    product is exact; the other columns are zeros."""
    rng = np.random.default_rng(group)
    codes = rng.integers(0, 16, (33, 256))
    for zero in (None, 0, 15):
        x = torch.zeros((rows, 256), dtype=torch.bfloat16)
        x[:, 77] = 2.0 ** 121
        y = moe.ep_matvec(int4(codes, group, zero, 2.0 ** -20), x.cuda())
        want = (codes[:, 77] - (8 if zero is None else zero)) * 2.0 ** 101
        assert np.array_equal(y.double().cpu().numpy(), np.broadcast_to(want, (rows, 33)))


# ---- router: batches whose threads pass 32 bits ------------------------------------

def test_gate_of_more_threads_than_32_bits():
    """2^26 tokens at one wave each are 2^32 threads."""
    N = (1 << 26) + 5
    lg = torch.randint(-2, 3, (N, 2), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    cfg = moe.GateConfig(2, 1, moe.EP_SCORE_SIGMOID, renormalize=False, scale=4.0)
    idx, w = moe.ep_gate(cfg, lg)
    second = lg[:, 1] > lg[:, 0]
    assert torch.equal(idx[:, 0], second.int())
    top = torch.where(second, lg[:, 1], lg[:, 0]).float()
    # the five logits' weights: sigmoids rounded once
    for v in range(-2, 3):
        got = w[:, 0][top == v]
        assert got.numel() == 0 or (got.min() == got.max() and
                                    abs(float(got[0]) / 4 * (1 + np.exp(-v)) - 1) <= 2 * R.F32_HALF)
    del w, top
    grad = moe.ep_gate_backward(cfg, lg, idx, torch.ones((N, 1), device="cuda"))
    assert torch.equal(grad != 0, torch.stack((~second, second), 1))
    assert (grad[-5:].float().sum(1) > 0).all()


def test_shuffle_of_more_threads_than_32_bits():
    """2^26 rows of one wave each: refused as one launch, right in two ranges."""
    N = (1 << 26) + 320
    cfg = ep.Config(hidden=8, num_topk=1, num_experts=1, num_ranks=1)
    h = ep.ep_handle_init(cfg, N)
    ep.ep_get_layout(h, torch.zeros((N, 1), dtype=torch.int32, device="cuda"), alloc_outputs=False)
    x = torch.randint(-9, 9, (N, 8), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    recv = torch.full_like(x, 77)
    out = torch.full_like(x, 77)
    for call in (lambda **kw: ep.ep_dispatch(h, x, recv, **kw), lambda **kw: ep.ep_combine(h, recv, None, out, **kw)):
        with pytest.raises(ep.EpError) as ei:
            call()
        assert ei.value.status == ep.EP_ERR_HIP and "configuration" in str(ei.value)
        call(token_begin=0, token_end=N // 2)
        call(token_begin=N // 2, token_end=N)
    assert torch.equal(recv, x) and torch.equal(out, x)
    assert ep.ep_check_error(h) == (ep.EP_OK, 0)


# ---- router: the weights' gradient through autograd ----------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gate_weights_have_the_gradient(score, renorm, dtype):
    N, E, K = 19, 40, 4
    cfg = moe.GateConfig(E, K, dict(softmax=0, sigmoid=1)[score], renorm, scale=2.5)
    g = torch.Generator().manual_seed(4)
    lg = torch.randn((N, E), generator=g).to(dtype).cuda().requires_grad_()
    gw = torch.randn((N, K), generator=g).cuda()
    mask = (torch.arange(N) % 5 != 0).cuda()
    bias = torch.randn(E, generator=g).cuda()
    idx, w = moe.ep_gate(cfg, lg, bias, mask)
    assert w.requires_grad and not idx.requires_grad
    with torch.no_grad():
        ridx, rw = moe.ep_gate(cfg, lg, bias, mask)
    assert torch.equal(idx, ridx) and torch.equal(w, rw) and not rw.requires_grad
    want = moe.ep_gate_backward(cfg, lg.detach(), idx, gw)
    assert (want[mask] != 0).any(1).all() and (want[~mask] == 0).all()
    w.backward(gw)
    assert lg.grad.dtype == dtype and torch.equal(lg.grad, want)
    # a gradient that is a broadcast scalar; a second use adds up
    lg.grad = None
    _, w = moe.ep_gate(cfg, lg, bias, mask)
    (w.sum() + (w * gw).sum()).backward()
    assert torch.equal(lg.grad, moe.ep_gate_backward(cfg, lg.detach(), idx, 1 + gw))
    # through what made the logits
    x, r = torch.randn((N, 8), generator=g).cuda(), torch.randn((8, E), generator=g).cuda().requires_grad_()
    z = x @ r
    _, w = moe.ep_gate(cfg, z, bias)
    w.backward(gw)
    with torch.no_grad():
        i, _ = moe.ep_gate(cfg, z, bias)
        assert torch.equal(r.grad, x.t() @ moe.ep_gate_backward(cfg, z.detach(), i, gw))


def test_gate_gradient_with_given_outputs():
    """Buffers that every step fills again: they keep no graph, and each step's
    gradient is that of its own choice."""
    cfg = moe.GateConfig(8, 2)
    a, b = (torch.randn((5, 8), device="cuda", requires_grad=True) for _ in range(2))
    idx, w = torch.empty((5, 2), dtype=torch.int32, device="cuda"), torch.empty((5, 2), device="cuda")
    gw = torch.randn((5, 2), device="cuda")
    want = []
    for z in (a, b):
        with torch.no_grad():
            i, _ = moe.ep_gate(cfg, z)
            want.append(moe.ep_gate_backward(cfg, z, i, gw))
    ia, wa = moe.ep_gate(cfg, a, topk_idx=idx, topk_weights=w)
    assert ia.data_ptr() == idx.data_ptr() and wa.data_ptr() == w.data_ptr()
    assert wa.requires_grad and not w.requires_grad and w.grad_fn is None
    _, wb = moe.ep_gate(cfg, b, topk_idx=idx, topk_weights=w)
    with torch.no_grad():
        assert torch.equal(w, moe.ep_gate(cfg, b)[1])
    wa.backward(gw)
    wb.backward(gw)
    assert torch.equal(a.grad, want[0]) and torch.equal(b.grad, want[1])
    for kw in (dict(topk_idx=idx), dict(topk_weights=w)):
        a.grad = None
        moe.ep_gate(cfg, a, **kw)[1].backward(gw)
        assert torch.equal(a.grad, want[0])


def test_gate_gradient_refusals():
    cfg = moe.GateConfig(8, 2)
    lg = torch.randn((3, 8), device="cuda", requires_grad=True)
    _, w = moe.ep_gate(cfg, lg)
    with pytest.raises(RuntimeError, match="first order"):
        torch.autograd.grad(w[:, 0].sum(), lg, create_graph=True)
    idx, w = moe.ep_gate(cfg, lg)
    idx.zero_()                                     # the choice was overwritten
    with pytest.raises(RuntimeError, match="inplace"):
        w.sum().backward()
    with pytest.MonkeyPatch.context() as mp:        # as inside a capture
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        _, w = moe.ep_gate(cfg, lg)
        with pytest.raises(RuntimeError, match="captured"):
            w.sum().backward()
        z = lg * 2                                  # not a leaf
        moe.ep_gate(cfg, z)[1][:, 0].sum().backward()
    assert lg.grad is not None
    empty = torch.zeros((0, 8), device="cuda", requires_grad=True)
    moe.ep_gate(cfg, empty)[1].sum().backward()
    assert empty.grad.shape == (0, 8)


def test_gate_graph_replays():
    """A captured choice and gradient against the eager ones."""
    cfg = moe.GateConfig(64, 6, moe.EP_SCORE_SIGMOID, num_groups=8, topk_groups=3, group_top=2)
    lg, gw = torch.randn((50, 64), device="cuda"), torch.randn((50, 6), device="cuda")
    out = [torch.empty((50, 6), dtype=torch.int32, device="cuda"), torch.empty((50, 6), device="cuda"), torch.empty_like(lg)]

    def step():
        moe.ep_gate(cfg, lg, topk_idx=out[0], topk_weights=out[1])
        moe.ep_gate_backward(cfg, lg, out[0], gw, out[2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        lg.normal_()
        gw.normal_()
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        idx, w = moe.ep_gate(cfg, lg)
        assert torch.equal(out[0], idx) and torch.equal(out[1], w)
        assert torch.equal(out[2], moe.ep_gate_backward(cfg, lg, idx, gw))


# ---- router: gradients, each element to its own bound ------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K,shift", [(1, 256, 8, 0), (33, 7, 3, 0), (70, 128, 8, 0), (70, 128, 8, 1), (5, 1024, 16, 0),
                                         (6, 300, 2, 0), (9, 64, 16, 0), (9, 513, 5, 0), (6, 1, 1, 0), (130, 260, 8, 2)])
def test_gate_backward_to_each_elements_bound(N, E, K, shift, dtype, renorm, score):
    """shift: elements by which the output stands off the vectors' alignment."""
    say(f"[gate grad] {N} {E} {K} {shift} {dtype} {renorm} {score}")
    z, idx, g = grad_case(N, E, K)
    lg = torch.from_numpy(z).to(dtype)
    cfg = moe.GateConfig(E, K, dict(softmax=0, sigmoid=1)[score], renorm, scale=2.5)
    out = torch.full((N * E + shift + 1,), 77.0, dtype=dtype, device="cuda")
    got = moe.ep_gate_backward(cfg, lg.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(g).cuda(),
                               out[shift:-1].view(N, E))
    want, tol = R.gate_grad_bound(lg.float().numpy(), idx, g, score, renorm, 2.5,
                                  R.BF16_HALF if dtype == torch.bfloat16 else R.F32_HALF)
    bad = ~(np.abs(got.double().cpu().numpy() - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got.cpu().numpy()[bad][:4] if dtype ==
                           torch.float32 else None, want[bad][:4], tol[bad][:4])
    assert (out[:shift] == 77).all() and out[-1] == 77


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [0, 8])
def test_gate_infinite_and_huge_biases(groups, score):
    """Biases of +infinity (chosen first, by id), near the largest float (sums of
    a group past fp32) and of both signs: the choice's order is the definition's,
    the weights know none of it."""
    rng = np.random.default_rng(7)
    E, K = 64, 6
    lg = rng.standard_normal((30, E)).astype(np.float32)
    kw = dict(num_groups=groups, topk_groups=3, group_top=2) if groups else {}
    rkw = dict(groups=groups, topk_groups=3, group_top=2) if groups else {}
    for special in ({5: np.inf}, {3: np.inf, 4: np.inf, 40: np.inf, 41: np.inf}, {8: 3.4e38, 9: 3.4e38, 50: 3.4e38},
                    {i: -3.4e38 for i in range(E)}, {20: np.inf, 21: -np.inf, 22: -3.4e38, 23: np.nan}):
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        for e, v in special.items():
            bias[e] = v
        cfg = moe.GateConfig(E, K, dict(softmax=0, sigmoid=1)[score], **kw)
        idx, w = moe.ep_gate(cfg, torch.from_numpy(lg).cuda(), torch.from_numpy(bias).cuda())
        ridx, rw = R.gate(lg, K, score, bias=bias, **rkw)
        assert np.array_equal(idx.cpu().numpy(), ridx), special
        assert np.allclose(w.cpu().numpy(), rw, rtol=2 * R.F32_HALF, atol=1e-44)
