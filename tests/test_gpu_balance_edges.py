"""GPU tests of the balance loss where a caller changes what it returned, and of
its gradient for tokens that are all but sure of one expert."""
import numpy as np
import pytest
import torch

import balance_reference as B
from combine_get_dispatch_layout_amd import moe
from test_gpu_balance import SCORE, cu, inputs, say

pytestmark = pytest.mark.gpu


def test_counts_summed_in_place_before_backward():
    """As an all-reduce leaves them, which raises no version: the loss's gradient
    stays that of the call."""
    z, idx, mask, start = inputs(200, 64, 6, 4, 0.1)
    cfg = moe.BalanceConfig(64, 6, coefficient=0.3)
    lg = cu(z).requires_grad_()
    with torch.no_grad():
        o = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
        want = moe.ep_balance_loss_backward(cfg, lg, o.counts, o.seq_tokens, torch.ones((), device="cuda"), cu(mask),
                                            cu(start))
    out = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
    assert torch.equal(out.counts, o.counts) and torch.equal(out.seq_tokens, o.seq_tokens)
    out.counts.data.mul_(8)
    out.seq_tokens.data.mul_(8)
    out.score_sums.data.mul_(8)
    out.loss.backward()
    assert torch.equal(lg.grad, want)


def sure_gradient(z, n, T, K, score, coefficient, g):
    """The gradient as p_e sum_j p_j (f_e - f_j), times 1 - s of a sigmoid, and its
    bound where one expert, c, has most of the score.  A kernel that measures the
    counts from f_c has errors that go with the differences that are left: with d_j
    = f_j - f_c, off by u, dot = sum_j p_j d_j is off by (rel_j + 25) u of each term,
    f_e - f_c - dot by u of d_e and of dot more; the rest as in balance_reference.
    No term goes with |f| itself."""
    p, rest, rel = B.scores(z, score, True)
    N, E = z.shape
    scale = g * coefficient * E / (K * float(T) ** 2)
    f = n.astype(np.float64)
    d = f[None, :] - f[z.argmax(1)][:, None]
    dot = (p * d).sum(1, keepdims=True)
    edot = (p * np.abs(d) * (rel + 25) * B.U).sum(1, keepdims=True)
    w = p * (rest if score == "sigmoid" else 1.0) * abs(scale)
    out = np.sign(scale) * w * (d - dot)
    err = w * (edot + 2 * B.U * (np.abs(d) + np.abs(dot))) + np.abs(out) * (rel + 17) * B.U
    return out, err + B.U * (np.abs(out) + err) + B.TINY


@pytest.mark.parametrize("E", [8, 40, 64, 130, 256, 300, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sure_tokens(score, E):
    """One logit 8 to 40 above the others: the gradient of its expert is what the
    others' small scores make, to their own relative bound, sign included."""
    say(f"[balance sure] {score} {E}")
    K, N = min(E, 4), 90
    rng = np.random.default_rng(E)
    z = rng.standard_normal((N, E)).astype(np.float32) * np.float32(0.5)
    top = rng.integers(0, E, N)
    gap = np.linspace(8, 40, N).astype(np.float32)
    z[np.arange(N), top] = 3 + z[np.arange(N), top]
    z -= np.where(np.arange(E)[None] == top[:, None], 0, gap[:, None]).astype(np.float32)
    n = rng.integers(0, 300000, E)
    n[:2] = 0, 250000
    T = np.array([40000])
    cfg = moe.BalanceConfig(E, K, SCORE[score], True, 0.5)
    got = moe.ep_balance_loss_backward(cfg, cu(z), cu(n[None].astype(np.int32)), cu(T.astype(np.int32)),
                                       torch.tensor(1.5, device="cuda")).double().cpu().numpy()
    want, err = sure_gradient(z, n, T[0], K, score, 0.5, 1.5)
    p, _, _ = B.scores(z, score, True)
    sure = p.max(1) > 0.75
    assert sure.sum() > 60
    bad = ~(np.abs(got - want) <= err)[sure]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[sure][bad][:4], want[sure][bad][:4],
                           err[sure][bad][:4])
    r = np.arange(N)
    assert np.median((err / np.maximum(np.abs(want), 1e-300))[r, top]) < 2.0 ** -15      # the bound tells


def test_captured_step_through_autograd():
    """Loss and gradient of logits that are no leaf in one graph, each replay against
    the eager calls, with eager work between."""
    N, E, K, Q = 600, 64, 4, 3
    cfg = moe.BalanceConfig(E, K)
    w = torch.randn((N, E), device="cuda", requires_grad=True)
    idx = torch.randint(-1, E, (N, K), dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 100, 400, 590], dtype=torch.int32, device="cuda")

    def step():
        lg = w * 2
        out = moe.ep_balance_loss(cfg, lg, idx, None, start)
        return out.loss.detach(), out.counts, torch.autograd.grad(out.loss, lg)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(5):
        with torch.no_grad():
            w.normal_()
        idx.random_(-1, E)
        start[1:3] += 5
        for t in got:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i
