"""GPU tests of the balance loss and its gradient against their plain 64-bit
definitions (balance_reference)."""
import numpy as np
import pytest
import torch

import balance_reference as B
from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu

SCORE = dict(softmax=moe.EP_SCORE_SOFTMAX, sigmoid=moe.EP_SCORE_SIGMOID)
MODES = [("softmax", True), ("sigmoid", True), ("sigmoid", False)]


def say(*a):
    print(*a, flush=True)


def cu(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype or torch.from_numpy(a).dtype)


def inputs(N, E, K, Q=0, masked=0.0, seed=0):
    """Logits, a choice with masked, foreign and repeated entries, a mask and
    ragged sequences (an empty one, tokens before the first and behind the last)."""
    rng = np.random.default_rng(seed + 7 * N + E)
    z = (rng.standard_normal((N, E)) + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K].astype(np.int32)
    idx[rng.random(idx.shape) < 0.05] = -1
    if N > 4:
        idx[3, 0], idx[3, K - 1] = E, -5
        idx[4] = idx[4, 0]
    mask = rng.random(N) >= masked if masked else None
    start = None
    if Q:
        start = np.sort(rng.integers(0, N + 1, Q + 1)).astype(np.int32)
        if Q > 2:
            start[Q // 2] = start[Q // 2 + 1]
    return z, idx, mask, start


def check(z, idx, mask=None, start=None, score="softmax", normalize=True, coefficient=0.5, dtype=torch.float32, g=1.5):
    """Loss, counts and gradient, each element to its own bound; returns them."""
    N, E = z.shape
    K = idx.shape[1]
    cfg = moe.BalanceConfig(E, K, SCORE[score], normalize, coefficient)
    lg = cu(z).to(dtype)
    zz = lg.float().cpu().numpy()
    m, s = cu(mask), cu(start)
    out = moe.ep_balance_loss(cfg, lg, cu(idx), m, s)
    loss, n, T, S, eloss, eS = B.balance(zz, idx, score, normalize, coefficient, start, mask)
    assert np.array_equal(out.counts.cpu().numpy(), n) and np.array_equal(out.seq_tokens.cpu().numpy(), T)
    assert (np.abs(out.score_sums.double().cpu().numpy() - S) <= eS).all()
    assert abs(float(out.loss) - loss) <= eloss, (float(out.loss), loss, eloss)
    grad = moe.ep_balance_loss_backward(cfg, lg, out.counts, out.seq_tokens, torch.tensor(g, device="cuda"), m, s)
    want, err = B.gradient(zz, n, T, K, score, normalize, coefficient, g, start, mask,
                           2.0 ** -8 if dtype == torch.bfloat16 else B.U)
    got = grad.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= err)
    assert grad.dtype == dtype and not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4],
                                                   want[bad][:4], err[bad][:4])
    return out, grad


@pytest.mark.parametrize("score,normalize", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K", [(1, 256, 8), (2, 1, 1), (17, 3, 2), (128, 16, 2), (33, 65, 4), (100, 64, 6),
                                   (257, 128, 8), (70, 130, 5), (129, 256, 8), (50, 260, 3), (31, 512, 8),
                                   (40, 1024, 16), (9, 1023, 16), (1500, 36, 3)])
def test_balance(N, E, K, dtype, score, normalize):
    say(f"[balance] {N} {E} {K} {dtype} {score} {normalize}")
    z, idx, mask, _ = inputs(N, E, K, masked=0.2)
    check(z, idx, None, None, score, normalize, dtype=dtype)
    check(z, idx, mask, None, score, normalize, dtype=dtype)


@pytest.mark.parametrize("score,normalize", MODES)
@pytest.mark.parametrize("N,E,K,Q,masked", [(1, 16, 2, 1, 0.0), (40, 16, 2, 5, 0.0), (300, 64, 4, 64, 0.1), (333, 100, 3, 65, 0.3),
                                            (2000, 32, 2, 7, 0.1), (130, 24, 2, 400, 0.0), (500, 1024, 8, 20, 0.5),
                                            (20000, 8, 2, 17, 0.1), (300, 256, 8, 5000, 0.0)])
def test_sequences(N, E, K, Q, masked, score, normalize):
    """Ragged sequences, empty ones, more of them than a wave or than tokens."""
    say(f"[balance sequences] {N} {E} {K} {Q} {masked} {score} {normalize}")
    z, idx, mask, start = inputs(N, E, K, Q, masked)
    check(z, idx, mask, start, score, normalize)
    check(z, idx, mask, start, score, normalize, dtype=torch.bfloat16)
    if Q > 2:       # cuts on every kind of border between chunks of tokens
        cuts = np.linspace(0, N, Q + 1).astype(np.int32)
        cuts[1:-1] = cuts[1:-1] // 16 * 16
        check(z, idx, mask, cuts, score, normalize)


@pytest.mark.parametrize("score,normalize", MODES)
def test_odd_logits(score, normalize):
    """Infinities, NaN, rows without a score, logits far apart or far from 0."""
    z, idx, _, _ = inputs(48, 40, 4)
    rng = np.random.default_rng(1)
    z[0], z[1] = -np.inf, np.nan
    z[2, 3:] = -np.inf
    z[3, ::2] = np.nan
    z[4, 7] = np.inf
    z[5, [2, 30]] = np.inf
    z[6], z[7] = 3e38, -3e38
    z[8] = rng.permutation(40) * 40 - 800
    z[9] = rng.standard_normal(40) - 90
    z[10] = rng.standard_normal(40) - 64
    z[11] = rng.standard_normal(40) - 300
    z[12] = rng.standard_normal(40) + 300
    z[13, 0], z[13, 1:] = 500, -500
    z[14] = -0.0
    say(f"[balance odd] {score} {normalize}")
    out, grad = check(z, idx, None, None, score, normalize)
    assert torch.isfinite(out.loss) and torch.isfinite(grad).all()
    assert (grad[:2] == 0).all()
    check(z, idx, None, np.array([0, 1, 2, 20, 48], np.int32), score, normalize)


def test_scores_far_from_zero():
    """A sigmoid alone, one token a sequence, so that score_sums holds it: 8 u at
    every magnitude (balance_reference: the exponential 4, the sum 1, the
    reciprocal 3), also where a rounded exponent would be off by 60."""
    z = np.linspace(-87, 87, 1000 * 40, dtype=np.float32)
    np.random.default_rng(2).shuffle(z)
    z = z.reshape(1000, 40)
    start = np.arange(1001, dtype=np.int32)
    out = moe.ep_balance_loss(moe.BalanceConfig(40, 1, moe.EP_SCORE_SIGMOID, False), cu(z),
                              cu(np.zeros((1000, 1), np.int32)), None, cu(start))
    want = 1 / (1 + np.exp(-z.astype(np.float64)))
    err = np.abs(out.score_sums.double().cpu().numpy() - want) / want
    assert err.max() <= 8 * B.U, err.max() / B.U


def test_nothing_left():
    """No token, all masked, no live entry, an expert that all take."""
    cfg = moe.BalanceConfig(24, 3, coefficient=2.0)
    for N in (0, 40):
        lg = torch.randn((N, 24), device="cuda")
        idx = torch.zeros((N, 3), dtype=torch.int32, device="cuda")
        for start in (None, torch.tensor([0, N // 2, N], dtype=torch.int32, device="cuda")):
            mask = torch.zeros(N, dtype=torch.bool, device="cuda")
            out = moe.ep_balance_loss(cfg, lg, idx, mask, start)
            assert float(out.loss) == 0 and not out.counts.any() and not out.seq_tokens.any() and not out.score_sums.any()
            grad = moe.ep_balance_loss_backward(cfg, lg, out.counts, out.seq_tokens, out.loss + 1, mask, start)
            assert grad.shape == lg.shape and not grad.any()
    out = moe.ep_balance_loss(cfg, lg, torch.full_like(idx, -1))
    assert float(out.loss) == 0 and int(out.seq_tokens) == 40
    check(np.zeros((40, 24), np.float32), np.zeros((40, 3), np.int32))
    check(np.zeros((40, 24), np.float32), np.zeros((40, 3), np.int32), coefficient=0.0)
    check(np.zeros((40, 24), np.float32), np.ones((40, 3), np.int32), coefficient=-1.0, g=-3.0)


def test_starts_outside_the_batch():
    """Held to its ends; what lies outside the buffers is not touched."""
    z, idx, _, _ = inputs(50, 20, 2)
    check(z, idx, None, np.array([-7, 10, 90, 2 ** 31 - 1], np.int32))
    cfg = moe.BalanceConfig(20, 2)
    start = torch.tensor([60, 40, -5, 30, 20, 50], dtype=torch.int32, device="cuda")   # decreasing: any value
    buf = torch.full((52, 20), 7.0, device="cuda")
    out = moe.ep_balance_loss(cfg, cu(z), cu(idx), None, start)
    moe.ep_balance_loss_backward(cfg, cu(z), out.counts, out.seq_tokens, torch.ones((), device="cuda"), None, start,
                                 buf[1:51])
    assert (buf[0] == 7).all() and (buf[51] == 7).all()


@pytest.mark.parametrize("shift", [1, 2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_rows(shift, dtype):
    """Logits and gradient off the vectors' alignment, guards around them."""
    z, idx, mask, start = inputs(70, 64, 4, 5, 0.1)
    cfg = moe.BalanceConfig(64, 4, coefficient=0.5)
    want = check(z, idx, mask, start, dtype=dtype)
    lg = torch.empty(70 * 64 + shift, dtype=dtype, device="cuda")[shift:].view(70, 64)
    lg.copy_(cu(z))
    out = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
    for a, b in zip(out, want[0]):
        assert torch.equal(a, b)
    buf = torch.full((70 * 64 + shift + 1,), 7.0, dtype=dtype, device="cuda")
    got = moe.ep_balance_loss_backward(cfg, lg, out.counts, out.seq_tokens, torch.tensor(1.5, device="cuda"), cu(mask),
                                       cu(start), buf[shift:-1].view(70, 64))
    assert torch.equal(got, want[1]) and (buf[:shift] == 7).all() and buf[-1] == 7


def test_large_batch():
    """Chunks of many tokens, as many pieces as a batch makes, and long ones."""
    rng = np.random.default_rng(3)
    z = rng.standard_normal((70001, 16)).astype(np.float32)
    idx = np.argsort(-z, axis=1)[:, :2].astype(np.int32)
    check(z, idx)
    check(z, idx, rng.random(70001) < 0.9, np.array([5, 30000, 30001, 69999], np.int32), "sigmoid")
    z = np.repeat(z[:1024], 1100, axis=0)          # over a million tokens: chunks of 1024
    idx = np.repeat(idx[:1024], 1100, axis=0)
    check(z, idx)


@pytest.mark.parametrize("N,E,real,padded", [(300, 24, 6, 3000), (2000, 64, 37, 5000), (1100, 256, 9, 1100)])
def test_padded_sequences(N, E, real, padded):
    """Many empty sequences in one place: behind the last, before the first,
    between two, with tokens of no sequence beside them."""
    say(f"[balance padded] {N} {E} {real} {padded}")
    z, idx, mask, _ = inputs(N, E, 4, masked=0.1)
    some = np.sort(np.random.default_rng(5).integers(N // 10, N - N // 10, real + 1)).astype(np.int32)
    for k in (real, 0, real // 2):
        start = np.insert(some, k, np.full(padded, some[k]))
        check(z, idx, mask, start)
        check(z, idx, None, start, "sigmoid", False, dtype=torch.bfloat16)


def test_long_sequences_by_the_thousand():
    """Sequences of several pieces each, more of them than the second kernel's
    blocks hold at a time.  The relative error of a sum of scores is below 128 u:
    |a| <= 16 and 32 of a score, 64 + 6 of the sums (balance_reference); the
    second kernel's are in 64 bits, its result is rounded once."""
    N, E, Q = 15_000_000, 4, 2049
    say(f"[balance long] {N} {E} {Q}")
    gen = torch.Generator("cuda").manual_seed(3)
    lg = torch.randn((N, E), device="cuda", generator=gen)
    idx = lg.argmax(1, keepdim=True).int()
    start = torch.linspace(0, N, Q + 1, dtype=torch.float64).round().int().cuda()
    out = moe.ep_balance_loss(moe.BalanceConfig(E, 1, coefficient=0.5), lg, idx, None, start)
    lens = start.diff().long()
    p = torch.softmax(lg.double(), 1)
    of = torch.repeat_interleave(torch.arange(Q, device="cuda"), lens)
    S = torch.zeros((Q, E), dtype=torch.float64, device="cuda").index_add_(0, of, p)
    n = torch.bincount(of * E + idx[:, 0], minlength=Q * E).view(Q, E)
    assert torch.equal(out.counts.long(), n) and torch.equal(out.seq_tokens.long(), lens)
    assert ((out.score_sums.double() - S).abs() <= 129 * B.U * S).all()
    loss = 0.5 / Q * (E / lens.double() ** 2 * (n * S).sum(1)).sum()
    assert abs(float(out.loss) - float(loss)) <= 129 * B.U * float(loss)


def test_counts_of_all_ranks():
    """The gradient takes counts and tokens summed over ranks."""
    z, idx, _, _ = inputs(64, 32, 4)
    cfg = moe.BalanceConfig(32, 4)
    n, T = 5 * B.counts(idx, 32) + 3, np.array([1000])
    got = moe.ep_balance_loss_backward(cfg, cu(z), cu(n.astype(np.int32)), cu(T.astype(np.int32)),
                                       torch.ones((), device="cuda"))
    want, err = B.gradient(z, n, T, 4)
    assert (np.abs(got.double().cpu().numpy() - want) <= err).all()


def test_given_outputs_and_repeats():
    """Buffers of the caller, a workspace full of anything, the same bits again."""
    z, idx, mask, start = inputs(3000, 256, 8, 9, 0.1)
    cfg = moe.BalanceConfig(256, 8, coefficient=0.1)
    lg, i, m, s = cu(z), cu(idx), cu(mask), cu(start)
    want = moe.ep_balance_loss(cfg, lg, i, m, s)
    outs = dict(loss=torch.empty((), device="cuda"), counts=torch.empty((9, 256), dtype=torch.int32, device="cuda"),
                seq_tokens=torch.empty(9, dtype=torch.int32, device="cuda"), score_sums=torch.empty((9, 256), device="cuda"))
    ws = torch.empty(moe.ep_balance_workspace_size(cfg, 3000, 9), dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 113):
        ws.fill_(fill)
        got = moe.ep_balance_loss(cfg, lg, i, m.to(torch.uint8), s, workspace=ws, **outs)
        for a, b, o in zip(got, want, outs.values()):
            assert torch.equal(a, b) and a.data_ptr() == o.data_ptr()
    with pytest.raises(ep.EpError):
        moe.ep_balance_loss(cfg, lg, i, m, s, workspace=ws[:-256])


# ---- autograd, graphs, streams ------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_autograd(dtype):
    """The loss's gradient, alone and beside the router's weights'."""
    z, idx, mask, start = inputs(200, 64, 6, 4, 0.1)
    cfg = moe.BalanceConfig(64, 6, coefficient=0.3)
    want = check(z, idx, mask, start, coefficient=0.3, g=2.0, dtype=dtype)[1]
    lg = cu(z).to(dtype).requires_grad_()
    out = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
    assert out.loss.requires_grad and not out.score_sums.requires_grad and not out.counts.requires_grad
    (2 * out.loss).backward()
    assert torch.equal(lg.grad, want) and lg.grad.dtype == dtype
    with torch.no_grad():
        assert not moe.ep_balance_loss(cfg, lg, cu(idx)).loss.requires_grad

    # a training step of the router: choice, weights, balance loss, one backward pass
    gate = moe.GateConfig(64, 6)
    x = torch.randn((200, 32), device="cuda")
    w = torch.randn((64, 32), device="cuda", requires_grad=True)
    logits = x @ w.t()
    i, wts = moe.ep_gate(gate, logits)
    c = torch.randn_like(wts)
    loss = moe.ep_balance_loss(cfg, logits, i, None, cu(start)).loss
    ((wts * c).sum() + loss).backward()
    with torch.no_grad():
        b = moe.ep_balance_loss(cfg, logits, i, None, cu(start))
        one = torch.ones((), device="cuda")
        g = moe.ep_gate_backward(gate, logits, i, c) + \
            moe.ep_balance_loss_backward(cfg, logits, b.counts, b.seq_tokens, one, None, cu(start))
        torch.testing.assert_close(w.grad, g.t() @ x, rtol=1e-5, atol=1e-5)


def test_autograd_buffers_and_refusals():
    cfg = moe.BalanceConfig(16, 2)
    a, b = (torch.randn((30, 16), device="cuda", requires_grad=True) for _ in range(2))
    idx = torch.randint(0, 16, (30, 2), dtype=torch.int32, device="cuda")
    bufs = dict(loss=torch.zeros((), device="cuda"), counts=torch.zeros((1, 16), dtype=torch.int32, device="cuda"),
                seq_tokens=torch.zeros(1, dtype=torch.int32, device="cuda"), score_sums=torch.zeros((1, 16), device="cuda"))
    want = []
    for t in (a, b):
        with torch.no_grad():
            o = moe.ep_balance_loss(cfg, t, idx)
            want.append(moe.ep_balance_loss_backward(cfg, t, o.counts, o.seq_tokens, torch.ones((), device="cuda")))
    la = moe.ep_balance_loss(cfg, a, idx, **bufs).loss
    lb = moe.ep_balance_loss(cfg, b, (idx + 1) % 16, **bufs).loss       # fills the buffers again
    assert la.requires_grad and not bufs["loss"].requires_grad and la.data_ptr() == bufs["loss"].data_ptr()
    la.backward()
    lb.backward()
    assert torch.equal(a.grad, want[0])
    loss = moe.ep_balance_loss(cfg, a, idx).loss
    with pytest.raises(RuntimeError, match="first order"):
        torch.autograd.grad(loss, a, create_graph=True)
    with pytest.MonkeyPatch.context() as mp:        # as inside a capture
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="captured"):
            moe.ep_balance_loss(cfg, a, idx).loss.backward()
        moe.ep_balance_loss(cfg, a * 2, idx).loss.backward()            # not a leaf
    empty = torch.zeros((0, 16), device="cuda", requires_grad=True)
    moe.ep_balance_loss(cfg, empty, idx[:0]).loss.backward()
    assert empty.grad.shape == (0, 16)


def test_graph_replays():
    """Both directions captured, each replay against the eager calls."""
    N, E, K, Q = 700, 64, 4, 3
    cfg = moe.BalanceConfig(E, K, moe.EP_SCORE_SIGMOID)
    lg, g = torch.randn((N, E), device="cuda"), torch.ones((), device="cuda")
    idx = torch.randint(-1, E, (N, K), dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 100, 400, 690], dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.ep_balance_workspace_size(cfg, N, Q), dtype=torch.uint8, device="cuda")
    outs = dict(loss=torch.empty((), device="cuda"), counts=torch.empty((Q, E), dtype=torch.int32, device="cuda"),
                seq_tokens=torch.empty(Q, dtype=torch.int32, device="cuda"), score_sums=torch.empty((Q, E), device="cuda"))
    grad = torch.empty_like(lg)

    def step():
        moe.ep_balance_loss(cfg, lg, idx, None, start, workspace=ws, **outs)
        moe.ep_balance_loss_backward(cfg, lg, outs["counts"], outs["seq_tokens"], g, None, start, grad)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        lg.normal_()
        idx.random_(-1, E)
        start[1:3] += 7
        for t in (*outs.values(), grad):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        want = moe.ep_balance_loss(cfg, lg, idx, None, start)
        for a, b in zip(outs.values(), want):
            assert torch.equal(a, b), i
        assert torch.equal(grad, moe.ep_balance_loss_backward(cfg, lg, want.counts, want.seq_tokens, g, None, start))


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    cfg = moe.BalanceConfig(256, 8)
    data = [inputs(20000, 256, 8, q, 0.1, seed=q) for q in (0, 40)]
    data = [tuple(cu(a) for a in d) for d in data]
    want = [moe.ep_balance_loss(cfg, z, i, m, s) for z, i, m, s in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(6):
        for k, (z, i, m, s) in enumerate(data):
            with torch.cuda.stream(streams[k]):
                got[k].append(moe.ep_balance_loss(cfg, z, i, m, s))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            for a, b in zip(out, want[k]):
                assert torch.equal(a, b)
