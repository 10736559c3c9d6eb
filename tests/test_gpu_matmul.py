"""GPU tests of the products in 8-bit integers against their definition: exact
sums, then (sum * row scale) * output scale in fp32 and one rounding to bf16."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu

U, BF16_HALF = 2.0 ** -24, 2.0 ** -8


def say(*a):
    print(*a, flush=True)


def codes(rng, *shape):
    return rng.integers(-128, 128, shape, dtype=np.int64).astype(np.int8)


def stack(rng, E, M, C):
    """Codes and scales, and the package's weights."""
    w, s = codes(rng, E, M, C), (rng.random((E, M)) + 0.5).astype(np.float32) * np.float32(C ** -0.5 / 64)
    s[rng.random(s.shape) < 0.1] *= -1
    return w, s, moe.Weights(moe.EP_WEIGHT_INT8, torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda())


def rows_of(rng, n, C):
    return codes(rng, n, C), (rng.random(n).astype(np.float32) + np.float32(0.01)) / 64


def sums(x, w):
    """Exact: float64 holds every sum."""
    return x.astype(np.float64) @ w.astype(np.float64).T


def plain(x, xs, w, ws):
    """What is stored without an activation, bit for bit: sum, both products and
    the result are each rounded to nearest."""
    y = sums(x, w).astype(np.float32) * xs[:, None] * ws[None, :]
    return torch.from_numpy(y).to(torch.bfloat16)


def gated(x, xs, w, ws):
    """(float64, bound): gate and up are each off by 3 u, a silu by at most 1.1
    of its argument's error, the exponential and the division are good to 2^-18
    for |gate| < 40, then one rounding."""
    a = sums(x, w) * xs[:, None].astype(np.float64) * ws[None, :].astype(np.float64)
    n = a.shape[1] // 2
    g, u = a[:, :n], a[:, n:]
    assert np.abs(g).max(initial=0) < 40
    out = g / (1 + np.exp(-g)) * u
    err = 1.1 * 3 * U * np.abs(g * u) + 3 * U * np.abs(out) + 2.0 ** -18 * np.abs(out)
    return out, err + BF16_HALF * (np.abs(out) + err) + 1e-38


def check(y, x, xs, w, ws, act):
    y = y.cpu()
    if not act:
        want = plain(x, xs, w, ws)
        bad = y != want
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4], want[bad][:4])
        return
    want, tol = gated(x, xs, w, ws)
    got = y.double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def dense(n, C, M, seed=0, acts=(0, 1)):
    rng = np.random.default_rng(seed + n + C + M)
    w, ws, W = stack(rng, 1, M, C)
    x, xs = rows_of(rng, n, C)
    for act in acts:
        if act and M % 2:
            continue
        y = torch.full((n + 1, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_matmul(W, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), y[:n], activation=act)
        check(y[:n], x, xs, w[0], ws[0], act)
        assert (y[n:] == 77).all()


ROWS = [1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513]


@pytest.mark.parametrize("n", ROWS)
def test_rows(n):
    """Every number of rows around the tiles' heights, odd outputs and columns."""
    say(f"[matmul rows] {n}")
    dense(n, 272, 70)
    dense(n, 128, 33)
    dense(n, 1040, 258)


@pytest.mark.parametrize("n", [3, 40, 140, 300])
@pytest.mark.parametrize("C", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 256, 272, 384, 512, 528, 656, 1024, 4112])
def test_columns(n, C):
    """Columns that end inside a step, one step and fewer, many."""
    say(f"[matmul columns] {n} {C}")
    dense(n, C, 50)
    dense(n, C, 260, acts=(n // 100 % 2,))


@pytest.mark.parametrize("n", [1, 20, 130, 280])
@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 30, 31, 32, 34, 63, 64, 66, 126, 127, 128, 130, 254, 255, 256, 258,
                               510, 514, 1026])
def test_outputs(n, M):
    say(f"[matmul outputs] {n} {M}")
    dense(n, 144, M)


@pytest.mark.parametrize("n,C,M", [(1, 7168, 4096), (5, 2048, 1536), (600, 2048, 1536), (1000, 1024, 2050),
                                   (2100, 512, 1300)])
def test_larger(n, C, M):
    say(f"[matmul larger] {n} {C} {M}")
    dense(n, C, M)


@pytest.mark.parametrize("n", [2, 18, 70, 260])
def test_sums_at_their_limits(n):
    """The longest rows of the largest codes: sums at both ends of 32 bits."""
    say(f"[matmul limits] {n}")
    C, M = (1 << 17) - 16, 20
    x, w = np.full((n, C), -128, np.int8), np.full((1, M, C), -128, np.int8)
    x[1::2], w[0, 1::2] = 127, 127
    xs, ws = np.full(n, 2.0 ** -12, np.float32), np.full((1, M), 2.0 ** -10, np.float32)
    W = moe.Weights(moe.EP_WEIGHT_INT8, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    y = moe.ep_matmul(W, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda())
    check(y, x, xs, w[0], ws[0], 0)


@pytest.mark.parametrize("n", [3, 150])
def test_scales_of_any_kind(n):
    """Zero, infinite and NaN scales stay with their rows and outputs."""
    rng = np.random.default_rng(n)
    w, ws, _ = stack(rng, 1, 40, 64)
    x, xs = rows_of(rng, n, 64)
    xs[0], ws[0, 3], ws[0, 5], ws[0, 7] = 0, np.inf, np.nan, 0
    xs[2] = np.inf
    W = moe.Weights(moe.EP_WEIGHT_INT8, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    y = moe.ep_matmul(W, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()).cpu()
    with np.errstate(invalid="ignore"):
        want = plain(x, xs, w[0], ws[0])
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, 0), torch.nan_to_num(want, 0))


def test_no_rows_and_two_dimensional_scales():
    rng = np.random.default_rng(0)
    w, ws, W = stack(rng, 1, 24, 64)
    one = moe.Weights(moe.EP_WEIGHT_INT8, torch.from_numpy(w[0]).cuda(), torch.from_numpy(ws[0]).cuda())
    x, xs = rows_of(rng, 9, 64)
    xc, sc = torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()
    assert moe.ep_matmul(W, xc[:0], sc[:0]).shape == (0, 24)
    want = moe.ep_matmul(W, xc, sc)
    assert torch.equal(moe.ep_matmul(one, xc, sc[:, None]), want)
    check(want, x, xs, w[0], ws[0], 0)


@pytest.mark.parametrize("n", [5, 300])
def test_stores_stay_inside(n):
    """y that is off every vector's alignment, guards before and behind."""
    rng = np.random.default_rng(n)
    for M, shift in ((64, 1), (66, 2), (33, 3), (256, 7), (512, 4)):
        w, ws, W = stack(rng, 1, M, 80)
        x, xs = rows_of(rng, n, 80)
        for act in (0, 1) if M % 2 == 0 else (0,):
            out = M // 2 if act else M
            buf = torch.full((n * out + shift + 9,), 77.0, dtype=torch.bfloat16, device="cuda")
            y = buf[shift:shift + n * out].view(n, out)
            moe.ep_matmul(W, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), y, activation=act)
            check(y, x, xs, w[0], ws[0], act)
            assert (buf[:shift] == 77).all() and (buf[shift + n * out:] == 77).all()


# ---- received rows -------------------------------------------------------------------

def routed(N, E, K, mask, seed, skew):
    rng = np.random.default_rng(seed)
    p = rng.random((N, E)) + (np.linspace(1.5, 0, E) if skew else 0)
    idx = np.argsort(-p, axis=1)[:, :K].astype(np.int32)
    idx[rng.random(idx.shape) < mask] = -1
    return idx


def segments(cfg, idx):
    """A handle with its layout, and each expert's first row and rows."""
    h = ep.ep_handle_init(cfg, idx.shape[0])
    ep.ep_get_layout(h, torch.from_numpy(idx).cuda())
    ep.ep_check_error(h)                   # a full segment's flag
    v = ep.ep_handle_view(h)
    first, count = v["psum_expert"].cpu().numpy(), v["num_unaligned"].cpu().numpy()
    return h, first, np.minimum(count, cfg.expert_capacity) if cfg.expert_capacity else count


CASES = [
    (1, 16, 2, 1, 0, 0.0, 1, False),
    (40, 8, 3, 1, 0, 0.1, 1, False),
    (40, 8, 3, 16, 0, 0.1, 1, True),
    (30, 33, 4, 1, 9, 0.0, 1, True),       # fixed capacity, some pairs dropped
    (24, 16, 2, 5, 0, 0.3, 4, False),      # stacked sources
    (300, 4, 2, 1, 0, 0.0, 1, False),      # many rows an expert
    (500, 6, 2, 1, 0, 0.1, 1, True),       # from none to hundreds
    (700, 3, 2, 128, 0, 0.2, 1, True),
    (900, 40, 3, 1, 50, 0.0, 1, True),
    (400, 1, 1, 1, 0, 0.0, 1, False),
    (260, 1024, 2, 1, 0, 0.0, 1, False),
    (2000, 600, 4, 3, 0, 0.05, 1, True),
]


@pytest.mark.parametrize("N,E,K,align,cap,mask,sources,skew", CASES)
@pytest.mark.parametrize("M,C", [(50, 256), (290, 144), (130, 656)])
def test_expert_matmul(M, C, N, E, K, align, cap, mask, sources, skew):
    say(f"[expert matmul] {N} {E} {K} {align} {cap} {M} {C}")
    cfg = ep.Config(hidden=C, num_topk=K, num_experts=E, num_ranks=1, expert_alignment=align, expert_capacity=cap,
                    num_sources=sources)
    h, first, count = segments(cfg, routed(N, E, K, mask, N, skew))
    rows = ep.ep_recv_capacity(cfg, N)
    rng = np.random.default_rng(E + M)
    w, ws, W = stack(rng, E, M, C)
    x, xs = rows_of(rng, rows, C)
    live = np.zeros(rows, bool)
    for e in range(E):
        live[first[e]:first[e] + count[e]] = True
    xs[~live] = np.nan                     # padding rows' scales are not used
    xc, sc = torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()
    for act in (moe.EP_ACT_NONE, moe.EP_ACT_SWIGLU):
        y = torch.full((rows, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_expert_matmul(h, W, xc, sc, y, activation=act)
        assert ep.ep_check_error(h) == (ep.EP_OK, 0)
        assert (y[torch.from_numpy(~live).cuda()] == 77).all()
        got = y.cpu()
        for e in range(E):
            s = slice(first[e], first[e] + count[e])
            if count[e]:
                check(got[s], x[s], xs[s], w[e], ws[e], act)


@pytest.mark.parametrize("N,have", [(20, 23), (600, 700), (600, 0), (600, 1)])
def test_short_buffer_is_flagged(N, have):
    cfg = ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=1)
    h, first, count = segments(cfg, routed(N, 4, 2, 0.0, 1, False))
    rng = np.random.default_rng(N)
    w, ws, W = stack(rng, 4, 24, 64)
    x, xs = rows_of(rng, 2 * N, 64)
    y = torch.full((2 * N, 24), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_expert_matmul(h, W, torch.from_numpy(x[:have]).cuda(), torch.from_numpy(xs[:have]).cuda(), y[:have])
    st, flags = ep.ep_check_error(h)
    assert st == ep.EP_ERR_CAPACITY and flags == ep.EP_FLAG_RECV_CAPACITY
    for e in range(4):
        s = slice(first[e], max(first[e], min(first[e] + count[e], have)))
        if s.stop > s.start:
            check(y[s], x[s], xs[s], w[e], ws[e], 0)
    assert (y[have:] == 77).all()


def test_states():
    rng = np.random.default_rng(0)
    _, _, W = stack(rng, 4, 24, 64)
    x, xs = (torch.from_numpy(t).cuda() for t in rows_of(rng, 8, 64))
    h = ep.ep_handle_init(ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=1), 4)
    hn = ep.ep_handle_init(ep.Config(hidden=64, num_topk=2, num_experts=4, num_ranks=2, non_expand=True), 4)
    ep.ep_get_layout(hn, torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
    h5 = ep.ep_handle_init(ep.Config(hidden=64, num_topk=2, num_experts=5, num_ranks=1), 4)
    for handle, status in ((h, ep.EP_ERR_STATE), (hn, ep.EP_ERR_INVALID_ARG), (h5, ep.EP_ERR_INVALID_ARG)):
        with pytest.raises(ep.EpError) as ei:
            moe.ep_expert_matmul(handle, W, x, xs)
        assert ei.value.status == status
    ep.ep_get_layout(h, torch.full((4, 2), -1, dtype=torch.int32, device="cuda"))   # nothing to do
    y = torch.full((8, 24), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_expert_matmul(h, W, x, xs, y)
    assert (y == 77).all() and ep.ep_check_error(h) == (ep.EP_OK, 0)


# ---- as it is used -------------------------------------------------------------------

def quantised_layer(cfg, cfg2, h, up, down, x, idx, wts, recv, scales, bufs, out):
    """Dispatch in int8, both projections in int8, combine."""
    ep.ep_get_layout(h, idx, alloc_outputs=False)
    ep.ep_dispatch(h, x, recv, scales)
    moe.ep_expert_matmul(h, up, recv, scales, bufs["a"], activation=moe.EP_ACT_SWIGLU)
    ep.ep_quantize_rows(cfg2, bufs["a"], bufs["q"], bufs["s"])
    moe.ep_expert_matmul(h, down, bufs["q"], bufs["s"], bufs["y"])
    ep.ep_combine(h, bufs["y"], wts, out)


@pytest.mark.parametrize("N,E,K,H,I", [(5, 8, 2, 256, 128), (300, 8, 3, 512, 256), (1200, 4, 2, 256, 384)])
def test_layer_in_int8(N, E, K, H, I):
    """The run of calls eagerly and as a graph, each step against its own
    definition on the inputs that the step before left."""
    say(f"[int8 layer] {N} {E} {K} {H} {I}")
    cfg = ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1, quant=ep.EP_QUANT_INT8, quant_group=H)
    cfg2 = ep.Config(hidden=I, num_topk=K, num_experts=E, num_ranks=1, combine_quant=ep.EP_QUANT_INT8, combine_group=I)
    rng = np.random.default_rng(N)
    (wu, su, up), (wd, sd, down) = stack(rng, E, 2 * I, H), stack(rng, E, H, I)
    h = ep.ep_handle_init(cfg, N)
    S = N * K
    cuda = dict(device="cuda")
    x = torch.empty((N, H), dtype=torch.bfloat16, **cuda)
    idx, wts = torch.empty((N, K), dtype=torch.int32, **cuda), torch.empty((N, K), **cuda)
    recv, scales = torch.empty((S, H), dtype=torch.int8, **cuda), torch.empty((S, 1), **cuda)
    bufs = dict(a=torch.empty((S, I), dtype=torch.bfloat16, **cuda), q=torch.empty((S, I), dtype=torch.int8, **cuda),
                s=torch.empty((S, 1), **cuda), y=torch.empty((S, H), dtype=torch.bfloat16, **cuda))
    out = torch.empty((N, H), dtype=torch.bfloat16, **cuda)
    args = (cfg, cfg2, h, up, down, x, idx, wts, recv, scales, bufs, out)

    def fresh(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.normal_(generator=g)
        wts.uniform_(generator=g)
        idx.copy_(torch.rand((N, E), generator=g, **cuda).topk(K, dim=1).indices)

    def verify():
        torch.cuda.synchronize()
        v = ep.ep_handle_view(h)
        first, slot = v["psum_expert"].cpu().numpy(), v["slot_idx"].cpu().numpy()
        r, rs, q, qs = (t.cpu().numpy() for t in (recv, scales, bufs["q"], bufs["s"]))
        assert np.array_equal(slot.reshape(-1)[np.argsort(idx.cpu().numpy().reshape(-1), kind="stable")], np.arange(S))
        for e in range(E):
            s = slice(first[e], first[e + 1])
            if s.stop > s.start:
                check(bufs["a"][s], r[s], rs[s, 0], wu[e], su[e], 1)
                check(bufs["y"][s], q[s], qs[s, 0], wd[e], sd[e], 0)
        y, w = bufs["y"].double().cpu().numpy(), wts.double().cpu().numpy()
        want = (y[slot.reshape(-1)].reshape(N, K, H) * w[..., None]).sum(1)
        tol = BF16_HALF * np.abs(want) + (K + 1) * 2 * U * (np.abs(y)[slot.reshape(-1)].reshape(N, K, H) * w[..., None]).sum(1)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()

    fresh(1)
    quantised_layer(*args)
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        quantised_layer(*args)
    for seed in (2, 3, 4):
        fresh(seed)
        for t in (recv, *bufs.values(), out):
            t.zero_()
        graph.replay()
        verify()
        got = out.clone()
        quantised_layer(*args)
        assert torch.equal(out, got)


@pytest.mark.parametrize("n", [4, 400])
def test_two_streams_at_once(n):
    rng = np.random.default_rng(n)
    data = []
    for C, M in ((512, 384), (1040, 770)):
        _, _, W = stack(rng, 1, M, C)
        data.append((W, *(torch.from_numpy(t).cuda() for t in rows_of(rng, n, C))))
    want = [moe.ep_matmul(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [[], []]
    for _ in range(8):
        for k, d in enumerate(data):
            with torch.cuda.stream(streams[k]):
                got[k].append(moe.ep_matmul(*d))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in range(2) for y in got[k])


def test_offsets_past_32_bits():
    """Weights, rows and outputs beyond 4 GiB."""
    g = torch.Generator(device="cuda").manual_seed(1)
    E, M, C = 1024, 2100, 2064          # 4.4 GB of weights
    W = torch.randint(-128, 128, (E, M, C), dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand((E, M), device="cuda", generator=g)
    w = moe.Weights(moe.EP_WEIGHT_INT8, W, s)
    for n in (2, 40):
        idx = torch.tensor([[0], [1023], [1022], [1023]] * n, dtype=torch.int32, device="cuda")
        h = ep.ep_handle_init(ep.Config(hidden=C, num_topk=1, num_experts=E, num_ranks=1), 4 * n)
        ep.ep_get_layout(h, idx)
        x = torch.randint(-128, 128, (4 * n, C), dtype=torch.int8, device="cuda", generator=g)
        xs = torch.rand(4 * n, device="cuda", generator=g)
        y = moe.ep_expert_matmul(h, w, x, xs)
        for e, a, b in ((0, 0, n), (1022, n, 2 * n), (1023, 2 * n, 4 * n)):
            want = (x[a:b].double() @ W[e].double().t().contiguous()).float() * xs[a:b, None] * s[e]
            assert torch.equal(y[a:b], want.to(torch.bfloat16)), (n, e)
    del W, w
    n, C, M = 300001, 16400, 64         # 4.9 GB of rows
    x = torch.empty((n, C), dtype=torch.int8, device="cuda").random_(-128, 128, generator=g)
    xs = torch.rand(n, device="cuda", generator=g)
    W = torch.randint(-128, 128, (1, M, C), dtype=torch.int8, device="cuda", generator=g)
    y = moe.ep_matmul(moe.Weights(moe.EP_WEIGHT_INT8, W, torch.ones((1, M), device="cuda")), x, xs)
    for a in (0, 261000, n - 200):
        want = (x[a:a + 200].double() @ W[0].double().t().contiguous()).float() * xs[a:a + 200, None]
        assert torch.equal(y[a:a + 200], want.to(torch.bfloat16)), a
    del x
    n, C, M = 70003, 16, 32800          # 4.6 GB of outputs
    x = torch.randint(-128, 128, (n, C), dtype=torch.int8, device="cuda", generator=g)
    W = torch.randint(-128, 128, (1, M, C), dtype=torch.int8, device="cuda", generator=g)
    y = moe.ep_matmul(moe.Weights(moe.EP_WEIGHT_INT8, W, torch.ones((1, M), device="cuda")), x, xs[:n].contiguous())
    for a in (0, 65000, n - 100):
        want = (x[a:a + 100].double() @ W[0].double().t().contiguous()).float() * xs[a:a + 100, None]
        assert torch.equal(y[a:a + 100], want.to(torch.bfloat16)), a
