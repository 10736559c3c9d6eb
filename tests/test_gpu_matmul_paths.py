"""GPU tests of each kernel of the products in 8-bit integers, at sizes that
reach it (asserted), against sums in 64 bits on the same device: without an
activation bit for bit, with the gate to the bound of test_gpu_matmul."""
import pytest
import torch

import matmul_paths as P
from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu

U, BF16_HALF = 2.0 ** -24, 2.0 ** -8


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def stack(g, E, M, C):
    w = torch.randint(-128, 128, (E, M, C), dtype=torch.int8, device="cuda", generator=g)
    s = (torch.rand((E, M), device="cuda", generator=g) + 0.5) * (C ** -0.5 / 64)
    return w, s, moe.Weights(moe.EP_WEIGHT_INT8, w, s)


def rows_of(g, n, C):
    return torch.randint(-128, 128, (n, C), dtype=torch.int8, device="cuda", generator=g), \
        (torch.rand(n, device="cuda", generator=g) + 0.01) / 64


def check(y, x, xs, w, s, act):
    sums = torch.mm(x.double(), w.double().t().contiguous())        # exact
    if not act:
        want = (sums.float() * xs[:, None] * s[None]).to(torch.bfloat16)
        bad = y != want
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4], want[bad][:4])
        return
    a = sums * xs.double()[:, None] * s.double()[None]
    n = a.shape[1] // 2
    gate, up = a[:, :n], a[:, n:]
    assert float(gate.abs().max()) < 40
    out = gate / (1 + torch.exp(-gate)) * up
    err = 1.1 * 3 * U * (gate * up).abs() + 3 * U * out.abs() + 2.0 ** -18 * out.abs()
    bad = ~((y.double() - out).abs() <= err + BF16_HALF * (out.abs() + err) + 1e-38)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4], out[bad][:4])


DENSE = [
    (P.THIN, 1, 16, 1, 0), (P.THIN, 3, 2048, 38, 0), (P.THIN, 5, 4112, 70, 0), (P.THIN, 16, 2064, 34, 1),
    (P.THIN, 17, 400, 34, 1), (P.THIN, 32, 2064, 514, 0), (P.THIN, 31, 7184, 4098, 0),
    (P.TILE128, 40, 256, 300, 0), (P.TILE128, 1000, 128, 66, 1), (P.TILE128, 3000, 16, 2050, 0),
    (P.TILE128, 9000, 144, 4098, 0), (P.TILE128, 9001, 112, 4100, 1), (P.TILE128, 30000, 256, 2050, 0),
    (P.TILE128, 30000, 128, 2050, 0), (P.TILE128, 30001, 48, 2062, 1), (P.TILE64X128, 700, 384, 2050, 0),
    (P.TILE64X64, 300, 512, 2050, 0),
    (P.TILE64X64, 33, 528, 130, 0), (P.TILE64X64, 65, 656, 66, 1), (P.TILE64X64, 300, 1040, 520, 0),
    (P.TILE64X64, 1, 2048, 20000, 0), (P.TILE64X64, 127, 528, 1, 0), (P.TILE64X64, 700, 2048, 2, 1),
    (P.TILE64X128, 1500, 528, 2050, 0), (P.TILE64X128, 1500, 528, 1500, 1), (P.TILE64X128, 1024, 640, 4096, 0),
    (P.TILE64X128, 900, 528, 4000, 1),
    (P.TILE64X128, 33, 272, 4000, 0), (P.TILE128, 2100, 272, 2050, 0), (P.TILE128, 2300, 384, 2062, 1),
    (P.TILE128, 3000, 528, 3002, 0), (P.TILE128, 4100, 400, 4110, 1),
    (P.TILE256, 3800, 272, 3900, 0), (P.TILE256, 3700, 272, 4000, 1), (P.TILE256, 4096, 400, 4096, 0),
    (P.TILE256, 4096, 1024, 4096, 1), (P.TILE256, 7900, 384, 3841, 0),
]


@pytest.mark.parametrize("path,n,C,M,act", DENSE)
def test_one_matrix(path, n, C, M, act):
    say(f"[matmul path] {path} {n} {C} {M} {act}")
    assert P.matmul(n, C, M, act) == path
    g = gen(n + C + M)
    w, s, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    y = torch.full((n + 1, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_matmul(W, x, xs, y[:n], activation=act)
    check(y[:n], x, xs, w[0], s[0], act)
    assert (y[n:] == 77).all()


# path, tokens, experts, entries a token, columns, weight rows, gate, alignment,
# capacity, share of masked entries, skew
RECEIVED = [
    (P.FEW, 100, 64, 3, 272, 9000, 0, 1, 0, 0.1, 1.0),
    (P.TILE128, 300, 30, 4, 128, 70, 1, 5, 0, 0.1, 1.0), (P.TILE128, 20000, 30, 4, 256, 700, 1, 5, 0, 0.1, 1.0),
    (P.TILE64X64, 3000, 200, 2, 512, 258, 0, 1, 0, 0.1, 0.5), (P.TILE64X128, 3000, 200, 2, 384, 514, 1, 1, 0, 0.1, 0.5),
    (P.TILE64X128, 3000, 200, 2, 384, 1026, 0, 1, 0, 0.1, 0.5),
    (P.TILE128, 6000, 128, 4, 128, 1026, 0, 1, 0, 0.1, 1.0), (P.TILE128, 30000, 4, 2, 256, 2000, 0, 1, 0, 0.0, 0.02),
    (P.TILE128, 30000, 4, 2, 16, 2000, 0, 1, 0, 0.0, 0.02),
    (P.FEW, 20, 8, 2, 4112, 66, 0, 1, 0, 0.1, 1.0), (P.FEW, 13, 9, 3, 7168, 514, 1, 8, 0, 0.0, 1.0),
    (P.TILE64X64, 250, 6, 2, 656, 130, 0, 1, 0, 0.1, 1.0),
    (P.TILE64X64, 90, 8, 4, 528, 258, 1, 16, 0, 0.0, 0.5),
    (P.TILE64X64, 60, 1024, 1, 656, 200, 0, 1, 0, 0.0, 0.0),
    (P.TILE64X128, 500, 40, 4, 528, 1000, 0, 1, 60, 0.05, 1.5),
    (P.TILE64X128, 750, 64, 2, 528, 700, 1, 1, 0, 0.0, 1.0),
    (P.TILE128, 1000, 40, 4, 528, 1000, 0, 128, 0, 0.1, 1.5),
    (P.TILE128, 2500, 40, 2, 272, 700, 1, 1, 150, 0.0, 1.0),
    (P.TILE128, 3000, 12, 2, 400, 1500, 0, 1, 0, 0.3, 1.5),
    (P.TILE256, 3900, 4, 2, 272, 2000, 0, 1, 0, 0.0, 0.02),
    (P.TILE256, 7700, 4, 1, 400, 2000, 1, 128, 0, 0.01, 0.1),
    (P.TILE256, 15000, 9, 2, 384, 1800, 0, 1, 0, 0.0, 1.0),
]


@pytest.mark.parametrize("path,N,E,K,C,M,act,align,cap,mask,skew", RECEIVED)
def test_received_rows(path, N, E, K, C, M, act, align, cap, mask, skew):
    """Experts from no rows to far more than the mean; rows that hold no token are
    neither read (their scales are NaN) nor written."""
    say(f"[matmul path] {path} {N} {E} {K} {C} {M} {act} {align} {cap}")
    assert P.matmul(N * K, C, M, act, E) == path
    g = gen(N + E)
    p = torch.rand((N, E), device="cuda", generator=g) + torch.linspace(skew, 0, E, device="cuda")
    if E > 2:
        p[:, 1] = -1                # nobody's expert
    idx = p.topk(K, dim=1).indices.to(torch.int32)
    idx[torch.rand((N, K), device="cuda", generator=g) < mask] = -1
    cfg = ep.Config(hidden=C, num_topk=K, num_experts=E, num_ranks=1, expert_alignment=align, expert_capacity=cap)
    h = ep.ep_handle_init(cfg, N)
    ep.ep_get_layout(h, idx)
    ep.ep_check_error(h)            # a full segment's flag
    v = ep.ep_handle_view(h)
    first, count = v["psum_expert"].tolist(), v["num_unaligned"].tolist()
    if cap:
        count = [min(n, cap) for n in count]
    rows = ep.ep_recv_capacity(cfg, N)
    w, s, W = stack(g, E, M, C)
    x, xs = rows_of(g, rows, C)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e in range(E):
        live[first[e]:first[e] + count[e]] = True
    xs[~live] = float("nan")
    y = torch.full((rows, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_expert_matmul(h, W, x, xs[:, None], y, activation=act)
    assert ep.ep_check_error(h) == (ep.EP_OK, 0)
    assert (y[~live] == 77).all()
    for e in range(E):
        if count[e]:
            r = slice(first[e], first[e] + count[e])
            check(y[r], x[r], xs[r], w[e], s[e], act)


@pytest.mark.parametrize("n,C,M", [(1, 7168, 7170), (5, 528, 8000), (16, 2064, 8191), (20, 1040, 3585), (32, 4112, 3599),
                                   (17, 16, 4090), (2, 7184, 8177)])
def test_thin_blocks_of_two_groups(n, C, M):
    """448 to 512 weight tiles of 16 for 16 rows: two to a block, of which the
    last one's second may be short or missing."""
    say(f"[matmul thin pairs] {n} {C} {M}")
    assert P.matmul(n, C, M) == P.THIN and P.splits(n, C, M) == 1
    assert 448 <= (n + 15) // 16 * ((M + 15) // 16) <= 512
    g = gen(n + M)
    w, s, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    buf = torch.full((n * M + 8,), 77.0, dtype=torch.bfloat16, device="cuda")
    y = buf[4:4 + n * M].view(n, M)
    moe.ep_matmul(W, x, xs, y)
    check(y, x, xs, w[0], s[0], 0)
    assert (buf[:4] == 77).all() and (buf[4 + n * M:] == 77).all()


@pytest.mark.parametrize("path,n,C,M", [(P.THIN, 20, 7168, 4096), (P.TILE64X64, 300, 1040, 520), (P.TILE64X128, 1024, 640, 4096),
                                        (P.TILE128, 2100, 272, 2050), (P.TILE256, 4096, 400, 4096)])
def test_replays_and_streams(path, n, C, M):
    """As a graph over changing rows, and two calls at once on two streams."""
    say(f"[matmul replays] {path} {n} {C} {M}")
    assert P.matmul(n, C, M) == path
    g = gen(n)
    w, s, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    y = torch.empty((n, M), dtype=torch.bfloat16, device="cuda")
    moe.ep_matmul(W, x, xs, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.ep_matmul(W, x, xs, y)
    for _ in range(3):
        x.random_(-128, 128, generator=g)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(y, x, xs, w[0], s[0], 0)
    x2, xs2 = rows_of(g, n, C)
    want = [y.clone(), moe.ep_matmul(W, x2, xs2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for k, (a, b) in enumerate(((x, xs), (x2, xs2))):
            with torch.cuda.stream(streams[k]):
                got[k].append(moe.ep_matmul(W, a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[k]) for k in range(2) for t in got[k])


@pytest.mark.parametrize("path,n,C,M", [(P.TILE64X64, 300, 1040, 520), (P.TILE64X128, 1024, 640, 4096),
                                        (P.TILE128, 2100, 272, 2048), (P.TILE256, 4096, 400, 4096),
                                        (P.TILE64X64, 20000, 512, 130), (P.TILE128, 20000, 256, 2048),
                                        (P.TILE128, 20000, 128, 2048)])
def test_scales_follow_their_tiles(path, n, C, M):
    """Tiles in a row on one block: scales that differ by powers of two from row
    to row and output to output would show another tile's."""
    say(f"[matmul scales] {path} {n} {C} {M}")
    assert P.matmul(n, C, M) == path
    g = gen(M)
    w, _, _ = stack(g, 1, M, C)
    s = torch.exp2((torch.arange(M, device="cuda") * 7 % 23 - 11).float())
    x, _ = rows_of(g, n, C)
    xs = torch.exp2((torch.arange(n, device="cuda") * 5 % 19 - 9).float())
    y = moe.ep_matmul(moe.Weights(moe.EP_WEIGHT_INT8, w, s[None]), x, xs)
    check(y, x, xs, w[0], s, 0)
