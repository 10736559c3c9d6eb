"""GPU tests of products in 8-bit integers whose columns are split over blocks
(ep_matmul_split): the bits of ep_matmul, which are checked against sums in 64
bits as in test_gpu_matmul_paths."""
import pytest
import torch

import matmul_paths as P
from combine_get_dispatch_layout_amd import ep, moe
from test_gpu_matmul_paths import check, gen, rows_of, say, stack

pytestmark = pytest.mark.gpu


def unsplit(W, x, xs, act=0):
    y = torch.empty((x.shape[0], W.rows // 2 if act else W.rows), dtype=torch.bfloat16, device="cuda")
    moe._call(x.device, moe._lib().ep_matmul, W._ref, x.data_ptr(), xs.data_ptr(), x.shape[0], act, y.data_ptr())
    return y


# rows, columns, weight rows, gate: whole and ragged tiles, a last step of few
# columns, shares of the steps that differ, outputs that no vector takes
CASES = [(33, 7168, 4096, 0), (64, 7168, 512, 1), (64, 16384, 1000, 0), (65, 7184, 130, 0), (1, 65536, 200, 0),
         (17, 32784, 66, 1), (40, 4112, 1002, 1), (40, 12304, 1003, 0), (128, 9232, 34, 1), (300, 8208, 1, 0),
         (700, 16400, 2, 1), (130, 131056, 48, 0), (5, 131056, 3, 0), (512, 7168, 1024, 0)]


@pytest.mark.parametrize("n,C,M,act", CASES)
def test_split(n, C, M, act):
    say(f"[matmul split] {n} {C} {M} {act}: {P.splits(n, C, M, act)}")
    split = P.splits(n, C, M, act)
    g = gen(n + C)
    w, s, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    out = M // 2 if act else M
    need = moe.ep_matmul_workspace_size(W, n, act)
    assert need == (4 * split * n * M if split > 1 else 0)
    ws = torch.full((need + 256,), 113, dtype=torch.uint8, device="cuda")
    buf = torch.full((n * out + 9,), 77.0, dtype=torch.bfloat16, device="cuda")
    want = unsplit(W, x, xs, act)
    check(want, x, xs, w[0], s[0], act)
    for shift in (0, 1):            # a y that is aligned, and one that is not
        y = buf[shift:shift + n * out].view(n, out)
        y.fill_(5.0)
        moe.ep_matmul(W, x, xs, y, act, ws[:need] if need else None)
        assert torch.equal(y, want)
        assert (ws[need:] == 113).all() and (buf[n * out + 1:] == 77).all()
    assert torch.equal(moe.ep_matmul(W, x, xs[:, None].contiguous(), activation=act), want)


def test_most_cases_are_split():
    assert sum(P.splits(*c) > 1 for c in CASES) >= 12


def test_scales_of_any_kind():
    """An infinite or NaN scale reaches its row or output alone."""
    g = gen(9)
    w, s, W = stack(g, 1, 96, 16384)
    x, xs = rows_of(g, 40, 16384)
    assert P.splits(40, 16384, 96) > 1
    want = moe.ep_matmul(W, x, xs)
    xs2, s2 = xs.clone(), s.clone()
    xs2[3], xs2[7], s2[0, 11], s2[0, 95] = float("inf"), float("nan"), float("nan"), 0.0
    got = moe.ep_matmul(moe.Weights(moe.EP_WEIGHT_INT8, w, s2), x, xs2)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    outs = torch.ones(96, dtype=torch.bool, device="cuda")
    rows[[3, 7]] = False
    outs[[11, 95]] = False
    assert torch.equal(got[rows][:, outs], want[rows][:, outs])
    assert got[7].isnan().all() and got[:, 11].isnan().all() and not got[3][outs].isfinite().any()
    assert (got[rows, 95] == 0).all()


def test_sums_at_their_limits():
    n, C, M = 3, 131056, 5
    say(f"[matmul split limits] {P.splits(n, C, M)}")
    W = moe.Weights(moe.EP_WEIGHT_INT8, torch.full((M, C), -128, dtype=torch.int8, device="cuda"),
                    torch.ones(M, device="cuda"))
    x = torch.full((n, C), -128, dtype=torch.int8, device="cuda")
    x[1] = 127
    y = moe.ep_matmul(W, x, torch.ones(n, device="cuda"))
    for r, v in enumerate((128 * 128 * C, -127 * 128 * C, 128 * 128 * C)):
        assert (y[r] == torch.tensor(float(v)).to(torch.bfloat16).item()).all()


def test_workspaces():
    g = gen(2)
    _, _, W = stack(g, 1, 256, 7168)
    x, xs = rows_of(g, 64, 7168)
    need = moe.ep_matmul_workspace_size(W, 64)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    with pytest.raises(ep.EpError):
        moe.ep_matmul(W, x, xs, workspace=ws[:-1])
    with pytest.raises(ep.EpError):
        moe.ep_matmul(W, x, xs, workspace=torch.empty(need + 128, dtype=torch.uint8, device="cuda")[128:])
    with pytest.raises(ValueError):
        moe.ep_matmul(W, x, xs, workspace=torch.empty(need, dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError):
        moe.ep_matmul(W, x, xs, workspace=torch.empty(need, dtype=torch.uint8))
    want = unsplit(W, x, xs)
    for fill in (0, 255, 113):      # needs no clearing
        ws.fill_(fill)
        assert torch.equal(moe.ep_matmul(W, x, xs, workspace=ws), want)


def test_replays_and_streams():
    """As a graph over changing rows, and two calls at once on two streams."""
    g = gen(4)
    n, C, M = 64, 7168, 1000
    assert P.splits(n, C, M) > 1
    _, _, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    y = torch.empty((n, M), dtype=torch.bfloat16, device="cuda")
    moe.ep_matmul(W, x, xs, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.ep_matmul(W, x, xs, y)
    for _ in range(4):
        x.random_(-128, 128, generator=g)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, unsplit(W, x, xs))
    x2, xs2 = rows_of(g, n, C)
    want = [y.clone(), unsplit(W, x2, xs2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(6):
        for k, (a, b) in enumerate(((x, xs), (x2, xs2))):
            with torch.cuda.stream(streams[k]):
                got[k].append(moe.ep_matmul(W, a, b))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[k]) for k in range(2) for t in got[k])
