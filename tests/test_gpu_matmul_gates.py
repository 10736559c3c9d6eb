"""GPU tests of the gated products in 8-bit integers at gates far from 0, where the
exponential leaves fp32's range, in each kernel."""
import pytest
import torch

import matmul_paths as P
from combine_get_dispatch_layout_amd import ep, moe
from test_gpu_matmul_paths import BF16_HALF, U, gen, rows_of, say

pytestmark = pytest.mark.gpu


def stack(g, E, M, C):
    """Gates some 90 from 0 and up to 400, ups near 1."""
    w = torch.randint(-128, 128, (E, M, C), dtype=torch.int8, device="cuda", generator=g)
    s = (torch.rand((E, M), device="cuda", generator=g) + 0.5) * (C ** -0.5 / 64)
    s[:, :M // 2] *= 120
    return w, s, moe.Weights(moe.EP_WEIGHT_INT8, w, s)


def check(y, x, xs, w, s):
    """Gate and up are off by 3 u each, which changes a silu by at most its slope:
    1.1, and |g| e^g below -2.  The exponential is good to 1.5 u of its argument and
    some u of itself, 2^-16 for |g| < 90; below -88.72 it is infinite and the silu,
    less than 89 * 2^-128 there, is -0.  Then one rounding."""
    a = torch.mm(x.double(), w.double().t().contiguous()) * xs.double()[:, None] * s.double()[None]
    g, up = a.chunk(2, dim=1)
    out = g / (1 + torch.exp(-g)) * up
    slope = torch.where(g < -2, 1.01 * g.abs() * torch.exp(g), 1.1)
    err = slope * 3 * U * (g * up).abs() + (3 * U + 2.0 ** -16) * out.abs()
    err = torch.where(g < -88, 2.0 ** -121 * up.abs(), err)
    assert float(g.min()) < -100 and float(g.max()) > 100 and bool(((g > -88) & (g < -40)).any())
    bad = ~((y.double() - out).abs() <= err + BF16_HALF * (out.abs() + err) + 1e-38)
    assert not bad.any(), (int(bad.sum()), y[bad][:4], out[bad][:4], g[bad][:4])


@pytest.mark.parametrize("path,n,C,M", [(P.THIN, 16, 2064, 34), (P.TILE64X64, 65, 656, 66), (P.TILE64X64, 40, 16384, 96),
                                        (P.TILE64X128, 1500, 528, 1500), (P.TILE128, 2300, 384, 2062),
                                        (P.TILE256, 3700, 272, 4000)])
def test_one_matrix(path, n, C, M):
    say(f"[matmul gates] {path} {n} {C} {M}")
    assert P.matmul(n, C, M, 1) == path and (P.splits(n, C, M, 1) > 1) == (C == 16384)
    g = gen(n)
    w, s, W = stack(g, 1, M, C)
    x, xs = rows_of(g, n, C)
    check(moe.ep_matmul(W, x, xs, activation=moe.EP_ACT_SWIGLU), x, xs, w[0], s[0])


def test_few_rows_of_experts():
    N, E, K, C, M = 13, 9, 3, 7168, 514
    say(f"[matmul gates] few {N} {E} {K} {C} {M}")
    assert P.matmul(N * K, C, M, 1, E) == P.FEW
    g = gen(N)
    idx = torch.rand((N, E), device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    h = ep.ep_handle_init(ep.Config(hidden=C, num_topk=K, num_experts=E, num_ranks=1), N)
    ep.ep_get_layout(h, idx)
    first = ep.ep_handle_view(h)["psum_expert"].tolist()
    w, s, W = stack(g, E, M, C)
    x, xs = rows_of(g, N * K, C)
    y = moe.ep_expert_matmul(h, W, x, xs, activation=moe.EP_ACT_SWIGLU)
    e = max(range(E), key=lambda i: first[i + 1] - first[i])
    r = slice(first[e], first[e + 1])
    check(y[r], x[r], xs[r], w[e], s[e])
