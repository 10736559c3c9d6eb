"""GPU tests of each kernel that the expert products and the layer choose from,
at sizes that reach it (asserted), against 64-bit definitions: blocks that walk
many tiles and several experts, batches that end at the limits of segments and
of LDS, x from memory, partial last lines, scale rows of any length."""
import math

import numpy as np
import pytest
import torch

import moe_paths as P
import moe_reference as R
from combine_get_dispatch_layout_amd import ep, moe

pytestmark = pytest.mark.gpu

FMT = dict(bf16=moe.EP_WEIGHT_BF16, mxfp4=moe.EP_WEIGHT_MXFP4, int4=moe.EP_WEIGHT_INT4)
KINDS = [("bf16", 0, False), ("mxfp4", 32, False), ("int4", 32, False), ("int4", 32, True),
         ("int4", 64, False), ("int4", 64, True), ("int4", 128, False), ("int4", 128, True)]


def say(*a):
    print(*a, flush=True)


class Stack:
    """A stack of weights on the GPU and its experts' matrices in 64 bits."""

    def __init__(self, fmt, group, zeros, E, M, C, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.fmt, self.group, self.n = fmt, group, R.terms(C, group if fmt == "int4" else 0)
        self.s = self.z = None
        if fmt == "bf16":
            self.d = torch.empty((E, M, C), dtype=torch.bfloat16, device="cuda").normal_(0, C ** -0.5, generator=g)
        else:
            byte = dict(dtype=torch.uint8, device="cuda", generator=g)
            self.d = torch.randint(0, 256, (E, M, C // 2), **byte)
            if fmt == "mxfp4":
                mid = 126 - round(0.5 * math.log2(C))
                self.s = torch.randint(mid - 2, mid + 2, (E, M, C // 32), **byte)
            else:
                s = torch.rand((E, M, C // group), device="cuda", generator=g) - 0.3
                self.s = (s * 0.4 * C ** -0.5).to(torch.bfloat16)
                self.z = torch.randint(0, 16, s.shape, **byte) if zeros else None
        self.w = moe.Weights(FMT[fmt], self.d, self.s, self.z, group=group)

    def matrix(self, e):
        """float64 [M, C] and the magnitudes that the products' sums run over
        (INT4: of 16 + code and 16 + zero)."""
        if self.fmt == "bf16":
            w = self.d[e].double()
            return w, w.abs()
        b = self.d[e].int()
        q = torch.stack((b & 15, b >> 4), dim=2).flatten(1)
        s = self.s[e].repeat_interleave(self.group, 1)
        if self.fmt == "mxfp4":
            w = torch.from_numpy(R.E2M1).cuda()[q] * torch.exp2(s.double() - 127)
            return w, w.abs()
        z = 8.0 if self.z is None else self.z[e].double().repeat_interleave(self.group, 1)
        s = s.double()
        return (q - z) * s, (32 + q + z) * s.abs()


def product64(x, stack, e, act):
    """act(x W[e]^T) in 64 bits and the bound of its fp32 sums' errors; the
    activation's as in moe_reference.product."""
    w, mag = stack.matrix(e)
    y = torch.mm(x, w.t().contiguous())
    err = stack.n * R.F32_HALF * torch.mm(x.abs(), mag.t().contiguous())
    if not act:
        return y, err
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    silu = g / (1 + torch.exp(-g))
    out = silu * u
    return out, 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -18 * out.abs()


def layer64(x, idx, wts, up, down):
    """The whole layer and its bound, as moe_reference.layer, expert by expert."""
    x = x.double()
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    K = idx.shape[1]
    for e in range(up.d.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        w = wts[t, k].double()[:, None]
        a, ea = product64(x[t], up, e, 1)
        a, ea = w * a, w.abs() * ea
        m, mag = down.matrix(e)
        y = torch.mm(a, m.t().contiguous())
        # a in two bf16 terms: 2^-16 of it is lost
        ey = torch.mm(ea + 2.0 ** -16 * a.abs(), m.abs().t().contiguous()) + \
            2 * down.n * R.F32_HALF * torch.mm(a.abs() + ea, mag.t().contiguous())
        out.index_add_(0, t, y)
        err.index_add_(0, t, ey + K * R.F32_HALF * y.abs())
    return out, err


def close(got, want, err, what=""):
    R.assert_close(got, want.cpu().numpy(), err.cpu().numpy(), what)


def randn(rows, C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, C), device="cuda", generator=g).to(torch.bfloat16)


def routed(N, E, K, mask=0.0, seed=0, skew=0.0):
    """Distinct experts per token, the first ones more often with skew."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = torch.rand((N, E), device="cuda", generator=g) + torch.linspace(skew, 0, E, device="cuda")
    idx = p.topk(K, dim=1).indices.int()
    idx[torch.rand((N, K), device="cuda", generator=g) < mask] = -1
    return idx, torch.rand((N, K), device="cuda", generator=g)


def run_experts(path, idx, E, M, C, fmt, group, zeros, align=1, acts=(0, 1), seed=1):
    """ep_expert_matvec over the layout of idx; rows without a token hold NaN and
    stay as they were."""
    N, K = idx.shape
    cfg = ep.Config(hidden=C, num_topk=K, num_experts=E, num_ranks=1, expert_alignment=align)
    h = ep.ep_handle_init(cfg, N)
    ep.ep_get_layout(h, idx)
    v = ep.ep_handle_view(h)
    first, count = v["psum_expert"].tolist(), v["num_unaligned"].tolist()
    rows = ep.ep_recv_capacity(cfg, N)
    st = Stack(fmt, group, zeros, E, M, C, seed)
    x = randn(rows, C, seed + 1)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e in range(E):
        live[first[e]:first[e] + count[e]] = True
    xn = torch.where(live[:, None], x, float("nan"))
    for act in acts:
        assert P.product(fmt, group, C, M, E, N * K, act)[0] == path
        y = torch.full((rows, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_expert_matvec(h, st.w, xn, y, activation=act)
        assert ep.ep_check_error(h) == (ep.EP_OK, 0)
        again = moe.ep_expert_matvec(h, st.w, xn, torch.full_like(y, 77.0), activation=act)
        assert torch.equal(y, again)
        assert (y[~live] == 77).all()
        for e in range(E):
            if count[e]:
                s = slice(first[e], first[e] + count[e])
                want, err = product64(x[s].double(), st, e, act)
                close(y[s], want, err, (fmt, act, e))


# ---- 16 rows at once, x in LDS: 512 tiles and more ----------------------------------

@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("N,E,K,M,C,mask,skew,align", [
    (48, 64, 4, 2060, 384, 0.1, 1.5, 1),    # a partial last line; scale rows of 3, 6 and 12
    (48, 64, 4, 2060, 1024, 0.0, 1.5, 4),   # whole lines
    (60, 33, 8, 2062, 1664, 0.0, 0.0, 1),   # scale rows of 13, 26 and 52
    (20, 16, 3, 1050, 2176, 0.0, 0.0, 1),   # two or four waves share a tile's columns
    (20, 18, 3, 2062, 2048, 0.0, 0.0, 1),
])
def test_experts_one_tile(N, E, K, M, C, mask, skew, align, fmt, group, zeros):
    """Blocks take several steps of eight tiles and end inside an expert."""
    say(f"[one tile] {N} {E} {K} {M} {C} {fmt} {group} {zeros}")
    idx, _ = routed(N, E, K, mask, seed=N, skew=skew)
    run_experts(P.ONE_TILE, idx, E, M, C, fmt, group, zeros, align)


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
def test_experts_one_tile_segment_limit(fmt, group, zeros):
    """963 experts of 17 rows, two passes of two tiles each: a block's 15 or 16
    tiles lie in up to nine passes, one more than are in LDS together."""
    say(f"[segments] {fmt} {group} {zeros}")
    ids = torch.randperm(1024, generator=torch.Generator().manual_seed(3))[:963].repeat(17)
    idx = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(4))].int().cuda()[:, None]
    run_experts(P.ONE_TILE, idx, 1024, 62, 128, fmt, group, zeros, acts=(0,))


@pytest.mark.parametrize("fmt,group,zeros", [KINDS[0], KINDS[1], KINDS[3], KINDS[6]])
def test_experts_one_tile_rows_limit(fmt, group, zeros):
    """Rows of x so wide that LDS holds four: passes of four rows for a mean of
    four, batches of one or a few passes."""
    say(f"[rows] {fmt} {group} {zeros}")
    C = 15360
    idx, _ = routed(64, 64, 4, seed=5, skew=1.0)
    assert P.product(fmt, group, C, 1060, 64, 256) == (P.ONE_TILE, 4)
    run_experts(P.ONE_TILE, idx, 64, 1060, C, fmt, group, zeros, acts=(0,))


# ---- x from memory ----------------------------------------------------------------

WIDE = dict(bf16=(5000, 8192), mxfp4=(5024, 8192), int4=(5248, 8192))


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("rows,M", [(16, 600), (13, 34)])
@pytest.mark.parametrize("whole", [False, True])
def test_matvec_memory(whole, rows, M, fmt, group, zeros):
    C = WIDE[fmt][whole]
    say(f"[memory] {rows} {M} {C} {fmt} {group} {zeros}")
    st, x = Stack(fmt, group, zeros, 1, M, C, M), randn(rows, C, rows)
    for act in (0, 1):
        assert P.product(fmt, group, C, M, 1, rows, act)[0] == P.MEMORY
        y = torch.full((rows + 1, M // 2 if act else M), 77.0, dtype=torch.bfloat16, device="cuda")
        moe.ep_matvec(st.w, x, y[:rows], activation=act)
        close(y[:rows], *product64(x.double(), st, 0, act))
        assert (y[rows:] == 77).all()


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
def test_matvec_memory_many_tiles(fmt, group, zeros):
    """More tiles than waves run at a time: each takes several, x loaded ahead."""
    C, M, rows = WIDE[fmt][0], 70002, 15
    say(f"[memory, tiles] {fmt} {group} {zeros}")
    st, x = Stack(fmt, group, zeros, 1, M, C, 3), randn(rows, C, 4)
    assert P.product(fmt, group, C, M, 1, rows)[0] == P.MEMORY
    close(moe.ep_matvec(st.w, x), *product64(x.double(), st, 0, 0))


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("M,skew", [(2060, 0.7), (130, 0.0)])
def test_experts_memory(M, skew, fmt, group, zeros):
    """Waves go from one expert's tiles to the next, with the next one's x."""
    say(f"[memory, experts] {M} {fmt} {group} {zeros}")
    idx, _ = routed(32, 4, 2, 0.0, seed=M, skew=skew)
    run_experts(P.MEMORY, idx, 4, M, WIDE[fmt][0], fmt, group, zeros)


def test_memory_keeps_columns_behind_the_row_apart():
    """An infinity at the start of the next row of x and NaN weights of the next
    output must not enter a row's partial last line."""
    for fmt, group in (("bf16", 0), ("mxfp4", 32), ("int4", 128)):
        C = WIDE[fmt][0]
        st, x = Stack(fmt, group, False, 1, 40, C, 3), randn(16, C, 4)
        assert P.product(fmt, group, C, 40, 1, 16)[0] == P.MEMORY
        want = moe.ep_matvec(st.w, x)
        x[8] = float("inf")
        if fmt == "bf16":
            st.d[0, 9] = float("nan")
        elif fmt == "mxfp4":
            st.s[0, 9] = 255
        else:
            st.s[0, 9] = float("nan")
        got = moe.ep_matvec(st.w, x)
        rows, outs = [r for r in range(16) if r != 8], [m for m in range(40) if m != 9]
        assert torch.equal(got[rows][:, outs], want[rows][:, outs]), fmt
        assert torch.isnan(got[:, 9]).all() and not torch.isfinite(got[8]).any()


# ---- 32 rows at once -----------------------------------------------------------------

@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("rows,M,C,at_once", [(70000, 40, 128, 32), (40, 1000, 1024, 31), (1000, 2050, 3328, 19)])
def test_matvec_two_tiles(rows, M, C, at_once, fmt, group, zeros):
    """Blocks over several passes; LDS too small for 32 rows (3328 columns)."""
    say(f"[two tiles] {rows} {M} {C} {fmt} {group} {zeros}")
    assert P.product(fmt, group, C, M, 1, rows) == (P.TWO_TILES, at_once)
    st, x = Stack(fmt, group, zeros, 1, M, C, 3), randn(rows, C, 4)
    close(moe.ep_matvec(st.w, x), *product64(x.double(), st, 0, 0))


# ---- layers ---------------------------------------------------------------------------

def run_layer(paths, N, E, K, H, I, fmt, group, zeros, mask=0.0, skew=0.0):
    assert P.layer(fmt, group, N, K, E, H, I) == paths
    idx, wts = routed(N, E, K, mask, seed=N, skew=skew)
    if N > 3:
        idx[2], idx[3] = -1, int(idx[3, 0])                  # no expert; one expert K times
    up, down = Stack(fmt, group, zeros, E, 2 * I, H, 1), Stack(fmt, group, zeros, E, H, I, 2)
    x = randn(N, H, 3)
    h = ep.ep_handle_init(ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1), 1)
    out = torch.full((N + 1, H), 77.0, dtype=torch.bfloat16, device="cuda")
    moe.ep_moe_layer(h, up.w, down.w, x, idx, wts, out[:N])
    assert ep.ep_check_error(h) == (ep.EP_OK, 0) and (out[N:] == 77).all()
    close(out[:N], *layer64(x, idx, wts, up, down))
    assert torch.equal(out[:N], moe.ep_moe_layer(h, up.w, down.w, x, idx, wts))
    return h, up, down, x, idx, wts, out[:N].clone()


def nan_expert(st, e):
    if st.fmt == "bf16":
        st.d[e] = float("nan")
    elif st.fmt == "mxfp4":
        st.s[e] = 255
    else:
        st.s[e] = float("inf")


def check_isolation(h, up, down, x, idx, wts, want):
    """One expert's weights become NaN: only the tokens that chose it see it."""
    live = [e for e in idx.unique().tolist() if e >= 0 and not (idx == e).any(1).all()]
    if not live:
        assert idx.shape[0] == 1
        return
    e = live[0]
    nan_expert(up, e)
    nan_expert(down, e)
    got = moe.ep_moe_layer(h, up.w, down.w, x, idx, wts)
    hit = (idx == e).any(1)
    assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()


LAYER = dict(bf16=(1032, 520), mxfp4=(1056, 544), int4=(1152, 640))


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("whole,N,K,mask,skew", [(False, 48, 4, 0.1, 1.5), (True, 200, 3, 0.0, 0.5)])
def test_layer_one_tile(whole, N, K, mask, skew, fmt, group, zeros):
    H, I = (1024, 1024) if whole else LAYER[fmt]
    say(f"[layer] {N} {K} {H} {I} {fmt} {group} {zeros}")
    c = run_layer((P.ONE_TILE, P.ONE_TILE), N, 64, K, H, I, fmt, group, zeros, mask, skew)
    check_isolation(*c)


LAYER_WIDE = dict(bf16=(5000, 2504), mxfp4=(5024, 2528), int4=(5248, 2688))


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
@pytest.mark.parametrize("whole", [False, True])
def test_layer_memory(whole, fmt, group, zeros):
    """Both projections' rows past LDS."""
    H, I = (5120, 2560) if whole else LAYER_WIDE[fmt]
    say(f"[layer, memory] {H} {I} {fmt} {group} {zeros}")
    check_isolation(*run_layer((P.MEMORY, P.MEMORY), 33, 4, 2, H, I, fmt, group, zeros, 0.0, 0.0))


@pytest.mark.parametrize("fmt,group,zeros", KINDS)
def test_layer_two_tiles(fmt, group, zeros):
    H, I = LAYER[fmt]
    say(f"[layer, two tiles] {H} {I} {fmt} {group} {zeros}")
    check_isolation(*run_layer((P.TWO_TILES, P.TWO_TILES), 150, 8, 2, H, I, fmt, group, zeros, 0.0, 0.4))


# the largest batches whose experts are added inside the down projection, and
# one step above each
@pytest.mark.parametrize("fmt,group,N,K,I,two", [
    ("bf16", 0, 16, 2, 448, True), ("bf16", 0, 16, 2, 456, False), ("bf16", 0, 11, 3, 64, False),
    ("bf16", 0, 17, 1, 64, False), ("bf16", 0, 2, 16, 448, True), ("mxfp4", 32, 16, 2, 256, True),
    ("mxfp4", 32, 15, 2, 512, True), ("mxfp4", 32, 16, 2, 512, False), ("mxfp4", 32, 11, 3, 256, False),
    ("mxfp4", 32, 16, 1, 768, True), ("mxfp4", 32, 16, 1, 1024, False), ("int4", 128, 8, 4, 256, True),
    ("int4", 128, 15, 2, 384, True), ("int4", 128, 3, 11, 256, False), ("int4", 64, 1, 8, 1728, True),
    ("int4", 64, 8, 1, 832, True), ("int4", 64, 9, 1, 832, False), ("int4", 32, 2, 4, 1760, True),
    ("int4", 32, 4, 2, 224, True), ("int4", 32, 3, 3, 224, False)])
def test_layer_handful_limits(fmt, group, N, K, I, two):
    say(f"[handful] {N} {K} {I} {fmt} {group}")
    paths = P.layer(fmt, group, N, K, 17, 256, I)
    assert (paths[1] == 0) == two
    c = run_layer(paths, N, 17, K, 256, I, fmt, group, fmt == "int4" and group != 64, 0.05)
    check_isolation(*c)


# ---- calls side by side ------------------------------------------------------------------

MIXED = [(("bf16", 0, False), ("mxfp4", 32, False)), (("mxfp4", 32, False), ("int4", 128, False)),
         (("int4", 32, True), ("bf16", 0, False)), (("int4", 64, False), ("int4", 32, True))]


@pytest.mark.parametrize("kinds", MIXED)
@pytest.mark.parametrize("N,E,K,H,I", [(1, 8, 2, 256, 128), (7, 8, 2, 384, 256), (40, 8, 3, 256, 384), (48, 64, 4, 1152, 640)])
def test_layer_of_two_formats(N, E, K, H, I, kinds):
    say(f"[two formats] {N} {H} {I} {kinds}")
    up, down = Stack(*kinds[0], E, 2 * I, H, 1), Stack(*kinds[1], E, H, I, 2)
    idx, wts = routed(N, E, K, 0.1, seed=N)
    x = randn(N, H, 3)
    h = ep.ep_handle_init(ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1), 1)
    close(moe.ep_moe_layer(h, up.w, down.w, x, idx, wts), *layer64(x, idx, wts, up, down))


def test_calls_at_once_on_two_streams():
    """Layers and products in flight together, sharing weights and the handle."""
    E, K, H, I, N = 64, 4, 1152, 640, 48
    up, down = Stack("mxfp4", 32, False, E, 2 * I, H, 1), Stack("mxfp4", 32, False, E, H, I, 2)
    h = ep.ep_handle_init(ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1), N)
    idx, wts = routed(N, E, K, 0.1, seed=1)
    ep.ep_get_layout(h, idx)
    recv = randn(N * K, H, 5)
    xs = [randn(N, H, 6 + i) for i in range(2)]
    want = [moe.ep_moe_layer(h, up.w, down.w, x, idx, wts) for x in xs]
    y0 = moe.ep_expert_matvec(h, up.w, recv, torch.zeros((N * K, I), dtype=torch.bfloat16, device="cuda"), activation=1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.ep_moe_layer(h, up.w, down.w, xs[i], idx, wts))
                got[i].append(moe.ep_expert_matvec(h, up.w, recv, torch.zeros_like(y0), activation=1))
    torch.cuda.synchronize()
    for i in range(2):
        for r in range(5):
            assert torch.equal(got[i][2 * r], want[i]) and torch.equal(got[i][2 * r + 1], y0)
    assert ep.ep_check_error(h) == (ep.EP_OK, 0)


@pytest.mark.parametrize("E,K,H,I,N", [(16, 3, 256, 128, 30), (64, 4, 1024, 640, 48)])
def test_shuffled_path_graph_replays(E, K, H, I, N):
    """Router, layout, dispatch, both products and combine as one graph, against
    the eager calls, with new logits and eager work between the replays."""
    up, down = Stack("int4", 64, True, E, 2 * I, H, 1), Stack("int4", 64, True, E, H, I, 2)
    cfg = ep.Config(hidden=H, num_topk=K, num_experts=E, num_ranks=1, expert_alignment=2)
    gcfg = moe.GateConfig(E, K, moe.EP_SCORE_SIGMOID)
    rows = ep.ep_recv_capacity(cfg, N)
    lg, x = torch.randn((N, E), device="cuda"), randn(N, H, 1)
    new = lambda r, c: torch.zeros((r, c), dtype=torch.bfloat16, device="cuda")  # noqa: E731

    def make():
        return dict(h=ep.ep_handle_init(cfg, N), recv=new(rows, H), act=new(rows, I), y=new(rows, H), out=new(N, H),
                    idx=torch.zeros((N, K), dtype=torch.int32, device="cuda"), w=torch.zeros((N, K), device="cuda"))

    def step(b):
        moe.ep_gate(gcfg, lg, topk_idx=b["idx"], topk_weights=b["w"])
        ep.ep_get_layout(b["h"], b["idx"], alloc_outputs=False)
        ep.ep_dispatch(b["h"], x, b["recv"])
        moe.ep_expert_matvec(b["h"], up.w, b["recv"], b["act"], activation=1)
        moe.ep_expert_matvec(b["h"], down.w, b["act"], b["y"])
        ep.ep_combine(b["h"], b["y"], b["w"], b["out"])

    a, b = make(), make()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for i in range(4):
        lg.normal_()
        x.copy_(randn(N, H, 20 + i))
        a["out"].fill_(77)
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["idx"], b["idx"]) and torch.equal(a["out"], b["out"]), i
    for c in (a, b):
        assert ep.ep_check_error(c["h"]) == (ep.EP_OK, 0)


def test_layout_that_waits_is_refused():
    """A layout that the next combine finishes is not there yet."""
    cfg = ep.Config(hidden=64, num_topk=2, num_experts=8, num_ranks=1)
    h, nxt = ep.ep_handle_init(cfg, 4000), ep.ep_handle_init(cfg, 4000)
    idx, wts = routed(4000, 8, 2, seed=1)
    ep.ep_get_layout(h, idx)
    recv, x, out = randn(8000, 64, 1), randn(4000, 64, 2), randn(4000, 64, 3)
    ep.ep_dispatch_overlap(h, x, recv, h_next=nxt, topk_next=idx)
    st = Stack("bf16", 0, False, 8, 40, 64, 1)
    want = moe.ep_expert_matvec(h, st.w, recv)
    try:
        got = moe.ep_expert_matvec(nxt, st.w, recv)
    except ep.EpError as e:
        assert e.status == ep.EP_ERR_STATE
        ep.ep_combine_overlap(h, recv, wts, out, h_next=nxt)
        got = moe.ep_expert_matvec(nxt, st.w, recv)
    assert torch.equal(got, want)
