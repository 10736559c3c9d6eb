"""The operators around the token shuffle -- the router, products with expert
weights, the whole expert layer for a few tokens -- as measured cases.

Each case is prepared on the GPU from a seed; `run` makes one pass, in plain
torch operations (own = False) or through the package's calls (own = True);
`exact` gives the same outputs from the definitions in 64 bits.

Weights are a stack [experts, rows, cols]: bf16; "mxfp4", two E2M1 codes a
byte (column 2i in the low nibble) and one E8M0 scale byte per 32 columns; or
"int4", value (code - zero) * scale with a bf16 scale and a zero byte (8 where
there are none) per group of columns.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases -----------------------------------------------------------------

def _gate(op, tokens, experts, topk, score="softmax", renorm=True, bias=False, groups=0, topk_groups=0,
          group_top=0, group_limit=False, dtype="fp32", scale=1.0, masked=0.0):
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, score=score, renorm=renorm, bias=bias,
                groups=groups, topk_groups=topk_groups, group_top=group_top, group_limit=group_limit,
                dtype=dtype, scale=scale, masked=masked)


def _matvec(tokens, cols, rows, fmt, group=0, zeros=False, act="none"):
    return dict(op="matvec", tokens=tokens, cols=cols, rows=rows, fmt=fmt, group=group, zeros=zeros, act=act)


def _experts(tokens, experts, topk, cols, rows, fmt, group=0, zeros=False, act="none", masked=0.0):
    return dict(op="experts", tokens=tokens, experts=experts, topk=topk, cols=cols, rows=rows, fmt=fmt,
                group=group, zeros=zeros, act=act, masked=masked)


def _layer(tokens, experts, topk, hidden, inter, fmt, group=0, zeros=False, masked=0.0):
    return dict(op="layer", tokens=tokens, experts=experts, topk=topk, hidden=hidden, inter=inter, fmt=fmt,
                group=group, zeros=zeros, masked=masked)


def listed():
    return [
        # the router of one decoded token
        dict(_gate("gate", 1, 256, 8), name="gate_token"),
        # a prefill batch under group-limited gating with a balancing bias
        dict(_gate("gate", 8192, 256, 8, score="sigmoid", bias=True, groups=32, topk_groups=4, group_top=2,
                   group_limit=True, scale=2.5), name="gate_prefill_groups"),
        # training: gradients of raw softmax weights, logits in bf16
        dict(_gate("gate_grad", 4096, 128, 8, renorm=False, dtype="bf16"), name="gate_grad_softmax"),
        # training: normalised sigmoid weights, a batch with masked tokens
        dict(_gate("gate_grad", 8191, 256, 8, score="sigmoid", scale=2.5, masked=0.1), name="gate_grad_sigmoid"),
        # one token through one small 4-bit matrix: launch latency
        dict(_matvec(1, 2048, 2048, "int4", 128), name="matvec_token_int4"),
        # a ragged handful of tokens through a large MXFP4 matrix
        dict(_matvec(13, 7168, 14336, "mxfp4", 32), name="matvec_batch_mxfp4"),
        # the up projection with its gated activation on a dispatched decode batch
        dict(_experts(128, 256, 8, 7168, 4096, "mxfp4", 32, act="swiglu"), name="experts_decode_mxfp4"),
        # a down projection, asymmetric 4-bit codes, few tokens, masked entries
        dict(_experts(23, 64, 6, 1024, 4096, "int4", 64, zeros=True, masked=0.05), name="experts_few_int4"),
        # one token through the whole layer, bf16 weights
        dict(_layer(1, 128, 8, 2048, 768, "bf16"), name="layer_token_bf16"),
        # the same with MXFP4 weights
        dict(_layer(1, 128, 8, 2048, 768, "mxfp4", 32), name="layer_token_mxfp4"),
        # a few concurrent sequences, fine groups with zero points
        dict(_layer(17, 128, 8, 2048, 768, "int4", 32, zeros=True), name="layer_few_int4"),
        # a full decode batch: every expert's weights are read
        dict(_layer(128, 256, 8, 7168, 2048, "int4", 128), name="layer_decode_int4"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gate", "gate_grad", "matvec", "experts", "layer", "layer"])
    if op in ("gate", "gate_grad"):
        per = rng.choice([4, 5, 8, 11, 16, 32])
        groups = rng.choice([2, 4, 8, 16, 32])
        topk_groups = rng.randint(1, min(4, groups))
        top = rng.randint(1, min(2, per))
        limited = rng.random() < 0.5
        topk = topk_groups * top if limited else rng.randint(1, min(8, topk_groups * per))
        if op == "gate_grad" or rng.random() < 0.5:
            groups = topk_groups = top = 0
            limited = False
            experts = _log(rng, 8, 256)
            topk = rng.randint(1, 8)
        else:
            experts = groups * per
        while experts > 256:
            groups //= 2
            experts = groups * per
            if topk_groups > groups:
                return draw(rng)
        return _gate(op, _log(rng, 1, 8192), experts, topk, rng.choice(["softmax", "sigmoid"]),
                     rng.random() < 0.6, op == "gate" and rng.random() < 0.4, groups, topk_groups, top, limited,
                     rng.choice(["fp32", "fp32", "bf16"]), rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.1]))
    fmt, group = rng.choice([("bf16", 0), ("mxfp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)])
    zeros = fmt == "int4" and rng.random() < 0.5
    unit = group or 8
    if op == "matvec":
        act = rng.choice(["none", "none", "swiglu"])
        rows = _log(rng, 33, 7168)
        return _matvec(_log(rng, 1, 64), unit * _log(rng, 256 // unit, 7168 // unit), 2 * rows if act == "swiglu" else rows,
                       fmt, group, zeros, act)
    experts = rng.choice([8, 16, 33, 64, 128])
    topk = rng.randint(1, min(8, experts))
    tokens, masked = _log(rng, 1, 128), rng.choice([0.0, 0.0, 0.05])
    cols = unit * _log(rng, 256 // unit, 4096 // unit)
    if op == "experts":
        act = rng.choice(["none", "swiglu"])
        rows = _log(rng, 65, 2048)
        return _experts(tokens, experts, topk, cols, 2 * rows if act == "swiglu" else rows, fmt, group, zeros, act, masked)
    return _layer(tokens, experts, topk, cols, unit * _log(rng, 128 // unit, 1024 // unit), fmt, group, zeros, masked)


# ---- inputs ----------------------------------------------------------------

def _weights(gen, experts, rows, cols, fmt, group, zeros):
    """Weights of a spread near 1/sqrt(cols), as a loaded checkpoint holds them."""
    if fmt == "bf16":
        w = torch.empty((experts, rows, cols), dtype=torch.bfloat16, device="cuda")
        return dict(fmt=fmt, group=group, data=w.normal_(0, cols ** -0.5, generator=gen), scales=None, zeros=None)
    a = torch.randint(0, 256, (experts, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    if fmt == "mxfp4":
        low = 126 - int(round(0.5 * math.log2(cols)))
        s = torch.randint(low - 2, low + 1, (experts, rows, cols // 32), dtype=torch.uint8, device="cuda", generator=gen)
        return dict(fmt=fmt, group=group, data=a, scales=s, zeros=None)
    # codes 0..14 with a peak at 7, as quantised normal weights have
    b = torch.randint(0, 256, (experts, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    codes = (a & 0x77) + (b & 0x77)
    s = torch.rand((experts, rows, cols // group), device="cuda", generator=gen)
    s = ((0.5 + s) * 0.3 * cols ** -0.5).to(torch.bfloat16)
    z = torch.randint(6, 10, s.shape, dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return dict(fmt=fmt, group=group, data=codes, scales=s, zeros=z)


def _routing(gen, tokens, experts, topk, masked):
    """Distinct uniform experts per token, some entries masked; softmax weights."""
    idx = torch.rand((tokens, experts), device="cuda", generator=gen).topk(topk, dim=1).indices.to(torch.int32)
    wts = torch.randn((tokens, topk), device="cuda", generator=gen).softmax(1)
    if masked:
        idx[torch.rand((tokens, topk), device="cuda", generator=gen) < masked] = -1
    return idx, wts


def _out_rows(c):
    return c["rows"] // 2 if c["act"] == "swiglu" else c["rows"]


def _randn(gen, *shape):
    return torch.randn(shape, device="cuda", generator=gen).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=c)
    if c["op"] in ("gate", "gate_grad"):
        N, E = c["tokens"], c["experts"]
        st["logits"] = torch.randn((N, E), device="cuda", generator=gen)
        if c["dtype"] == "bf16":
            st["logits"] = st["logits"].to(torch.bfloat16)
        st["bias"] = 0.1 * torch.randn(E, device="cuda", generator=gen) if c["bias"] else None
        st["mask"] = torch.rand(N, device="cuda", generator=gen) >= c["masked"] if c["masked"] else None
        if c["op"] == "gate_grad":
            idx = st["logits"].float().topk(c["topk"], dim=1).indices.to(torch.int32)
            if c["masked"]:
                idx[~st["mask"]] = -1
            st["idx"] = idx
            st["grad"] = torch.randn((N, c["topk"]), device="cuda", generator=gen)
        return st
    if c["op"] == "matvec":
        st["w"] = _weights(gen, 1, c["rows"], c["cols"], c["fmt"], c["group"], c["zeros"])
        st["x"] = _randn(gen, c["tokens"], c["cols"])
        return st
    st["idx"], st["wts"] = _routing(gen, c["tokens"], c["experts"], c["topk"], c["masked"])
    if c["op"] == "layer":
        st["up"] = _weights(gen, c["experts"], 2 * c["inter"], c["hidden"], c["fmt"], c["group"], c["zeros"])
        st["down"] = _weights(gen, c["experts"], c["hidden"], c["inter"], c["fmt"], c["group"], c["zeros"])
        st["x"] = _randn(gen, c["tokens"], c["hidden"])
        return st
    # a dispatched batch: rows grouped by expert, (token, k) order inside
    st["w"] = _weights(gen, c["experts"], c["rows"], c["cols"], c["fmt"], c["group"], c["zeros"])
    ids = st["idx"].reshape(-1)
    ids = ids[ids >= 0].sort(stable=True).values.long()
    st["row_expert"] = ids
    st["most"] = int(torch.bincount(ids, minlength=c["experts"]).max()) if ids.numel() else 0
    # the receive buffer is sized for every entry; masked ones leave rows at its end unused
    st["x"] = _randn(gen, c["tokens"] * c["topk"], c["cols"])
    st["y"] = torch.zeros((c["tokens"] * c["topk"], _out_rows(c)), dtype=torch.bfloat16, device="cuda")
    return st


# ---- plain form ------------------------------------------------------------

def _dequant(w, pick=None):
    """fp32 weights [n, rows, cols] of the picked experts (all by default)."""
    def part(t):
        return t if pick is None or t is None else t[pick]
    data = part(w["data"])
    if w["fmt"] == "bf16":
        return data.float()
    n, rows, half = data.shape
    codes = torch.stack((data & 15, data >> 4), dim=3).reshape(n, rows, 2 * half // w["group"], w["group"])
    if w["fmt"] == "mxfp4":
        v = torch.tensor(E2M1, device=data.device)[codes.int()]
        v *= torch.exp2(part(w["scales"]).float() - 127)[..., None]
    else:
        v = codes.float()
        v -= 8.0 if w["zeros"] is None else part(w["zeros"]).float()[..., None]
        v *= part(w["scales"]).float()[..., None]
    return v.reshape(n, rows, 2 * half)


def _swiglu(a):
    g, u = a.chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def _plain_gate(st):
    c = st["case"]
    z = st["logits"].double()
    N, E = z.shape
    s = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    choice = s if st["bias"] is None else s + st["bias"].double()
    key = z if st["bias"] is None else choice
    if c["groups"]:
        per = E // c["groups"]
        grouped = choice.reshape(N, c["groups"], per)
        best = grouped.sort(dim=2, descending=True, stable=True).values[..., :c["group_top"]].sum(2)
        chosen = best.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, chosen, True)[..., None].expand(-1, -1, per)
        if c["group_limit"]:
            order = key.reshape(N, c["groups"], per).sort(dim=2, descending=True, stable=True).indices
            first = torch.zeros_like(grouped, dtype=torch.bool).scatter_(2, order[..., :c["group_top"]], True)
            allowed = allowed & first
        key = key.masked_fill(~allowed.reshape(N, E), -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w, idx = (w * c["scale"]).float(), idx.to(torch.int32)
    if st["mask"] is not None:
        idx = torch.where(st["mask"][:, None], idx, -1)
        w = torch.where(st["mask"][:, None], w, 0.0)
    return idx, w


def _plain_gate_grad(st):
    c = st["case"]
    z, g = st["logits"].float(), st["grad"]
    live = st["idx"] >= 0
    at = st["idx"].clamp(min=0).long()
    g = torch.where(live, g, 0.0) * c["scale"]
    if c["score"] == "softmax":
        if c["renorm"]:
            p = torch.softmax(z.gather(1, at), 1)
            return _scattered(z, at, torch.where(live, p * (g - (p * g).sum(1, keepdim=True)), 0.0), st)
        p = torch.softmax(z, 1)
        per = torch.zeros_like(p).scatter_add_(1, at, g)
        return (p * (per - (p * per).sum(1, keepdim=True))).to(st["logits"].dtype)
    s = torch.sigmoid(z.gather(1, at))
    d = s * (1 - s)
    if c["renorm"]:
        total = s.sum(1, keepdim=True)
        d = d / total * (g - (s * g).sum(1, keepdim=True) / total)
    else:
        d = d * g
    return _scattered(z, at, torch.where(live, d, 0.0), st)


def _scattered(z, at, d, st):
    return torch.zeros_like(z).scatter_add_(1, at, d).to(st["logits"].dtype)


def _plain_matvec(st):
    y = st["x"].float() @ _dequant(st["w"])[0].t()
    return (_swiglu(y) if st["case"]["act"] == "swiglu" else y).to(torch.bfloat16)


def _plain_experts(st):
    ids, E = st["row_expert"], st["case"]["experts"]
    x = st["x"][:ids.numel()].float()
    if ids.numel() <= E:      # few rows: each row's own matrix
        y = torch.bmm(_dequant(st["w"], ids), x[:, :, None])[:, :, 0]
    else:                     # rows padded per expert to the fullest one
        first = torch.searchsorted(ids, torch.arange(E, device="cuda"))
        at = torch.arange(ids.numel(), device="cuda") - first[ids]
        padded = torch.zeros((E, st["most"], x.shape[1]), device="cuda")
        padded[ids, at] = x
        y = torch.bmm(padded, _dequant(st["w"]).transpose(1, 2))[ids, at]
    st["y"][:ids.numel()] = (_swiglu(y) if st["case"]["act"] == "swiglu" else y).to(torch.bfloat16)
    return st["y"]


def _plain_layer(st):
    c, x, idx = st["case"], st["x"].float(), st["idx"]
    N, K = idx.shape
    live, at = idx >= 0, idx.clamp(min=0).long()
    wts = torch.where(live, st["wts"], 0.0)
    if N * K <= c["experts"]:     # few pairs: each pair's own matrices
        a = torch.bmm(_dequant(st["up"], at.reshape(-1)), x.repeat_interleave(K, 0)[:, :, None])[:, :, 0]
        y = torch.bmm(_dequant(st["down"], at.reshape(-1)), _swiglu(a)[:, :, None])[:, :, 0]
        return (y.reshape(N, K, -1) * wts[..., None]).sum(1).to(torch.bfloat16)
    # every expert on every token, weighted by the routing
    w = torch.zeros((N, c["experts"]), device="cuda").scatter_add_(1, at, wts)
    a = _swiglu((x @ _dequant(st["up"]).reshape(-1, c["hidden"]).t()).reshape(N, c["experts"], -1))
    y = torch.bmm((a * w[..., None]).transpose(0, 1).contiguous(), _dequant(st["down"]).transpose(1, 2))
    return y.sum(0).to(torch.bfloat16)


# ---- the package's calls ---------------------------------------------------

def _stack(w):
    from combine_get_dispatch_layout_amd import moe
    fmt = dict(bf16=moe.EP_WEIGHT_BF16, mxfp4=moe.EP_WEIGHT_MXFP4, int4=moe.EP_WEIGHT_INT4)[w["fmt"]]
    return moe.Weights(fmt, w["data"], w["scales"], w["zeros"], group=w["group"])


def _own_gate_config(c):
    from combine_get_dispatch_layout_amd import moe
    return moe.GateConfig(c["experts"], c["topk"],
                          scoring=moe.EP_SCORE_SOFTMAX if c["score"] == "softmax" else moe.EP_SCORE_SIGMOID,
                          renormalize=c["renorm"], num_groups=c["groups"], topk_groups=c["topk_groups"],
                          group_top=c["group_top"], group_limit=c["group_limit"], scale=c["scale"])


def _own_setup(st):
    """What a program keeps between calls: descriptors, handle, workspace."""
    from combine_get_dispatch_layout_amd import ep, moe
    c = st["case"]
    kept = st["kept"] = {}
    if c["op"] in ("gate", "gate_grad"):
        kept["cfg"] = _own_gate_config(c)
    elif c["op"] == "matvec":
        kept["w"] = _stack(st["w"])
        kept["act"] = moe.EP_ACT_SWIGLU if c["act"] == "swiglu" else moe.EP_ACT_NONE
    else:
        hidden = c["hidden"] if c["op"] == "layer" else c["cols"]
        cfg = ep.Config(hidden=hidden, num_topk=c["topk"], num_experts=c["experts"], num_ranks=1)
        kept["h"] = ep.ep_handle_init(cfg, c["tokens"])
        if c["op"] == "layer":
            kept["up"], kept["down"] = _stack(st["up"]), _stack(st["down"])
            size = moe.ep_moe_workspace_size(kept["h"], kept["up"], kept["down"], c["tokens"])
            kept["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        else:
            kept["w"] = _stack(st["w"])
            kept["act"] = moe.EP_ACT_SWIGLU if c["act"] == "swiglu" else moe.EP_ACT_NONE
            ep.ep_get_layout(kept["h"], st["idx"], alloc_outputs=False)
    return kept


def _own_run(st):
    from combine_get_dispatch_layout_amd import moe
    op = st["case"]["op"]
    k = st.get("kept") or _own_setup(st)
    if op == "gate":
        return moe.ep_gate(k["cfg"], st["logits"], st["bias"], st["mask"])
    if op == "gate_grad":
        return moe.ep_gate_backward(k["cfg"], st["logits"], st["idx"], st["grad"])
    if op == "matvec":
        return moe.ep_matvec(k["w"], st["x"], activation=k["act"])
    if op == "experts":
        return moe.ep_expert_matvec(k["h"], k["w"], st["x"], st["y"], activation=k["act"])
    return moe.ep_moe_layer(k["h"], k["up"], k["down"], st["x"], st["idx"], st["wts"], workspace=k["ws"])


def run(state):
    if own:
        return _own_run(state)
    return dict(gate=_plain_gate, gate_grad=_plain_gate_grad, matvec=_plain_matvec, experts=_plain_experts,
                layer=_plain_layer)[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------

def _weight_bytes(experts, rows, cols, fmt, group, zeros):
    if fmt == "bf16":
        return 2.0 * experts * rows * cols
    per = {"mxfp4": 1.0, "int4": 3.0 if zeros else 2.0}[fmt] / group
    return experts * rows * cols * (0.5 + per)


def work(case):
    c = case
    if c["op"] in ("gate", "gate_grad"):
        N, E, K = c["tokens"], c["experts"], c["topk"]
        size = 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "gate":
            return dict(bytes=N * (E * size + 8 * K) + (4 * E if c["bias"] else 0), flops=8.0 * N * E)
        return dict(bytes=N * (E * size * 2 + 8 * K), flops=8.0 * N * E)
    kind = (c["fmt"], c["group"], c["zeros"])
    if c["op"] == "matvec":
        out = _out_rows(c)
        return dict(bytes=_weight_bytes(1, c["rows"], c["cols"], *kind) + 2.0 * c["tokens"] * (c["cols"] + out),
                    flops=2.0 * c["tokens"] * c["rows"] * c["cols"])
    live = 1 - c["masked"]
    used = c["experts"] * (1 - (1 - live * c["topk"] / c["experts"]) ** c["tokens"])   # expected experts with a row
    pairs = c["tokens"] * c["topk"] * live
    if c["op"] == "experts":
        out = _out_rows(c)
        return dict(bytes=_weight_bytes(used, c["rows"], c["cols"], *kind) + 2.0 * pairs * (c["cols"] + out),
                    flops=2.0 * pairs * c["rows"] * c["cols"])
    return dict(bytes=_weight_bytes(used, 3 * c["inter"], c["hidden"], *kind) + 4.0 * c["tokens"] * c["hidden"]
                + 8.0 * c["tokens"] * c["topk"], flops=6.0 * pairs * c["inter"] * c["hidden"])


# ---- 64 bits, apart from the plain form ------------------------------------

def _expert64(w, e):
    """Expert e's matrix in 64 bits, from the storage formats' definitions."""
    if w["fmt"] == "bf16":
        return w["data"][e].to(torch.float64)
    b = w["data"][e]
    m = torch.empty((b.shape[0], 2 * b.shape[1]), dtype=torch.float64, device=b.device)
    for half, nib in ((0, b.bitwise_and(15)), (1, b.bitwise_right_shift(4))):
        if w["fmt"] == "int4":
            m[:, half::2] = nib.double()
        else:       # sign, two exponent bits, one mantissa bit
            ex, man = ((nib >> 1) & 3).double(), (nib & 1).double()
            mag = torch.where(ex == 0, man / 2, torch.ldexp(1 + man / 2, ex - 1))
            m[:, half::2] = torch.where(nib >= 8, -mag, mag)
    G = w["group"]
    rep = lambda t: t[e].double().repeat_interleave(G, 1)  # noqa: E731
    if w["fmt"] == "mxfp4":
        return torch.ldexp(m, rep(w["scales"]) - 127)
    return (m - (8 if w["zeros"] is None else rep(w["zeros"]))) * rep(w["scales"])


def _act64(v):
    n = v.shape[-1] // 2
    return v[..., :n] / (1 + torch.exp(-v[..., :n])) * v[..., n:]


def _exact_gate(st):
    c = st["case"]
    z = st["logits"].double().cpu().numpy()
    N, E = z.shape
    bias = np.zeros(E) if st["bias"] is None else st["bias"].double().cpu().numpy()
    mask = np.ones(N, bool) if st["mask"] is None else st["mask"].cpu().numpy()
    e = np.exp(z - z.max(1, keepdims=True))
    s = e / e.sum(1, keepdims=True) if c["score"] == "softmax" else 1 / (1 + np.exp(-z))
    out = np.zeros((N, c["topk"]))
    ids = np.arange(E)
    for t in range(N):
        if not mask[t]:
            continue
        pref = s[t] + bias
        order = np.lexsort((ids, -z[t] if st["bias"] is None else -pref))
        if c["groups"]:
            per = E // c["groups"]
            rank = np.sort(pref.reshape(c["groups"], per), 1)[:, ::-1][:, :c["group_top"]].sum(1)
            good = set(np.lexsort((np.arange(c["groups"]), -rank))[:c["topk_groups"]].tolist())
            taken, left = {g: 0 for g in good}, []
            for i in order:
                g = int(i) // per
                if g in good and not (c["group_limit"] and taken[g] == c["group_top"]):
                    taken[g] += 1
                    left.append(int(i))
            order = np.array(left)
        w = s[t, order[:c["topk"]]]
        out[t] = c["scale"] * (w / w.sum() if c["renorm"] else w)
    return None, torch.from_numpy(out)


def _exact_gate_grad(st):
    c = st["case"]
    z, g = st["logits"].double().cpu().numpy(), st["grad"].double().cpu().numpy()
    idx = st["idx"].cpu().numpy()
    N, K = idx.shape
    out = np.zeros_like(z)
    row = np.arange(N)[:, None]
    ok = idx >= 0
    zc = np.where(ok, z[row, idx], -np.inf)
    zc[~ok.any(1)] = 0.0
    g = np.where(ok, g, 0.0) * c["scale"]
    # weights as a function f of the chosen scores; d f / d z by the chain rule
    if c["score"] == "softmax":
        e = np.exp(zc - zc.max(1, keepdims=True))
        if c["renorm"]:
            w = e / e.sum(1, keepdims=True)
        else:
            full = np.exp(z - z.max(1, keepdims=True))
            full /= full.sum(1, keepdims=True)
            w = np.where(ok, full[row, idx], 0.0)
            out -= full * (w * g).sum(1, keepdims=True)
            np.add.at(out, (np.broadcast_to(row, idx.shape)[ok], idx[ok]), (w * g)[ok])
            return torch.from_numpy(out)
        d = w * g - w * (w * g).sum(1, keepdims=True)
    else:
        s = np.where(ok, 1 / (1 + np.exp(-np.where(ok, zc, 0.0))), 0.0)
        d = g
        if c["renorm"]:
            total = np.maximum(s.sum(1, keepdims=True), 1e-300)
            d = g / total - (g * s).sum(1, keepdims=True) / total ** 2
        d = d * s * (1 - s)
    np.add.at(out, (np.broadcast_to(row, idx.shape)[ok], idx[ok]), d[ok])
    return torch.from_numpy(out)


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "gate":
        return _exact_gate(st)
    if c["op"] == "gate_grad":
        return _exact_gate_grad(st)
    x = st["x"].to(torch.float64)
    if c["op"] == "matvec":
        y = torch.mm(_expert64(st["w"], 0), x.t().contiguous()).t()
        return _act64(y) if c["act"] == "swiglu" else y
    if c["op"] == "experts":
        out = x.new_zeros((x.shape[0], _out_rows(c)))
        at = 0
        for e, n in enumerate(torch.bincount(st["row_expert"], minlength=c["experts"]).tolist()):
            if n:
                y = torch.mm(x[at:at + n], _expert64(st["w"], e).t().contiguous())
                out[at:at + n] = _act64(y) if c["act"] == "swiglu" else y
                at += n
        return out
    out = torch.zeros_like(x)
    idx, wts = st["idx"], st["wts"].double()
    for e in range(c["experts"]):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            a = _act64(torch.mm(x[t], _expert64(st["up"], e).t().contiguous()))
            out.index_add_(0, t, wts[t, k][:, None] * torch.mm(a, _expert64(st["down"], e).t().contiguous()))
    return out
