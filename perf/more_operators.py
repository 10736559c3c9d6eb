"""Operators beside the router and the int8 dispatch, as measured cases: the
balance loss with its per-expert counts and its gradient, and products in 8-bit
integers with a scale for each token and each weight channel, of one matrix or
of the rows that a dispatch received.

Each case is prepared on the GPU from a seed; `run` makes one pass, in plain
torch operations (own = False) or through the package's calls (own = True);
`exact` gives the same outputs from the definitions in 64 bits.

Balance loss: with V_q the unmasked tokens of sequence q, T_q their number,
count[q,e] the entries of their topk_idx that name expert e and p the scores,
  loss = coefficient / Q * sum_q E / (K T_q^2) * sum_e count[q,e] sum_{t in V_q} p[t,e].
Products: y = act((x W^T) * x_scale[row] * w_scale[channel]).
"""
import math

import torch

own = False


# ---- cases -----------------------------------------------------------------

def _balance(op, tokens, experts, topk, score="softmax", normalize=True, dtype="fp32", sequences=0, masked=0.0,
             coefficient=1e-2):
    """sequences = 0: the whole batch as one, without a table of starts."""
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, score=score, normalize=normalize, dtype=dtype,
                sequences=sequences, masked=masked, coefficient=coefficient)


def _matmul(tokens, cols, rows, act="none"):
    return dict(op="matmul", tokens=tokens, cols=cols, rows=rows, act=act)


def _experts(tokens, experts, topk, cols, rows, act="none", masked=0.0):
    return dict(op="experts", tokens=tokens, experts=experts, topk=topk, cols=cols, rows=rows, act=act, masked=masked)


def listed():
    return [
        # a tiny training step: launch latency
        dict(_balance("balance", 128, 16, 2), name="balance_tiny"),
        # a micro-batch as one sequence, logits in bf16
        dict(_balance("balance", 4096, 128, 8, dtype="bf16"), name="balance_batch"),
        # sequence-wise loss of normalised sigmoid scores over packed, ragged sequences with padding
        dict(_balance("balance", 65536, 256, 8, score="sigmoid", sequences=37, masked=0.1), name="balance_sequences"),
        # its gradients: a micro-batch in bf16, and the packed sequences
        dict(_balance("balance_grad", 4096, 128, 8, dtype="bf16"), name="balance_grad_batch"),
        dict(_balance("balance_grad", 65536, 256, 8, score="sigmoid", sequences=37, masked=0.1),
             name="balance_grad_sequences"),
        # one decoded token through a dense layer
        dict(_matmul(1, 7168, 4096), name="matmul_token"),
        # a ragged handful of sequences through a gated up projection of odd sizes
        dict(_matmul(29, 4112, 2 * 2085, act="swiglu"), name="matmul_few"),
        # a prompt through a dense layer
        dict(_matmul(4096, 7168, 4096), name="matmul_prompt"),
        # the gated up projection of a dispatched decode batch: every expert's weights are read
        dict(_experts(128, 256, 8, 7168, 4096, act="swiglu"), name="experts_decode"),
        # the same of a prompt, some 256 rows an expert
        dict(_experts(4096, 128, 8, 2048, 2 * 768, act="swiglu"), name="experts_prompt"),
        # a ragged batch of some 47 rows an expert, masked entries
        dict(_experts(1000, 128, 6, 4096, 1408, masked=0.05), name="experts_ragged"),
        # the down projection of a long prompt, some 770 rows an expert
        dict(_experts(8192, 64, 6, 1536, 4096), name="experts_long"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "matmul", "matmul", "experts", "experts"])
    if op in ("balance", "balance_grad"):
        experts = rng.choice([8, 16, 33, 64, 100, 128, 256, 256])
        tokens = _log(rng, 1, 65536)
        return _balance(op, tokens, experts, rng.randint(1, 8), rng.choice(["softmax", "sigmoid"]),
                        rng.random() < 0.7, rng.choice(["fp32", "bf16"]),
                        rng.choice([0, 0, 1, _log(rng, 1, min(64, tokens))]), rng.choice([0.0, 0.0, 0.1, 0.5]),
                        rng.choice([1e-3, 1e-2]))
    act = rng.choice(["none", "swiglu"])
    cols = 16 * _log(rng, 16, 7168 // 16)
    if op == "matmul":
        rows = _log(rng, 65, 4096)
        return _matmul(_log(rng, 1, 4096), cols, 2 * rows if act == "swiglu" else rows, act)
    experts = rng.choice([8, 16, 33, 64, 128])
    topk = rng.randint(1, min(8, experts))
    cols, rows = min(cols, 4096), _log(rng, 65, 2048)
    rows = 2 * rows if act == "swiglu" else rows
    # no more products than the largest listed case has
    most = max(1, int(8192 * 6 * 1536 * 4096 / (topk * cols * rows)))
    return _experts(_log(rng, 1, min(8192, most)), experts, topk, cols, rows, act, rng.choice([0.0, 0.0, 0.05]))


# ---- inputs ----------------------------------------------------------------

def _weights(gen, experts, rows, cols):
    """Codes with a normal spread, four deviations to 127, and channel scales
    that bring the values near 1/sqrt(cols)."""
    codes = torch.empty((experts, rows, cols), dtype=torch.int8, device="cuda")
    for e in range(experts):
        v = torch.randn((rows, cols), device="cuda", generator=gen)
        codes[e] = v.mul_(127 / 4).round_().clamp_(-127, 127).to(torch.int8)
    scales = (0.5 + torch.rand((experts, rows), device="cuda", generator=gen)) * (cols ** -0.5 * 4 / 127)
    return dict(codes=codes, scales=scales)


def _tokens(gen, rows, cols):
    """Rows of different magnitude in int8, as a dispatch quantises them."""
    x = torch.randn((rows, cols), device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn((rows, 1), device="cuda", generator=gen))
    scales = x.abs().amax(1, keepdim=True).clamp_(min=1e-4) / 127
    return (x / scales).round_().clamp_(-127, 127).to(torch.int8), scales


def _out_rows(c):
    return c["rows"] // 2 if c["act"] == "swiglu" else c["rows"]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=c)
    if c["op"] in ("balance", "balance_grad"):
        N, E, K, Q = c["tokens"], c["experts"], c["topk"], c["sequences"]
        # popular experts, as an unbalanced router has
        logits = torch.randn((N, E), device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)
        st["logits"] = logits.to(torch.bfloat16) if c["dtype"] == "bf16" else logits
        st["idx"] = st["logits"].float().topk(K, dim=1).indices.to(torch.int32)
        st["mask"] = torch.rand(N, device="cuda", generator=gen) >= c["masked"] if c["masked"] else None
        if st["mask"] is not None:
            st["idx"][~st["mask"]] = -1
        st["start"] = None
        if Q:
            # cuts at random places: ragged lengths, some of them small or none; the last tokens belong to no sequence
            cuts = torch.rand(Q, device="cuda", generator=gen).sort().values
            cuts = (cuts / cuts[-1] * (N - N // 64)).to(torch.int32)
            st["start"] = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), cuts))
        if c["op"] == "balance_grad":
            # what the forward call left, and the gradient of the loss in a scaled step
            st["counts"], st["seq_tokens"] = _plain_counts(st)
            st["grad"] = 1 + torch.rand((), device="cuda", generator=gen)
        return st
    if c["op"] == "matmul":
        st["w"] = _weights(gen, 1, c["rows"], c["cols"])
        st["x"], st["x_scales"] = _tokens(gen, c["tokens"], c["cols"])
        return st
    # a dispatched batch: rows grouped by expert, (token, k) order inside
    N, E, K = c["tokens"], c["experts"], c["topk"]
    st["w"] = _weights(gen, E, c["rows"], c["cols"])
    st["idx"] = torch.rand((N, E), device="cuda", generator=gen).topk(K, dim=1).indices.to(torch.int32)
    if c["masked"]:
        st["idx"][torch.rand((N, K), device="cuda", generator=gen) < c["masked"]] = -1
    ids = st["idx"].reshape(-1)
    ids = ids[ids >= 0].sort(stable=True).values.long()
    st["row_expert"] = ids
    st["most"] = int(torch.bincount(ids, minlength=E).max()) if ids.numel() else 0
    # the receive buffer is sized for every entry; masked ones leave rows at its end unused
    st["x"], st["x_scales"] = _tokens(gen, N * K, c["cols"])
    st["y"] = torch.zeros((N * K, _out_rows(c)), dtype=torch.bfloat16, device="cuda")
    return st


# ---- plain form ------------------------------------------------------------

def _sequence_of(st):
    """Each token's sequence (Q for those behind the last, or masked)."""
    N, start, mask = st["logits"].shape[0], st["start"], st["mask"]
    Q = 1 if start is None else start.numel() - 1
    seq = torch.zeros(N, dtype=torch.long, device="cuda")
    if start is not None:
        seq = torch.searchsorted(start[1:].long(), torch.arange(N, device="cuda"), right=True)
    return (seq if mask is None else torch.where(mask, seq, Q)), Q


def _per_sequence(st, rows):
    """Sums of rows [N, E] over the tokens of each sequence, in 64 bits."""
    rows = rows.double()
    if st["mask"] is not None:
        rows = rows * st["mask"][:, None]
    if st["start"] is None:
        return rows.sum(0, keepdim=True)
    rows = rows.t().contiguous()
    upto = torch.cat((torch.zeros_like(rows[:, :1]), rows.cumsum(1)), dim=1)[:, st["start"].long()]
    return (upto[:, 1:] - upto[:, :-1]).t()


def _plain_counts(st):
    N, E = st["logits"].shape
    hit = torch.zeros((N, E + 1), device="cuda")
    idx = torch.where(st["idx"] >= 0, st["idx"], E).long()
    hit.scatter_add_(1, idx, torch.ones_like(idx, dtype=torch.float32))
    hit[:, E] = 1       # the token itself
    both = _per_sequence(st, hit).to(torch.int32)
    return both[:, :E].contiguous(), both[:, E].contiguous()


def _plain_scores(st):
    c, z = st["case"], st["logits"].float()
    if c["score"] == "softmax":
        return torch.softmax(z, 1)
    s = torch.sigmoid(z)
    return s / s.sum(1, keepdim=True) if c["normalize"] else s


def _plain_balance(st):
    c = st["case"]
    E, K = c["experts"], c["topk"]
    counts, tokens = _plain_counts(st)
    sums = _per_sequence(st, _plain_scores(st))
    per = (counts.double() * sums).sum(1) / tokens.clamp(min=1).double() ** 2
    loss = per.mean() * (c["coefficient"] * E / K)
    return loss.float(), counts, tokens, sums.float()


def _plain_balance_grad(st):
    c = st["case"]
    E, K = c["experts"], c["topk"]
    seq, Q = _sequence_of(st)
    T = st["seq_tokens"].clamp(min=1).float()[:, None]
    # counts less their mean: a constant changes no gradient of scores that sum to one
    f = st["counts"].float()
    if c["score"] == "softmax" or c["normalize"]:
        f = f - f.mean(1, keepdim=True)
    f = f / (T * T) * (c["coefficient"] / Q * E / K) * st["grad"]
    f = torch.cat((f, torch.zeros_like(f[:1])))[seq]
    p = _plain_scores(st)
    if c["score"] == "softmax":
        g = p * (f - (p * f).sum(1, keepdim=True))
    else:
        s = torch.sigmoid(st["logits"].float())
        g = p * (1 - s) * (f - (p * f).sum(1, keepdim=True) if c["normalize"] else f)
    g = torch.where((seq < Q)[:, None], g, 0.0)
    return g.to(st["logits"].dtype)


def _finish(y, x_scales, w_scales, act):
    """Scales and activation on sums [.., rows]."""
    y = y * x_scales * w_scales
    if act == "swiglu":
        g, u = y.chunk(2, dim=-1)
        y = g * torch.sigmoid(g) * u
    return y


def _plain_matmul(st):
    y = st["x"].float() @ st["w"]["codes"][0].float().t()
    return _finish(y, st["x_scales"], st["w"]["scales"], st["case"]["act"]).to(torch.bfloat16)


def _plain_experts(st):
    ids, E, act = st["row_expert"], st["case"]["experts"], st["case"]["act"]
    w, scales = st["w"]["codes"], st["w"]["scales"]
    x = st["x"][:ids.numel()].float()
    if ids.numel() <= E:      # few rows: each row's own matrix
        y = torch.bmm(w[ids].float(), x[:, :, None])[:, :, 0]
    else:                     # rows padded per expert to the fullest one
        first = torch.searchsorted(ids, torch.arange(E, device="cuda"))
        at = torch.arange(ids.numel(), device="cuda") - first[ids]
        padded = torch.zeros((E, st["most"], x.shape[1]), device="cuda")
        padded[ids, at] = x
        y = torch.bmm(padded, w.float().transpose(1, 2))[ids, at]
    st["y"][:ids.numel()] = _finish(y, st["x_scales"][:ids.numel()], scales[ids], act).to(torch.bfloat16)
    return st["y"]


# ---- the package's calls ---------------------------------------------------

def _own_setup(st):
    """What a program keeps between calls: descriptors, handle, workspace."""
    from combine_get_dispatch_layout_amd import ep, moe
    c = st["case"]
    kept = st["kept"] = {}
    if c["op"] in ("balance", "balance_grad"):
        kept["cfg"] = moe.BalanceConfig(
            c["experts"], c["topk"],
            scoring=moe.EP_SCORE_SOFTMAX if c["score"] == "softmax" else moe.EP_SCORE_SIGMOID,
            normalize=c["normalize"], coefficient=c["coefficient"])
        if c["op"] == "balance":
            size = moe.ep_balance_workspace_size(kept["cfg"], c["tokens"], max(1, c["sequences"]))
            kept["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return kept
    kept["w"] = moe.Weights(moe.EP_WEIGHT_INT8, st["w"]["codes"], st["w"]["scales"])
    kept["act"] = moe.EP_ACT_SWIGLU if c["act"] == "swiglu" else moe.EP_ACT_NONE
    if c["op"] == "experts":
        cfg = ep.Config(hidden=c["cols"], num_topk=c["topk"], num_experts=c["experts"], num_ranks=1,
                        quant=ep.EP_QUANT_INT8, quant_group=c["cols"])
        kept["h"] = ep.ep_handle_init(cfg, c["tokens"])
        ep.ep_get_layout(kept["h"], st["idx"], alloc_outputs=False)
    return kept


def _own_run(st):
    from combine_get_dispatch_layout_amd import moe
    op = st["case"]["op"]
    k = st.get("kept") or _own_setup(st)
    if op == "balance":
        return tuple(moe.ep_balance_loss(k["cfg"], st["logits"], st["idx"], st["mask"], st["start"],
                                         workspace=k["ws"]))
    if op == "balance_grad":
        return moe.ep_balance_loss_backward(k["cfg"], st["logits"], st["counts"], st["seq_tokens"], st["grad"],
                                            st["mask"], st["start"])
    if op == "matmul":
        return moe.ep_matmul(k["w"], st["x"], st["x_scales"], activation=k["act"])
    return moe.ep_expert_matmul(k["h"], k["w"], st["x"], st["x_scales"], st["y"], activation=k["act"])


def run(state):
    if own:
        return _own_run(state)
    return dict(balance=_plain_balance, balance_grad=_plain_balance_grad, matmul=_plain_matmul,
                experts=_plain_experts)[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c = case
    if c["op"] in ("balance", "balance_grad"):
        N, E, K, Q = c["tokens"], c["experts"], c["topk"], max(1, c["sequences"])
        size = 2 if c["dtype"] == "bf16" else 4
        mask = N if c["masked"] else 0
        if c["op"] == "balance":
            return dict(bytes=N * (E * size + 4 * K) + mask + 8 * Q * E, flops=8.0 * N * E)
        return dict(bytes=2.0 * N * E * size + mask + 4 * Q * E, flops=12.0 * N * E)
    out = _out_rows(c)
    if c["op"] == "matmul":
        return dict(bytes=float(c["rows"] * (c["cols"] + 4) + c["tokens"] * (c["cols"] + 4 + 2 * out)),
                    flops=2.0 * c["tokens"] * c["rows"] * c["cols"])
    live = 1 - c["masked"]
    used = c["experts"] * (1 - (1 - live * c["topk"] / c["experts"]) ** c["tokens"])   # expected experts with a row
    pairs = c["tokens"] * c["topk"] * live
    return dict(bytes=used * c["rows"] * (c["cols"] + 4.0) + pairs * (c["cols"] + 4 + 2 * out),
                flops=2.0 * pairs * c["rows"] * c["cols"])


# ---- 64 bits, apart from the plain form ------------------------------------

def _scores64(c, z):
    """Scores, and d score / d (its own logit) for the unnormalised sigmoid."""
    if c["score"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), None
    s = 1 / (1 + torch.exp(-z))
    return s, s / (1 + torch.exp(z))


def _spans(st):
    """(first, behind the last) token of each sequence."""
    if st["start"] is None:
        return [(0, st["logits"].shape[0])]
    b = st["start"].tolist()
    return list(zip(b[:-1], b[1:]))


def _live64(st, a, b):
    live = torch.arange(a, b, device="cuda")
    return live if st["mask"] is None else live[st["mask"][a:b]]


def _exact_balance(st):
    c = st["case"]
    E, K = c["experts"], c["topk"]
    spans = _spans(st)
    loss, sums = 0.0, []
    for a, b in spans:
        live = _live64(st, a, b)
        p, _ = _scores64(c, st["logits"][live].double())
        if c["score"] != "softmax" and c["normalize"]:
            p = p / p.sum(1, keepdim=True)
        ids = st["idx"][live].reshape(-1)
        n = torch.bincount(ids[ids >= 0].long(), minlength=E).double()
        mean = p.mean(0) if live.numel() else torch.zeros_like(n)
        loss += float((E / (K * max(1, live.numel())) * n * mean).sum())
        sums.append(p.sum(0))
    return torch.tensor(c["coefficient"] * loss / len(spans), dtype=torch.float64), None, None, torch.stack(sums)


def _exact_balance_grad(st):
    c = st["case"]
    E, K = c["experts"], c["topk"]
    spans = _spans(st)
    out = torch.zeros(st["logits"].shape, dtype=torch.float64, device="cuda")
    for a, b in spans:
        live = _live64(st, a, b)
        if not live.numel():
            continue
        ids = st["idx"][live].reshape(-1)
        n = torch.bincount(ids[ids >= 0].long(), minlength=E).double()
        # d loss / d score, the same for every token of the sequence
        d = float(st["grad"]) * c["coefficient"] / len(spans) * E / (K * live.numel()) * n / live.numel()
        s, own_slope = _scores64(c, st["logits"][live].double())
        if c["score"] == "softmax":
            out[live] = s * (d - (s @ d)[:, None])
        elif c["normalize"]:
            total = s.sum(1, keepdim=True)
            out[live] = own_slope * (d / total - (s @ d)[:, None] / total ** 2)
        else:
            out[live] = own_slope * d
    return out


def _act64(v, act):
    if act == "none":
        return v
    n = v.shape[-1] // 2
    return v[..., :n] / (1 + torch.exp(-v[..., :n])) * v[..., n:]


def _product64(x, x_scales, codes, scales):
    y = torch.mm(x.double(), codes.double().t().contiguous())
    return y * x_scales.double() * scales.double()


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "balance":
        return _exact_balance(st)
    if c["op"] == "balance_grad":
        return _exact_balance_grad(st)
    codes, scales = st["w"]["codes"], st["w"]["scales"]
    if c["op"] == "matmul":
        return _act64(_product64(st["x"], st["x_scales"], codes[0], scales[0]), c["act"])
    out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for e, n in enumerate(torch.bincount(st["row_expert"], minlength=c["experts"]).tolist()):
        if n:
            y = _product64(st["x"][at:at + n], st["x_scales"][at:at + n], codes[e], scales[e])
            out[at:at + n] = _act64(y, c["act"])
            at += n
    return out
