"""Plain 64-bit definitions of the router, the products with expert weights
and the whole expert layer (include/ep_moe.h), for the tests, and the error
bounds their outputs are held to.

Rounding: a value stored in a type is off by at most half a step, eps / 2 of
its magnitude (bf16 2^-8).  A sum of n terms in fp32 is off by at most
n * 2^-24 * sum |terms|, in any order.
"""
import numpy as np
import torch

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


# ---- weights ---------------------------------------------------------------

def make_weights(fmt, E, M, C, group=0, zeros=False, seed=0):
    """Tensors of a stack in the format, on the CPU: (data, scales, zeros)."""
    g = torch.Generator().manual_seed(seed)
    if fmt == "bf16":
        return (torch.randn((E, M, C), generator=g) * C ** -0.5).to(torch.bfloat16), None, None
    data = torch.randint(0, 256, (E, M, C // 2), dtype=torch.uint8, generator=g)
    if fmt == "mxfp4":
        return data, torch.randint(118, 124, (E, M, C // 32), dtype=torch.uint8, generator=g), None
    s = ((0.5 + torch.rand((E, M, C // group), generator=g)) * 0.2 * C ** -0.5).to(torch.bfloat16)
    s[torch.rand(s.shape, generator=g) < 0.1] *= -1
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, generator=g) if zeros else None
    return data, s, z


def dequant(fmt, data, scales, zeros, group):
    """float64 [E, M, C], and the magnitudes that the products' sums run over
    (for INT4 the offset codes |128 + q| + |128 + zero| times the scale)."""
    if fmt == "bf16":
        w = data.double().numpy()
        return w, np.abs(w)
    b = data.numpy()
    q = np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], 2 * b.shape[-1])
    if fmt == "mxfp4":
        s = np.ldexp(1.0, scales.numpy().astype(np.int64) - 127)
        w = E2M1[q] * np.repeat(s, 32, axis=-1)
        return w, np.abs(w)
    s = np.repeat(scales.double().numpy(), group, axis=-1)
    z = 8.0 if zeros is None else np.repeat(zeros.double().numpy(), group, axis=-1)
    return (q - z) * s, (256.0 + q + z) * np.abs(s)


def terms(C, group):
    """Additions that a column sum goes through: inside a group (codes and
    offsets), then over the groups."""
    return 2 * group + C // group + 8 if group else C + 8


# ---- products ----------------------------------------------------------------

def silu(v):
    return v / (1 + np.exp(-v))


def product(x, w, mag, n_terms, act):
    """act(x W^T) in 64 bits and the bound of its fp32 sums' errors."""
    y = x @ w.T
    err = n_terms * F32_HALF * (np.abs(x) @ mag.T)
    if not act:
        return y, err
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    # |silu'| <= 1.1; the exponential and the division are good to 2^-18 for
    # the |g| < 40 of these inputs (an ulp or two of exp2's argument g log2 e)
    out = silu(g) * u
    return out, 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -18 * np.abs(out)


def assert_close(got, want, err, what=""):
    """bf16 results: one rounding of a value within err of want."""
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    tol = err + BF16_HALF * (np.abs(want) + err) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           got[bad][:4], want[bad][:4], tol[bad][:4])
    # and as a whole no worse than every element's rounding at its largest
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= BF16_HALF * norm + 1e-38, (
        what, np.linalg.norm(got - want) / norm)


def layer(x, idx, wts, up, down, n_up, n_down):
    """The whole layer; up, down: (w, mag) per expert.  Returns (out, err)."""
    out, err = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(x.shape[0]):
        for k in range(idx.shape[1]):
            e = idx[t, k]
            if e < 0 or e >= up[0].shape[0]:
                continue
            w = 1.0 if wts is None else float(wts[t, k])
            a, ea = product(x[t:t + 1], up[0][e], up[1][e], n_up, True)
            a, ea = w * a, abs(w) * ea
            y = a @ down[0][e].T
            # a in two bf16 terms: 2^-16 of it is lost
            ey = (ea + 2.0 ** -16 * np.abs(a)) @ np.abs(down[0][e]).T + \
                2 * n_down * F32_HALF * ((np.abs(a) + ea) @ down[1][e].T)
            out[t] += y[0]
            err[t] += ey[0] + idx.shape[1] * F32_HALF * np.abs(y[0])
    return out, err


# ---- router ------------------------------------------------------------------

def gate(logits, K, score="softmax", renorm=True, bias=None, groups=0, topk_groups=0, group_top=0,
         limit=False, scale=1.0, mask=None):
    """(idx, weights) row by row from the definition, float64."""
    N, E = logits.shape
    idx, wts = np.full((N, K), -1, np.int32), np.zeros((N, K))
    fmax = float(np.finfo(np.float32).max)
    for t in range(N):
        if mask is not None and not mask[t]:
            continue
        z = logits[t].astype(np.float64)
        ok = ~np.isnan(z) & (z > -np.inf)
        z = np.where(ok, np.minimum(z, fmax), -np.inf)
        if not ok.any():
            continue
        with np.errstate(over="ignore"):
            s = np.exp(z - z.max()) if score == "softmax" else 1 / (1 + np.exp(-z))
        s = np.where(ok, s, 0.0)
        if score == "softmax":
            s = s / s.sum()
        c = s + (0.0 if bias is None else bias.astype(np.float64))
        ok = ok & ~np.isnan(c) & (c > -np.inf)
        key = z if bias is None else c
        cand = sorted(np.flatnonzero(ok), key=lambda e: (-key[e], e))
        if groups > 1:
            per = E // groups
            best = {g: [e for e in cand if e // per == g][:group_top] for g in range(groups)}
            rank = sorted((g for g in best if best[g]),
                          key=lambda g: (-sum(c[e] for e in best[g]), g))[:topk_groups]
            cand = [e for e in cand if e // per in rank and (not limit or e in best[e // per])]
        cand = cand[:K]
        idx[t, :len(cand)] = cand
        v = s[cand]
        if renorm and len(cand):
            if score == "softmax" or v.sum() == 0:
                v = np.exp(z[cand] - z[cand].max())
            v = v / v.sum()
        wts[t, :len(cand)] = scale * v
    return idx, wts


def gate_weights(logits, idx, score, renorm, scale):
    """Weights of a fixed choice, float64, as a function of the logits."""
    w = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        live = [(k, e) for k, e in enumerate(idx[t]) if 0 <= e < logits.shape[1]]
        if not live:
            continue
        z = logits[t].astype(np.float64)
        s = np.exp(z - z.max()) if score == "softmax" else 1 / (1 + np.exp(-z))
        s = s / s.sum() if score == "softmax" else s
        v = np.array([s[e] for _, e in live])
        w[t, [k for k, _ in live]] = scale * (v / v.sum() if renorm else v)
    return w


def gate_grad(logits, idx, g, score, renorm, scale):
    """Gradient of sum(g * gate_weights) with respect to the logits."""
    out = np.zeros(logits.shape)
    E = logits.shape[1]
    for t in range(idx.shape[0]):
        live = [(k, int(e)) for k, e in enumerate(idx[t]) if 0 <= e < E]
        if not live:
            continue
        z = logits[t].astype(np.float64)
        s = np.exp(z - z.max()) if score == "softmax" else 1 / (1 + np.exp(-z))
        s = s / s.sum() if score == "softmax" else s
        ks, es = [k for k, _ in live], [e for _, e in live]
        gk, v = g[t, ks] * scale, s[es]
        if renorm:      # w = v / sum v: dw/dv
            gk = (gk - (gk * v).sum() / v.sum()) / v.sum()
        ds = np.zeros(E)
        np.add.at(ds, es, gk)
        out[t] = s * (ds - (ds * s).sum()) if score == "softmax" else ds * s * (1 - s)
    return out


def gate_grad_bound(logits, idx, g, score, renorm, scale, out_half):
    """(gate_grad, what an fp32 evaluation and one rounding by out_half may be off
    it), element by element.  In units u = 2^-24, the relative errors are
      a score p = exp(a) / sum: |a| for the rounding of a (softmax: a difference
        of logits; log sigmoid twice that, for its own rounding and the
        difference's), 4 for the exponential, at most 24 for the sum's additions,
        4 for the rest: |a| + 32;
      1 - s: 8;  g * scale: 1;
    sums of g over K entries lose K + 8 units of the magnitudes they run over."""
    u = F32_HALF
    out, err = np.zeros(logits.shape), np.zeros(logits.shape)
    E, K = logits.shape[1], idx.shape[1]
    for t in range(idx.shape[0]):
        ks = [k for k in range(K) if 0 <= idx[t, k] < E]
        if not ks:
            continue
        es = idx[t, ks].astype(int)
        z, gk = logits[t].astype(np.float64), g[t, ks].astype(np.float64) * scale
        if score == "softmax":
            a = z - (z[es] if renorm else z).max()
            rel = (np.abs(a) + 32) * u
        else:
            a = -np.logaddexp(0, -z)
            rel = (2 * (np.abs(a) + np.abs(a[es]).max()) + 32) * u
            if renorm:
                a = a - a[es].max()
        p = np.exp(a)
        if renorm:
            p = p / p[es].sum()
        elif score == "softmax":
            p = p / p.sum()
        dot = (gk * p[es]).sum() if renorm or score == "softmax" else 0.0
        edot = (np.abs(gk) * p[es] * (rel[es] + (K + 9) * u)).sum() if renorm or score == "softmax" else 0.0
        if score == "softmax" and not renorm:
            sg, eg = np.zeros(E), np.zeros(E)
            np.add.at(sg, es, gk)
            np.add.at(eg, es, np.abs(gk) * (K + 9) * u)
            out[t] = p * (sg - dot)
            err[t] = p * (eg + edot) + np.abs(out[t]) * (rel + 4 * u)
        else:
            q = 1 / (1 + np.exp(z[es])) if score == "sigmoid" else np.ones(len(es))
            d = p[es] * q * (gk - dot)
            np.add.at(out[t], es, d)
            np.add.at(err[t], es, p[es] * q * (edot + 2 * u * np.abs(gk)) + np.abs(d) * (rel[es] + (K + 16) * u))
    return out, err + out_half * (np.abs(out) + err) + 1e-38
