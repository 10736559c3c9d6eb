"""Plain 64-bit definitions of the balance loss and its gradient
(include/ep_moe.h), for the tests, and the error bounds their outputs are held
to.

In units u = 2^-24, the relative errors of an fp32 evaluation are
  a softmax score exp(a) / sum: |a| for the rounding of a, a difference of
    logits; 4 for the exponential, 24 for the sum's additions (at most 16 in a
    lane and 6 across lanes), 4 for the reciprocal and the product: |a| + 32;
  sigmoid and 1 - sigmoid: 4 for the exponential, 1 for the sum, 3 for the
    reciprocal and a product: 8;  normalised: 32 more, and |a| where a token's
    logits are all below -64 and the scores come from differences;
  scores below 2^-126, the smallest normal fp32, may be 0: TINY for the few
    additions and factors (below 64 each) that such a score meets here;
  a sum of scores over tokens: at most 64 additions in a lane, 2 across lanes, 2
    across waves: 70; the rest is in 64 bits.
"""
import numpy as np

U, TINY = 2.0 ** -24, 64 * 64 * 2.0 ** -126
FMAX = float(np.finfo(np.float32).max)


def clean(z):
    """NaN and -inf: -inf (no score); +inf: the largest float."""
    return np.where(np.isnan(z), -np.inf, np.minimum(z.astype(np.float64), FMAX))


def scores(z, score, normalize):
    """(p, 1 - s of a sigmoid, relative error of p in u), float64 [N, E]."""
    z = clean(z)
    ok = z > -np.inf
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        top = np.where(ok.any(1), z.max(1), 0.0)[:, None]
        if score == "softmax":
            e = np.where(ok, np.exp(z - top), 0.0)
            total = e.sum(1, keepdims=True)
            return e / np.where(total > 0, total, 1), np.ones_like(z), \
                np.where(ok, np.minimum(np.abs(z - top), 200), 0) + 32
        s = np.where(ok, 1 / (1 + np.exp(-z)), 0.0)
        rest = np.where(ok, 1 / (1 + np.exp(z)), 1.0)
        if not normalize:
            return s, rest, np.full(z.shape, 8.0)
        # in proportion to e^(z - top): the same for any common factor
        s = np.where(top < -64, np.where(ok, np.exp(z - top) * rest, 0.0), s)
        total = s.sum(1, keepdims=True)
        far = np.where(ok & (top < -64), np.minimum(np.abs(z - top), 200), 0)
        return s / np.where(total > 0, total, 1), rest, 40 + far


def spans(start, N):
    if start is None:
        return [(0, N)]
    b = np.clip(np.asarray(start, np.int64), 0, N)
    return [(int(a), int(max(a, c))) for a, c in zip(b[:-1], b[1:])]


def tokens_of(start, mask, N):
    live = np.ones(N, bool) if mask is None else np.asarray(mask, bool)
    return [np.arange(a, b)[live[a:b]] for a, b in spans(start, N)]


def counts(idx, E, start=None, mask=None):
    out = [np.bincount(i[(i >= 0) & (i < E)], minlength=E)
           for i in (idx[t].reshape(-1) for t in tokens_of(start, mask, idx.shape[0]))]
    return np.stack(out).astype(np.int64)


def balance(z, idx, score="softmax", normalize=True, coefficient=1.0, start=None, mask=None):
    """loss, counts, seq_tokens, score_sums and the bounds of the first and last."""
    N, E = z.shape
    K = idx.shape[1]
    p, _, rel = scores(z, score, normalize)
    n, groups = counts(idx, E, start, mask), tokens_of(start, mask, N)
    T = np.array([len(t) for t in groups])
    S = np.stack([p[t].sum(0) for t in groups])
    eS = np.stack([(p[t] * (rel[t] + 70) * U).sum(0) for t in groups])
    f = coefficient / len(groups) * E / (K * np.maximum(T, 1.0) ** 2)
    loss, eloss = (f * (n * S).sum(1)).sum(), (abs(f) * (n * eS).sum(1)).sum()
    return loss, n, T, S, eloss + U * (abs(loss) + eloss) + TINY, eS + U * (S + eS) + TINY


def gradient(z, n, T, K, score="softmax", normalize=True, coefficient=1.0, g=1.0, start=None, mask=None,
             out_half=U):
    """d (g * loss) / d z for the given counts and tokens, and its bound."""
    N, E = z.shape
    p, rest, rel = scores(z, score, normalize)
    out, err = np.zeros((N, E)), np.zeros((N, E))
    Q = len(T)
    divide = score == "softmax" or normalize
    for q, t in enumerate(tokens_of(start, mask, N)):
        if T[q] <= 0 or not len(t):
            continue
        scale = g * coefficient / Q * E / (K * float(T[q]) ** 2)
        # a constant in f has no effect where scores sum to one
        f = (n[q] - (K * int(T[q]) // E if divide else 0)).astype(np.float64)
        dot = (p[t] @ f)[:, None] if divide else 0.0
        ps = p[t].sum(1, keepdims=True)
        if divide:      # rows without a score have no gradient; else sum p = 1
            assert ((np.abs(ps - 1) < 1e-9) | (ps == 0)).all()
        edot = ((p[t] * (rel[t] + 24) * U) @ np.abs(f))[:, None] if divide else 0.0
        w = p[t] * abs(scale) * (rest[t] if score == "sigmoid" else 1.0)
        out[t] = np.sign(scale) * w * (f - dot)
        err[t] = w * (edot + U * (np.abs(f) + np.abs(dot))) + np.abs(out[t]) * (rel[t] + 16) * U
    return out, err + out_half * (np.abs(out) + err) + TINY
