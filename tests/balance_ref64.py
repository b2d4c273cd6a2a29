"""The balance loss, the experts' counts and the gradient in 64 bits, sequence by sequence, with bounds of the kernels'
fp32 error.

U = 2^-24.  A probability: the exponent's difference, and its product with 1 / ln 2, are off by at most U |l - m| each
(|l - m| <= 20 in the tests, smaller probabilities weigh nothing), the exponential and the reciprocal by 2 U each, its
sum of E <= 256 positive terms by 24 U (sixteen a lane, then four steps) beside its terms' own 42 U, weighted by p: 128 U
of p in all.  A sum over tokens of positive terms adds U for each step of its order: at
most T / 32 + 300.  log and the logsumexp: 66 U from the sum, and 3 U |lse| from its own roundings.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def scores(l, score):
    """(p, lse, 1 - s) of logits in 64 bits; -inf is a masked expert."""
    masked = l == -np.inf
    if score == "softmax":
        m = l.max(1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        with np.errstate(invalid="ignore"):
            e = np.where(masked, 0.0, np.exp(l - m))
        total = e.sum(1, keepdims=True)
        none = total[:, 0] == 0.0
        with np.errstate(invalid="ignore", divide="ignore"):
            p = np.where(masked, 0.0, e / total)
            lse = np.where(none, 0.0, m[:, 0] + np.log(total[:, 0]))
        return p, lse, np.ones_like(p)
    with np.errstate(over="ignore"):
        s = np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-l)))
        return np.where(masked, 0.0, s / (s.sum(1, keepdims=True) + 1e-20)), np.zeros(len(l)), 1.0 / (1.0 + np.exp(l))


def sequences(T, offsets, mask):
    """The live tokens of every sequence."""
    live = np.ones(T, bool) if mask is None else mask.astype(bool)
    offsets = [0, T] if offsets is None else list(offsets)
    return [np.flatnonzero(live[a:b]) + a for a, b in zip(offsets[:-1], offsets[1:])]


def balance(l, idx, score, offsets=None, mask=None):
    """(dict of the results, dict of their error bounds)"""
    l = l.astype(np.float64)
    (T, E), k = l.shape, idx.shape[1]
    rows = sequences(T, offsets, mask)
    S = len(rows)
    r = dict(loss=np.zeros(S), z=np.zeros(S), prob=np.zeros((S, E)), counts=np.zeros((S, E), np.int32),
             tokens=np.zeros(S, np.int32))
    b = dict(loss=np.zeros(S), z=np.zeros(S), prob=np.zeros((S, E)))
    steps = (T / 32 + 300 + 128) * U
    for s, at in enumerate(rows):
        n = len(at)
        if not n:
            continue
        p, lse, _ = scores(l[at], score)
        i = idx[at].ravel()
        r["counts"][s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        r["tokens"][s], r["prob"][s] = n, p.mean(0)
        r["loss"][s] = E / (k * n) * np.sum(np.where(r["counts"][s] > 0, r["counts"][s] * r["prob"][s], 0.0))
        r["z"][s] = (lse * lse).mean()
        b["prob"][s] = steps * r["prob"][s] + 2.0 ** -149
        b["loss"][s] = (steps + 4 * U) * r["loss"][s]
        b["z"][s] = steps * r["z"][s] + (2 * np.abs(lse) * (66 * U + 3 * U * np.abs(lse))).mean()
    return r, b


def gradient(l, counts, tokens, grad_loss, grad_z, k, score, dtype, offsets=None, mask=None):
    l = l.astype(np.float64)
    T, E = l.shape
    out, bound = np.zeros((T, E)), np.zeros((T, E))
    for s, at in enumerate(sequences(T, offsets, mask)):
        n = float(tokens[s])
        if not len(at) or not n:
            continue
        p, lse, rest = scores(l[at], score)
        g = (0.0 if grad_loss is None else grad_loss[s]) * E / (k * n * n) * counts[s][None, :].astype(np.float64)
        zt = (0.0 if grad_z is None else grad_z[s]) * 2.0 / n * lse[:, None]
        dot = (np.where(p != 0, g * p, 0.0)).sum(1, keepdims=True)
        v = np.where(p != 0, p * (g - dot + zt) * rest, 0.0)
        out[at] = v
        # p and every term of the bracket to 128 U and the rounding of each step; the sum of 256 products 24 U more
        terms = np.abs(g) + (np.abs(g) * p).sum(1, keepdims=True) + np.abs(zt)
        mag = np.where(p != 0, p * terms * rest, 0.0)
        bound[at] = 300 * U * mag + HALF[dtype] * np.abs(v) + TINY[dtype]
    return out, bound
