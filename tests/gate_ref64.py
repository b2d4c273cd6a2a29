"""The routing gate, its gradient and the per-request adapters in 64-bit numpy,
written from their definitions (include/moe.h), for the tests."""
import numpy as np

EPS = 1e-20


def scores64(l, score):
    """fp64 scores of logits [T, E]; a masked expert (-inf) has score 0."""
    l = np.asarray(l, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = np.max(l, axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(l - m)
        z = e.sum(1, keepdims=True)
        return np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))


def rank_order(keys):
    """Indices of every row by descending key, equal keys (and NaN, the lowest) by index."""
    k = np.where(np.isnan(keys), -np.inf, keys)
    low = np.isnan(keys)  # NaN after every number
    return np.lexsort((np.broadcast_to(np.arange(k.shape[1]), k.shape), -k, low), axis=1)


def select64(l, k, score="softmax", bias=None, groups=0, group_k=0, group_best=1, **_):
    l = np.asarray(l, np.float64)
    T, E = l.shape
    by_score = bias is not None or (groups > 1 and group_best == 2)
    keys = l if not by_score else scores64(l, score) + (0.0 if bias is None else np.asarray(bias, np.float64))
    keys = np.where(np.isneginf(l), -np.inf, keys)  # a mask holds against any bias
    live = np.ones((T, E), bool)
    if groups > 1:
        gs = E // groups
        worth = np.zeros((T, groups))
        for g in range(groups):
            part = keys[:, g * gs:(g + 1) * gs]
            order = rank_order(part)[:, :group_best]
            best = np.take_along_axis(part, order, 1)
            worth[:, g] = best[:, 0] + np.where(np.isneginf(best[:, 1:]), 0.0, best[:, 1:]).sum(1)
        kept = rank_order(worth)[:, :group_k]
        live[:] = False
        for t in range(T):
            for g in kept[t]:
                live[t, g * gs:(g + 1) * gs] = True
    out = np.zeros((T, k), np.int32)
    order = rank_order(keys)
    for t in range(T):
        out[t] = [e for e in order[t] if live[t, e]][:k]
    return out


def weights64(l, idx, score="softmax", renorm=True, scale=1.0, **_):
    l = np.asarray(l, np.float64)
    sel = np.take_along_axis(l, idx.astype(np.int64), 1)
    if score == "softmax":
        s = scores64(sel, "softmax") if renorm else np.take_along_axis(scores64(l, "softmax"), idx.astype(np.int64), 1)
        return scale * s
    s = scores64(sel, "sigmoid")
    return scale * (s / (s.sum(1, keepdims=True) + EPS) if renorm else s)


def grad64(l, idx, dw, score="softmax", renorm=True, scale=1.0, **_):
    """(gradient [T, E], magnitude [T, E]): the same sums over absolute values, which rounding errors scale with.
    Indices outside [0, E) have no part; equal ones add up."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = [(s, int(e)) for s, e in enumerate(idx[t]) if 0 <= e < E]
        es = np.array([e for _, e in ok], int)
        g = np.array([scale * float(dw[t, s]) for s, _ in ok])
        if score == "softmax" and not renorm:
            p = scores64(l[t:t + 1], "softmax")[0]
            g = np.where(p[es] > 0, g, 0.0)
            G = np.zeros(E)
            M = np.zeros(E)
            np.add.at(G, es, g)
            np.add.at(M, es, np.abs(g))
            out[t] = p * (G - (G * p).sum())
            mag[t] = p * (M + (M * p).sum())
            continue
        if not len(es):
            continue
        s = scores64(l[t:t + 1, es], "softmax")[0] if score == "softmax" else scores64(l[t:t + 1, es], "sigmoid")[0]
        g = np.where(s > 0, g, 0.0)
        if score == "softmax":
            v, a = s * (g - (g * s).sum()), s * (np.abs(g) + (np.abs(g) * s).sum())
        else:
            d = s / (1.0 + np.exp(l[t, es]))
            tot = s.sum() + EPS if renorm else 1.0
            v = (g - (g * s).sum() / tot) / tot * d if renorm else g * d
            a = (np.abs(g) + (np.abs(g) * s).sum() / tot) / tot * d if renorm else np.abs(g) * d
        np.add.at(out[t], es, v)
        np.add.at(mag[t], es, a)
    return out, mag


def lora64(x, base, ids, a, b, scale=None, ranks=None):
    """(result, magnitude of the sums, |v| part) of base + scale (x A^T) B^T in fp64."""
    out = np.asarray(base, np.float64).copy()
    mag, vmag = np.zeros_like(out), np.zeros_like(out)
    L, R, _ = a.shape
    for t in range(len(out)):
        i = int(ids[t])
        if not 0 <= i < L:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        c = 1.0 if scale is None else float(scale[i])
        A, B, row = a[i, :r].astype(np.float64), b[i, :, :r].astype(np.float64), np.asarray(x[t], np.float64)
        v = A @ row
        out[t] += c * (B @ v)
        mag[t] = abs(c) * (np.abs(B) @ (np.abs(A) @ np.abs(row)))
        vmag[t] = abs(c) * (np.abs(B) @ np.abs(v))
    return out, mag, vmag
