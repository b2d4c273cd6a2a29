"""The gate's order where logits are NaN or infinite, against 64-bit numpy.

A NaN logit is the last choice of all, after the masked experts: the softmax that orders the others leaves it out, and
it adds nothing to its group's worth as the second best.  A logit of +inf has the softmax's limit as its score: 1 / n
for each of n, and 0 for the others.  Weights of such rows are NaN where their formula is, and 0 for masked experts all
the same.
"""
import numpy as np
import pytest
import torch

from gate_ref64 import rank_order, weights64


def scores64(l, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        s = np.zeros_like(l)
        for t, row in enumerate(l):
            known = ~np.isnan(row)
            m = row[known].max() if known.any() else -np.inf
            if m == np.inf:
                s[t] = row == np.inf
            elif m > -np.inf:
                s[t] = np.exp(row - m)
            s[t, known] /= max(s[t, known].sum(), 1e-300)
            s[t, ~known] = np.nan
        return s


def select64(l, k, score, bias=None, groups=0, group_k=0, group_best=1):
    T, E = l.shape
    by_score = bias is not None or (groups > 1 and group_best == 2)
    keys = l if not by_score else scores64(l, score) + (0.0 if bias is None else bias)
    keys = np.where(np.isneginf(l), -np.inf, keys)
    order = rank_order(keys)
    if groups <= 1:
        return order[:, :k]
    gs = E // groups
    worth = np.zeros((T, groups))
    for g in range(groups):
        part = keys[:, g * gs:(g + 1) * gs]
        best = np.take_along_axis(part, rank_order(part)[:, :group_best], 1)
        worth[:, g] = best[:, 0] + np.where(best[:, 1:] > -np.inf, best[:, 1:], 0.0).sum(1)
    kept = rank_order(worth)[:, :group_k]
    return np.stack([[e for e in order[t] if e // gs in kept[t]][:k] for t in range(T)])


def test_worked_rows():
    inf, nan = np.inf, np.nan
    zero = np.zeros(5)
    l = np.array([[nan, 1.0, -inf, 2.0, nan]])
    for score in ("softmax", "sigmoid"):
        assert select64(l, 5, score, zero).tolist() == [[3, 1, 2, 0, 4]]
    # softmax of (1, 2) without the NaN: 0.27 and 0.73, so a bias of 0.4 changes the order and one of 0.5 does more
    assert select64(l, 2, "softmax", np.array([0, 0.4, 0, 0, 0])).tolist() == [[3, 1]]
    assert select64(l, 2, "softmax", np.array([0, 0.5, 0, 0, 0])).tolist() == [[1, 3]]
    # two of +inf: a half each, the others 0
    l = np.array([[0.0, inf, nan, inf, -inf]])
    assert select64(l, 5, "softmax", np.array([0.4, 0, 9, 0, 9])).tolist() == [[1, 3, 0, 4, 2]]
    assert select64(l, 3, "softmax", np.array([0.6, 0, 9, 0, 9])).tolist() == [[0, 1, 3]]
    # groups {valid, NaN}, {masked, masked}, {NaN, NaN}
    l = np.array([[nan, nan, -inf, -inf, -5.0, nan]])
    assert select64(l, 2, "sigmoid", None, 3, 1, 2).tolist() == [[4, 5]]
    assert select64(l, 4, "softmax", None, 3, 2, 2).tolist() == [[4, 2, 3, 5]]


def rows(seed, E):
    """Eleven kinds of row, each eight times."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(88, E, generator=g) * 1.5
    some = lambda p: torch.rand(8, E, generator=g) < p  # noqa: E731
    kind = [l[i::11] for i in range(11)]  # views
    kind[0][:, E // 3] = torch.nan
    kind[1][some(0.3)] = torch.nan
    kind[1][some(0.4)] = -torch.inf
    kind[2][some(0.9)] = torch.nan
    kind[3].fill_(torch.nan)
    kind[4].fill_(-torch.inf)
    kind[4][:, ::3] = torch.nan
    kind[5].fill_(torch.nan)
    kind[5][:, E - 2] = 0.5
    kind[6][:, E // 2] = torch.inf
    kind[7][some(0.2)] = torch.inf
    kind[7][some(0.2)] = -torch.inf
    kind[8][some(0.1)] = torch.inf
    kind[8][some(0.2)] = torch.nan
    kind[8][some(0.2)] = -torch.inf
    kind[9][some(0.3)] = -torch.inf  # without any of them
    kind[10][:, 1::2] = torch.nan    # one NaN to every valid expert
    return l


SHAPES = [(16, 5, 0, 0, 1), (40, 8, 0, 0, 1), (40, 5, 8, 2, 2), (40, 5, 8, 2, 1), (64, 6, 32, 4, 2), (100, 7, 0, 0, 1),
          (96, 6, 6, 3, 2), (256, 8, 8, 4, 2), (256, 8, 0, 0, 1), (250, 8, 50, 7, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,groups,group_k,group_best", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_order_of_rows_that_are_not_finite(score, with_bias, E, k, groups, group_k, group_best):
    import mixture_experts_router_amd as moe
    l = rows(E + k, E)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.1 if with_bias else None
    kw = dict(groups=groups, group_k=group_k, group_best=group_best)
    want = select64(l.double().numpy(), k, score, None if bias is None else bias.double().numpy(), **kw)
    for renorm in (True, False):
        r = moe.gate_from_logits(l.cuda(), k, score=score, bias=None if bias is None else bias.cuda(), renorm=renorm, **kw)
        idx = r["idx"].cpu().numpy()
        bad = np.flatnonzero((idx != want).any(1))
        assert bad.size == 0, (bad[:5], idx[bad[:3]], want[bad[:3]])


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,groups,group_k,group_best", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_of_rows_that_are_not_finite(score, renorm, E, k, groups, group_k, group_best):
    import mixture_experts_router_amd as moe
    l = rows(E + k, E)
    r = moe.gate_from_logits(l.cuda(), k, score=score, renorm=renorm, groups=groups, group_k=group_k, group_best=group_best)
    idx, w, l64 = r["idx"].cpu().numpy(), r["w"].double().cpu().numpy(), l.double().numpy()
    with np.errstate(all="ignore"):
        want = weights64(l64, idx, score, renorm)
    masked = np.isneginf(np.take_along_axis(l64, idx.astype(np.int64), 1))
    assert masked.any() and np.all(w[masked] == 0)
    want[masked] = 0.0
    assert np.isnan(want).any() and np.array_equal(np.isnan(w), np.isnan(want))
    # 2^-17: an exponent of up to 40 rounded once, two ulps each of exponential, division and logistic, eight sums
    assert np.all(np.abs(np.nan_to_num(w) - np.nan_to_num(want)) <= 2.0 ** -17 * np.nan_to_num(want) + 1e-37)
