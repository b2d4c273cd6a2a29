"""The tests' 64-bit gate: its gradient against differences, and worked rows."""
import numpy as np
import pytest

from gate_ref64 import grad64, select64, weights64


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, E, k, h = 5, 11, 3, 1e-5
    l, dw = rng.normal(0, 1.5, (T, E)), rng.normal(0, 1, (T, k))
    idx = select64(l, k, score)
    f = lambda v: (weights64(v, idx, score, renorm, 2.5) * dw).sum(1)  # noqa: E731
    got, _ = grad64(l, idx, dw, score, renorm, 2.5)
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        want = (f(l + d) - f(l - d)) / (2 * h)
        # the difference is off by h^2 / 6 times a third derivative of a few units, and by 1e-16 / h
        assert np.max(np.abs(got[:, e] - want)) < 1e-9


def test_worked_selections():
    l = np.array([[0.0, 2.0, 1.0, 2.0, -np.inf, np.nan]])
    assert select64(l, 6).tolist() == [[1, 3, 2, 0, 4, 5]]  # ties by index, masked, then NaN
    # the bias changes the choice and not the weights: sigmoid(0) = 1/2, sigmoid(ln 3) = 3/4
    l = np.array([[np.log(3.0), 0.0, 0.0]])
    idx = select64(l, 2, "sigmoid", bias=np.array([0.0, 0.5, 0.3]))
    assert idx.tolist() == [[1, 2]]
    assert np.allclose(weights64(l, idx, "sigmoid", True), [[0.5, 0.5]])
    # groups {0,1}, {2,3}: by the best one the second, by the sum of two the first
    l = np.array([[2.0, 2.0, 3.0, -9.0]])
    assert select64(l, 1, groups=2, group_k=1).tolist() == [[2]]
    assert select64(l, 2, "sigmoid", groups=2, group_k=1, group_best=2).tolist() == [[0, 1]]
