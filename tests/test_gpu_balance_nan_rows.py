"""Rows of logits that hold nothing but NaN, or NaN beside masked experts, against the definition in 64 bits: the mean
squared logsumexp shows them as the loss and the probabilities do, and a row that masks every expert stays a row of 0."""
import numpy as np
import pytest
import torch

import mixture_experts_router_amd as moe
from test_gpu_balance import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 700])  # one launch, and two
@pytest.mark.parametrize("E", [1, 7, 70, 256])
def test_a_row_of_nan(T, E, dtype, score):
    l, idx = make(T + E, T, E, 1, dtype)
    l[3] = np.nan
    l[9] = -np.inf
    if E > 1:
        l[20] = -np.inf
        l[20, E // 2] = np.nan
        l[26, :E - 1] = np.nan  # one number beside NaN
    offsets = torch.tensor([0, 8, 16, 24, 32, T], dtype=torch.int32)
    got, grad = check(l, idx, score, dtype, offsets=offsets)
    lost = [True, False, E > 1, E > 1, False]
    assert got["prob"].isnan().any(1).tolist() == lost
    if score == "softmax":
        assert got["z"].isnan().tolist() == lost
    assert bool(grad[3].isnan().all()) and bool((grad[9] == 0).all())


@pytest.mark.parametrize("T", [12, 600])
def test_z_alone(T):
    """A step that trains on z alone sees a token whose hidden state was NaN."""
    l, idx = make(3, T, 32, 4)
    l[5] = np.nan
    leaf = l.cuda().requires_grad_()
    z = moe.balance_loss(leaf, idx.cuda())["z"]
    assert bool(z.isnan().all())
    z.sum().backward()
    assert bool(leaf.grad[5].isnan().all()) and bool(torch.isfinite(leaf.grad[:5]).all())
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[5] = False
    assert bool(torch.isfinite(moe.balance_loss(l.cuda(), idx.cuda(), mask=mask)["z"]).all())
