"""Products beyond fp16's range: the kept product is infinite there, and the gradient takes the activation's limits."""
import pytest
import torch

import mixture_experts_router_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "sigmoid"])
def test_activations(act):
    """z = 76800 and -76800: exact in fp32, infinite in fp16; slopes 1 and 0 (sigmoid: 0 and 0) and no NaN."""
    x = torch.full((3, 64), 300.0, dtype=torch.float16, device="cuda")
    x[1] = -300.0
    x[2] = 0.5
    w = torch.full((8, 64), 4.0, dtype=torch.float16, device="cuda")
    out, z = moe.linear(x, w, act=act, out_dtype=torch.float32, want_preact=True)
    assert torch.equal(z[:2].float(), torch.tensor([[float("inf")], [-float("inf")]], device="cuda").expand(2, 8))
    high = {"none": 76800.0, "sigmoid": 1.0}.get(act, 76800.0)
    low = {"none": -76800.0}.get(act, 0.0)
    assert torch.equal(out[0], torch.full_like(out[0], high)) and torch.equal(out[1], torch.full_like(out[1], low))
    g = torch.full((3, 8), 0.25, dtype=torch.float16, device="cuda")
    r = moe.linear_backward(g, x, w, act=act, preact=z, want=("x", "bias"))
    slopes = {"none": (1.0, 1.0), "sigmoid": (0.0, 0.0)}.get(act, (1.0, 0.0))
    for t, s in enumerate(slopes):
        assert torch.equal(r["x"][t], torch.full_like(r["x"][t], 8.0 * s)), (act, t)  # 8 columns of 4 times 0.25
    assert bool(torch.isfinite(r["bias"]).all())


def test_swiglu():
    """A gate beyond the range: silu is its argument above, 0 below; NaN stays NaN."""
    x = torch.full((3, 64), 300.0, dtype=torch.float16, device="cuda")
    x[1], x[2, 0] = -300.0, float("nan")
    w = torch.full((16, 64), 4.0, dtype=torch.float16, device="cuda")
    w[8:] = 2.0 ** -10
    g = torch.full((3, 8), 0.25, dtype=torch.float16, device="cuda")
    out, z = moe.linear(x, w, act="swiglu", out_dtype=torch.float32, want_preact=True)
    assert bool(z[:2, :8].isinf().all()) and bool(torch.isfinite(z[:2, 8:]).all())
    assert bool((out[0] == 76800.0 * 18.75).all()) and bool((out[1] == 0).all())
    r = moe.linear_backward(g, x, w, act="swiglu", preact=z, row_scale=torch.ones(3, device="cuda"),
                            want=("x", "row_scale"))
    # below: slope 0 and silu 0, so that nothing comes back
    assert bool((r["x"][1] == 0).all()) and float(r["row_scale"][1]) == 0
    assert bool(r["x"][2].isnan().all()) and bool(r["row_scale"][2].isnan())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_of_the_scale(act):
    z = torch.tensor([[float("-inf")] * 8, [float("nan")] * 8, [1.0] * 8], dtype=torch.float16, device="cuda")
    x, w = torch.zeros(3, 8, dtype=torch.float16, device="cuda"), torch.zeros(8, 8, dtype=torch.float16, device="cuda")
    g = torch.ones(3, 8, dtype=torch.float16, device="cuda")
    r = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=torch.ones(3, device="cuda"), want=("row_scale",))
    assert float(r["row_scale"][0]) == 0 and bool(r["row_scale"][1].isnan()) and 5.0 < float(r["row_scale"][2]) < 8.0
