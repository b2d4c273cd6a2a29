"""Adapters with infinite or huge values on the GPU against 64-bit numpy: infinite and NaN where the definition is,
and within the bounds of test_gpu_lora.py elsewhere."""
import numpy as np
import pytest
import torch

from gate_ref64 import lora64
from test_gpu_lora import call, check, f64, make

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "same"), ("f16", "same"), ("bf16", "f32"), ("f16", "f32")]


def compare(c, **kw):
    got = f64(call(c, **kw))
    ref = {n: None if v is None else f64(v) if n == "scale" else v.numpy() for n, v in kw.items()}
    with np.errstate(all="ignore"):
        want, mag, vmag = lora64(f64(c["x"]), f64(c["base"]), c["ids"].numpy(), f64(c["a"]), f64(c["b"]), **ref)
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]), "infinities"
    fin = np.isfinite(want)
    K, R, dt = c["x"].shape[1], c["a"].shape[1], c["base"].dtype
    left = 2.0 ** -17 if c["x"].dtype == torch.bfloat16 and dt != torch.float32 else 2.0 ** -21
    with np.errstate(all="ignore"):
        tol = (K + 3 * R + 64) * 2.0 ** -24 * (mag + np.abs(want)) + left * vmag
        if dt != torch.float32:
            tol += torch.finfo(dt).eps / 2 * (np.abs(want) + tol)
        assert np.all(np.abs(got - want)[fin] <= tol[fin] + 1e-37)
    return want


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("R", [16, 128])
def test_an_infinite_rank_beside_values_beyond_fp16(out, R):
    """An infinite row of A makes its own rank infinite; the other ranks, past fp16's range, still count as numbers."""
    c = make(R, 20, 64, 48, 2, R, "f16", out)
    c["x"], c["a"], c["b"] = c["x"].abs() + 50, c["a"].abs() * 8 + 30, c["b"].abs() + 0.5
    c["a"][0, 0, 7], c["a"][1, R - 1, 8] = torch.inf, -torch.inf
    c["b"][0, :, 3], c["b"][1, :, 4] = -1.0, 2.0
    c["b"][:, ::2, 0] *= -1
    want = compare(c)
    ids = c["ids"].numpy()
    assert np.isinf(want[ids >= 0]).all() and (want[ids == 0] > 0).any() and (want[ids == 0] < 0).any()


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("R", [8, 32, 64])
def test_values_beyond_bf16(out, R):
    """v = 3.4e38 is an fp32 number that rounds to infinity in bf16 (whose largest is 3.3895e38)."""
    c = make(R, 20, 64, 40, 2, R, "bf16", out)
    c["a"].zero_()
    c["a"][:, 0, 0] = 1.0
    c["x"][:, 0] = 1.0
    c["x"][3:9, 0] = -1.0
    c["base"].zero_()
    c["b"] *= 2.0 ** -20
    check(c, scale=torch.tensor([3.4e38, -3.4e38]))


@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 128])
@pytest.mark.parametrize("N", [40, 1100])
@pytest.mark.parametrize("dtype,out", FORMS)
def test_infinities_in_b(R, N, dtype, out):
    """An infinite element of B gives the infinity that its product with v has, whether v needs one 16-bit part (whole
    numbers) or more (the parts then have either sign); two of them that cancel, and one that meets v = 0, give NaN."""
    c = make(R + N, 40, 72, N, 4, R, dtype, out)
    c["ids"] = torch.arange(40, dtype=torch.int32) % 4
    g = torch.Generator().manual_seed(R)
    c["a"][1] = torch.randint(-2, 3, (R, 72), generator=g).to(c["a"].dtype)
    c["x"][1::4] = torch.randint(-2, 3, (10, 72), generator=g).to(c["x"].dtype)
    c["a"][1, 5] = 0
    for i in range(3):  # adapter 3 is finite
        c["b"][i, 3, 0] = torch.inf
        c["b"][i, 17, R - 1] = -torch.inf
        c["b"][i, 8, 2], c["b"][i, 8, 4] = torch.inf, torch.inf
        c["b"][i, 9, 2], c["b"][i, 9, 4] = torch.inf, -torch.inf
        c["b"][i, 39, 5] = torch.inf
        c["b"][i, N - 1, 1] = torch.inf
        c["b"][i, 20, 6] = torch.nan
    want = compare(c, scale=torch.tensor([1.0, 1.0, -0.375, 2.0]))
    # columns 3 and 17 of the 20 tokens of adapters 0 and 2 meet one infinity each
    assert np.isinf(want).sum() >= 40 and np.isnan(want[:, [9, 39]]).any() and np.isfinite(want[3::4]).all()


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("R", [16, 32, 128])
def test_the_smallest_of_a_tokens_values_meets_an_infinity(out, R):
    """v of one rank 2^-45 of another's: fp16 parts, scaled by the largest, round it to 0, yet it is not."""
    c = make(5, 9, 64, 40, 1, R, "f16", out)
    c["ids"].zero_()
    c["a"].zero_()
    c["x"][:, 0], c["x"][:, 1] = 2.0 ** 14, 2.0 ** -10
    c["a"][0, 0, 0], c["a"][0, 1, 1], c["a"][0, 2, 1] = 2.0 ** 10, 2.0 ** -11, -2.0 ** -11
    c["b"] *= 2.0 ** -12
    c["b"][0, 5, 1], c["b"][0, 6, 2] = torch.inf, torch.inf
    want = compare(c)
    assert np.all(want[:, 5] == np.inf) and np.all(want[:, 6] == -np.inf)
