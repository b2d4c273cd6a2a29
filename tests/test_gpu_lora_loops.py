"""The adapters' main loops against 64-bit numpy: several blocks of K and of the columns a wave.

Sixteen waves up to 32 ranks and eight above take 128-column blocks of K and 32-column blocks of the output; these
sizes give each wave more than one of both, with a remainder, and one to eight parts of the columns.  Bounds as in
test_gpu_lora.py.
"""
import numpy as np
import pytest
import torch

import mixture_experts_router_amd as moe
from gate_ref64 import lora64
from test_gpu_lora import call, check, f64, make

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "same"), ("f16", "same"), ("bf16", "f32"), ("f16", "f32")]


@pytest.mark.parametrize("T,K,N", [(1, 4104, 4100), (20, 4104, 4100), (20, 2184, 1064), (70, 4096, 600), (70, 1288, 4096),
                                   (1, 8192, 40)])
@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,out", FORMS)
def test_several_blocks_a_wave(T, K, N, R, dtype, out):
    c = make(T + K + R, T, K, N, 3, R, dtype, out)
    c["ids"][0] = 2
    check(c, scale=torch.tensor([0.5, 1.0, -1.5]), ranks=torch.tensor([R, R - 3, R], dtype=torch.int32))


@pytest.mark.parametrize("T,K,N", [(1, 4104, 4100), (20, 2184, 1064), (70, 4096, 600)])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype,out", FORMS)
def test_whole_numbers_are_exact(T, K, N, R, dtype, out):
    """|v| <= 3 K < 2^16, which two parts hold, and sums stay below 2^24: a block left out, taken twice or misplaced
    changes a result.  A 16-bit output rounds each result once; those beyond fp16 are infinite on both sides."""
    g = torch.Generator().manual_seed(R + K)
    i = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()  # noqa: E731
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    odt = dt if out == "same" else torch.float32
    c = dict(x=i(-1, 1, T, K).to(dt), base=i(-9, 9, T, N).to(odt),
             ids=torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32), a=i(-3, 3, 3, R, K).to(dt),
             b=i(-2, 2, 3, N, R).to(dt))
    c["ids"][0] = 1
    want, _, vmag = lora64(f64(c["x"]), f64(c["base"]), c["ids"].numpy(), f64(c["a"]), f64(c["b"]))
    assert vmag.max() < 2 ** 24 - 9
    assert np.array_equal(f64(call(c)), f64(torch.from_numpy(want).to(odt)))


def test_the_last_of_many_adapters():
    """The adapter 2^32 bytes from the first, at 8192 columns, against the reference."""
    L, K, N, R = 2100, 8192, 8192, 128
    c = make(13, 20, K, N, 1, R)
    c["ids"] = torch.zeros(20, dtype=torch.int32)
    a = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    a[L - 1].copy_(c["a"][0])
    b[L - 1].copy_(c["b"][0])
    last = torch.full((20,), L - 1, dtype=torch.int32, device="cuda")
    check(c, got=moe.lora_add(c["x"].cuda(), c["base"].cuda(), last, a, b))
