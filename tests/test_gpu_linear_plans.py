"""Which form each size takes: the choice by expected time, row by row, and that the rows reach every form there is, so
that a change of the choice which leaves a form without a test shows."""
import pytest

import mixture_experts_router_amd as moe
from test_gpu_linear import make, rand
from test_gpu_linear_forms import form

pytestmark = pytest.mark.gpu

# T, K, N (rows of W), form, form with swiglu (None: not looked at; an odd N has none)
FORWARD = [
    (20, 72, 17, "linear_stream_1", None), (20, 72, 18, "linear_stream_1", "linear_stream_1"),
    (23, 72, 5001, "linear_stream_2", None), (33, 72, 5002, None, "linear_stream_2"),
    (33, 520, 9002, "linear_64x64", "linear_64x128"), (33, 4104, 2602, "linear_64x64+join", "linear_64x64+join"),
    (1500, 72, 2002, "linear_128x128", "linear_128x128"), (1500, 136, 2000, "linear_128x128", "linear_128x128"),
    (70, 4104, 3302, "linear_128x128+join", "linear_128x128+join"),
    (501, 72, 9002, "linear_192x128", "linear_stream_2"), (501, 264, 9016, "linear_192x128", "linear_128x256"),
    (2001, 72, 4002, "linear_128x256", "linear_128x256"), (2001, 328, 4008, "linear_128x256", "linear_128x256"),
    (3001, 200, 2608, "linear_192x256", "linear_192x256"), (2501, 328, 4992, "linear_256x256", "linear_256x256"),
    (1237, 1096, 4010, "linear_192x128", None),
]
PLAIN = {"linear_stream_1", "linear_stream_2", "linear_64x64", "linear_64x64+join", "linear_128x128",
         "linear_128x128+join", "linear_128x256", "linear_192x128", "linear_192x256", "linear_256x256"}
GATED = (PLAIN - {"linear_64x64", "linear_192x128"}) | {"linear_64x128"}


@pytest.mark.parametrize("T,K,N,plain,gated", FORWARD)
def test_forward(T, K, N, plain, gated):
    for dtype in ("bf16", "f16"):
        x, w = make(T, T, K, N, dtype)
        for act, name in (("none", plain), ("gelu", plain), ("swiglu", gated)):
            if name:
                moe.linear(x, w, act=act)
                assert form(moe.last_plan()) == name


def test_forward_reaches_every_form():
    assert {r[3] for r in FORWARD} - {None} == PLAIN and {r[4] for r in FORWARD} - {None} == GATED


# a product M x N over K of the backward pass
PRODUCTS = [
    (30, 72, 100, "linear_64x64"), (33, 3304, 2051, "linear_64x64+join"), (203, 9000, 77, "linear_128x128"),
    (70, 3304, 4103, "linear_128x128+join"), (2001, 4008, 201, "linear_128x256"), (501, 9016, 201, "linear_192x128"),
    (1237, 4008, 1029, "linear_192x128"), (3001, 2600, 301, "linear_192x256"), (2501, 4992, 333, "linear_256x256"),
]


@pytest.mark.parametrize("M,N,K,name", PRODUCTS)
def test_gradients(M, N, K, name):
    """A 16-bit gradient: dz W with M tokens and K rows of W, then dz^T x with K tokens and M rows of W."""
    for dtype in ("bf16", "f16"):
        x, w = make(M, M, N, K, dtype)
        z = rand(5, M, K).to(x.dtype)
        moe.linear_backward(rand(4, M, K).to(x.dtype), x, w, act="silu", preact=z, want=("x",))
        assert moe.last_plan()[0] == "linear_dz" and form(moe.last_plan()[1:]) == name
        x, w = make(M, K, N, M, dtype)
        z = rand(5, K, M).to(x.dtype)
        moe.linear_backward(rand(4, K, M).to(x.dtype), x, w, act="silu", preact=z, want=("w",))
        assert moe.last_plan()[0] == "linear_dz" and form(moe.last_plan()[1:]) == name


def test_gradients_reach_every_form():
    assert {r[3] for r in PRODUCTS} == {f for f in PLAIN if "stream" not in f}
