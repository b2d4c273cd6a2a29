"""Every kernel form of the dense products, at sizes that end inside its tiles, against 64 bits (bounds: linear_ref64).
The forms are chosen by expected time; the lists name the one each size took when they were written."""
import pytest
import torch

import linear_ref64 as ref
import mixture_experts_router_amd as moe
from test_gpu_linear import make, near, rand

pytestmark = pytest.mark.gpu

# T, K, N (rows of W), form, form with swiglu
FORWARD = [
    (20, 72, 17, "linear_stream_1", None), (20, 72, 18, None, "linear_stream_1"),
    (23, 72, 5001, "linear_stream_2", None), (33, 72, 5002, None, "linear_stream_2"),
    (33, 328, 9000, "linear_64x64", None), (33, 520, 9002, "linear_64x64", "linear_64x128"),
    (33, 2056, 3301, "linear_64x64+join", None), (33, 4104, 2602, "linear_64x64+join", "linear_64x64+join"),
    (200, 72, 9001, "linear_128x128", None), (1500, 72, 2002, "linear_128x128", "linear_128x128"),
    (1500, 136, 2000, "linear_128x128", "linear_128x128"),
    (70, 4104, 3302, "linear_128x128+join", "linear_128x128+join"),
    (501, 72, 9002, "linear_128x256", "linear_128x256"), (501, 264, 9016, "linear_128x256", "linear_128x256"),
    (3001, 72, 2602, "linear_192x256", "linear_192x256"), (3001, 200, 2608, "linear_192x256", "linear_192x256"),
    (2501, 72, 5002, "linear_256x256", "linear_256x256"), (2501, 328, 4992, "linear_256x256", "linear_256x256"),
    (1237, 1096, 4010, "linear_192x128", None), (1333, 2056, 4000, "linear_192x128", None),
    (2001, 72, 4002, "linear_128x256", "linear_128x256"), (2001, 328, 4008, "linear_128x256", "linear_128x256"),
]


FORMS = {f for row in FORWARD for f in row[3:] if f}


def form(plan):
    return plan[0] + ("+join" if plan[1:] == ["linear_join"] else "")


@pytest.mark.parametrize("T,K,N,plain,gated", FORWARD)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward(T, K, N, plain, gated, dtype):
    x, w = make(T, T, K, N, dtype)
    b, s = 0.3 * rand(1, N), rand(2, T)
    for act, want_form in (("gelu", plain), ("swiglu", gated)):
        if want_form is None:
            continue
        C = N // 2 if act == "swiglu" else N
        r = rand(3, T, C).to(x.dtype)
        got, z = moe.linear(x, w, b, act=act, residual=r, row_scale=s, want_preact=True)
        assert form(moe.last_plan()) in FORMS
        want, bound, wz, zb = ref.forward(x, w, b, act, r, s)
        near(got, want, bound, act)
        near(z, wz, zb, "preact")
        out = torch.full((T, C + 3), 7.0, device="cuda")  # fp32, rows that do not start aligned
        moe.linear(x, w, act=act, out_dtype=torch.float32, out=out[:, 1:1 + C])
        want, bound, *_ = ref.forward(x, w, None, act, None, None, torch.float32)
        near(out[:, 1:1 + C], want, bound, act)
        assert bool((out[:, 0] == 7.0).all()) and bool((out[:, 1 + C:] == 7.0).all())


# a product M x N over K of the backward pass: its form
PRODUCTS = [
    (30, 72, 100, "linear_64x64"), (33, 9000, 325, "linear_64x64"), (33, 3304, 2051, "linear_64x64+join"),
    (203, 9000, 77, "linear_128x128"), (70, 3304, 4103, "linear_128x128+join"), (501, 9016, 201, "linear_128x256"),
    (3001, 2608, 70, "linear_192x256"), (3001, 2600, 301, "linear_192x256"), (2501, 5000, 65, "linear_256x256"),
    (2501, 4992, 333, "linear_256x256"), (5, 8, 3, "linear_64x64"),
    (1237, 4008, 1029, "linear_192x128"), (1333, 4000, 2051, "linear_192x128"),
    (2001, 4008, 201, "linear_128x256"),
]


@pytest.mark.parametrize("M,N,K,name", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradient_of_x(M, N, K, name, dtype):
    x, w = make(M, M, N, K, dtype)  # M tokens of N columns, K rows of W
    g, z = rand(4, M, K), rand(5, M, K).to(x.dtype)
    r = moe.linear_backward(g, x, w, act="silu", preact=z, want=("x",))
    assert moe.last_plan()[0] == "linear_dz" and form(moe.last_plan()[1:]) in FORMS
    near(r["x"], *ref.backward(g, x, w, "silu", z)["x"], "x")


@pytest.mark.parametrize("M,N,K,name", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradient_of_w(M, N, K, name, dtype):
    x, w = make(M, K, N, M, dtype)  # K tokens of N columns, M rows of W
    g = rand(4, K, M)
    r = moe.linear_backward(g, x, w, want=("w",))
    assert moe.last_plan()[0] == "linear_dz" and form(moe.last_plan()[1:]) in FORMS
    near(r["w"], *ref.backward(g, x, w)["w"], "w")


def test_the_gradient_itself_as_operand():
    """Nothing to form: no launch for dz, and rows inside a wider tensor as they are."""
    x, w = make(1, 130, 256, 96)
    wide = torch.full((130, 112), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 8:104] = rand(2, 130, 96).to(x.dtype)
    g = wide[:, 8:104]
    r = moe.linear_backward(g, x, w)
    assert "linear_dz" not in moe.last_plan()
    want = ref.backward(g, x, w)
    near(r["x"], *want["x"], "x")
    near(r["w"], *want["w"], "w")
    r = moe.linear_backward(g, x, w, want=("bias",))
    assert moe.last_plan() == ["linear_dz", "linear_sums"]
    near(r["bias"], *want["bias"], "bias")
    r = moe.linear_backward(g[:16], x[:16], w, want=("bias",))  # one block of rows: its sums are the result
    assert moe.last_plan() == ["linear_dz"]
    near(r["bias"], *ref.backward(g[:16], x[:16], w)["bias"], "bias")


def test_plans_of_the_balance_loss():
    l = torch.randn(513, 8, device="cuda")
    idx = torch.zeros(513, 1, dtype=torch.int32, device="cuda")
    moe.balance_loss(l[:512], idx[:512])
    assert moe.last_plan() == ["balance_whole"]
    r = moe.balance_loss(l, idx)
    assert moe.last_plan() == ["balance_part", "balance_join"]
    moe.balance_loss_backward(l, r["counts"], r["tokens"], r["loss"], 1)
    assert moe.last_plan() == ["balance_backward"]


def test_very_many_tokens():
    """Millions of rows of a few columns; outputs of more than 2^32 elements."""
    T = (1 << 22) + 37
    x = rand(1, T, 8).bfloat16()
    w = rand(2, 3, 8).bfloat16()
    got = moe.linear(x, w, out_dtype=torch.float32)
    want, bound, *_ = ref.forward(x, w, out_dtype=torch.float32)
    near(got, want, bound)
    g = rand(3, T, 3)
    r = moe.linear_backward(g, x, w, want=("x", "w", "bias"))
    exact = ref.backward(g, x, w)
    for n in r:
        near(r[n], *exact[n], n)
    del want, bound, exact
    T, N = 2_100_000, 2100  # 4.4e9 elements, rows that do not start aligned
    x, w = rand(4, T, 8).bfloat16(), rand(5, N, 8).bfloat16()
    out = moe.linear(x, w)
    for rows in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 40, T)):
        want, bound, *_ = ref.forward(x[rows], w)
        near(out[rows], want, bound)
    back = moe.linear_backward(out, x, w, want=("x", "bias"))
    for rows in (slice(0, 40), slice(T - 40, T)):
        near(back["x"][rows], *ref.backward(out[rows], x[rows], w)["x"], "x")
