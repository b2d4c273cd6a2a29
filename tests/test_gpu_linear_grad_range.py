"""Gradients of linear from an fp32 gradient: what its 32 bits hold beyond the operands' 16, against 64 bits.

dz enters the products in two 16-bit parts (bf16: up to 256 columns, and rounded once for more).  With bf16 the first is
off by less than 2^-7 of dz and the second rounds what is left by half a step, 2^-8 of it: 2^-15 in all, over bf16's range
of exponents, which is fp32's.  With fp16 the first part holds dz 2^-8, a step of 2^-10 of it or 2^-24, so what is left is
below max(2^-10 |dz|, 2^-16); the second holds that times 2^12, rounded by 2^-11 of it or 2^-25: off by at most
max(2^-21 |dz|, min(2^-11 |dz|, 2^-27)) + 2^-37 up to 2^13.  Above that what is left has no room in the second part, which
then holds 2^-36 in place of it, and the first is rounded to 2^-11 of dz; above 65504 * 2^8 it is infinite.  A part of 2^-36
(bf16: 2^-126) stands where the second would be 0.
"""
import math

import pytest
import torch

import linear_ref64 as ref
import mixture_experts_router_amd as moe
import test_gpu_linear
from test_gpu_linear import rand

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def near(got, want, bound, what):
    """Where the value leaves the type's range by more than the bound, the infinity of its sign."""
    top = torch.finfo(got.dtype).max
    past = want.abs() > top + bound
    assert torch.equal(got.double()[past], want.sign()[past] * float("inf")), what
    here = ~past & (got.isfinite() | (want.abs() < top - bound))
    test_gpu_linear.near(got[here], want[here], bound[here], what)


def off_by(dz, dt):
    a = dz.abs()
    if dt is torch.bfloat16:
        return (2.0 ** -15 if dz.shape[1] <= 256 else ref.HALF[dt]) * a + 2.0 ** -126
    low = torch.maximum(2.0 ** -21 * a, torch.minimum(2.0 ** -11 * a, torch.full_like(a, 2.0 ** -27)))
    return torch.where(a < 2.0 ** 13, low, 2.0 ** -11 * a) + 2.0 ** -36 + 2.0 ** -37


def gradients(g, x, w, act="none", z=None, rs=None):
    """(gradient, bound) of x and w in 64 bits."""
    dz = g.double() if rs is None else g.double() * rs.double()[:, None]
    mag = dz.abs()
    fp32 = torch.zeros_like(dz) if z is None else None
    if z is not None:
        _, *slopes = ref.act(act, z.double())
        if act == "swiglu":
            gate, up = z.double().chunk(2, 1)
            mag = torch.cat((mag * up.abs(), mag * gate.abs()), 1)
        dz = torch.cat([dz * v for v in slopes], 1)
        fp32 = 24 * ref.U * (mag + dz.abs())
    if rs is not None:
        fp32 = fp32 + ref.U * dz.abs()
    rounded = fp32 + off_by(dz, x.dtype) + ref.HALF[x.dtype] * fp32
    h, t = ref.HALF[x.dtype], ref.TINY[x.dtype]

    def product(p, bound, q, n):
        v, b = p @ q, bound @ q.abs()
        b = b + ref.steps(2 * n + 128) * 1.01 * (p.abs() @ q.abs() + b)  # both parts
        return v, b + h * (v.abs() + b) + t

    return dict(x=product(dz, rounded, w.double(), dz.shape[1]), w=product(dz.t(), rounded.t(), x.double(), len(dz)))


def check(g, x, w, act="none", z=None, rs=None):
    r = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=rs)
    want = gradients(g, x, w, act, z, rs)
    for n in r:
        near(r[n], *want[n], n)
    again = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=rs)
    assert all(torch.equal(r[n], again[n]) for n in r)
    for n in r:  # each alone gives the same
        assert torch.equal(moe.linear_backward(g, x, w, act=act, preact=z, row_scale=rs, want=(n,))[n], r[n])
    return r


def operands(seed, T, K, N, dtype, of_x=1.0, of_w=1.0):
    return (of_x * rand(seed, T, K)).to(TYPES[dtype]), (of_w * rand(seed + 1, N, K) / math.sqrt(K)).to(TYPES[dtype])


# one token; the router; one part ends inside a step of k; every tile; k split over workgroups, at a part's end and inside
SHAPES = [(1, 64, 64), (2, 8, 1), (33, 72, 65), (100, 4096, 64), (300, 328, 1026), (777, 1024, 320), (33, 3304, 2051),
          (70, 3304, 4103), (2001, 4008, 201), (501, 9016, 201), (3001, 2600, 301), (2501, 4992, 333), (4100, 512, 64),
          (17000, 64, 48)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_products(T, K, N, dtype):
    x, w = operands(T, T, K, N, dtype)
    check(rand(T + 7, T, N), x, w)
    check(rand(T + 8, T, N) * torch.exp(3.0 * rand(T + 9, T, N)), x, w, rs=rand(T + 10, T))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "sigmoid", "swiglu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_activations(dtype, act):
    T, K, N = 130, 520, 322
    x, w = operands(3, T, K, N, dtype)
    z = (1.5 * rand(4, T, N)).to(x.dtype)
    check(rand(5, T, N // 2 if act == "swiglu" else N), x, w, act, z, rand(6, T))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N", [(40, 264, 64), (2100, 512, 64), (700, 1024, 1026)])
def test_small_and_large_gradients(T, K, N, dtype):
    """About 1e-8 (a balance loss over thousands of tokens) and 1e5, with weights and inputs that bring the results into
    fp16's range; and both in one tensor."""
    x, w = operands(11, T, K, N, dtype, 30.0, 300.0)
    r = check(1e-8 * rand(12, T, N), x, w)
    for v in r.values():
        assert float((v != 0).double().mean()) > 0.5
    x, w = operands(13, T, K, N, dtype, 1e-3, 1e-3)
    r = check(1e5 * rand(14, T, N), x, w)
    assert all(bool(torch.isfinite(v).all()) for v in r.values())
    g = torch.exp(torch.rand(T, N, generator=torch.Generator("cuda").manual_seed(15), device="cuda") * 30.0 - 20.0)
    x, w = operands(16, T, K, N, dtype, 1e-2, 1e-2)
    check(g * rand(17, T, N).sign(), x, w)


def test_the_router_of_a_balance_loss():
    """fp16 hidden states: the balance loss's own gradient, a few 1e-9 a logit, reaches W."""
    T, K, E, k = 4096, 256, 64, 4
    x, w = (8.0 * rand(21, T, K)).half(), (rand(22, E, K) / K ** 0.5 / 8).half()
    logits = moe.linear(x, w, out_dtype=torch.float32)
    gate = moe.gate_from_logits(logits, k)
    bal = moe.balance_loss(logits, gate["idx"])
    g = moe.balance_loss_backward(logits, bal["counts"], bal["tokens"], torch.full((1,), 0.01, device="cuda"), k)
    assert float(g.abs().max()) < 1e-6
    r = check(g, x, w)
    assert float((r["w"] != 0).double().mean()) > 0.5


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N", [(20, 72, 40), (300, 512, 64)])
def test_infinities(T, K, N, dtype):
    """An infinity in W or x beside finite dz gives the infinity that its products have, also where dz is a power of two
    (nothing is left for a second part); one in the gradient stays in its row of x's gradient and its column of W's."""
    x, w = operands(31, T, K, N, dtype)
    g = rand(32, T, N)
    g = torch.where(g.abs() < 0.01, torch.full_like(g, 0.25), g)
    g[1], g[2, 3], g[3] = 1.0, -0.5, 0.125
    plain = check(g, x, w)
    wi, xi = w.clone(), x.clone()
    wi[5, 7], wi[6, 8] = float("inf"), float("-inf")
    r = moe.linear_backward(g, x, wi, want=("x",))["x"]
    assert torch.equal(r[:, 7].double(), torch.sign(g[:, 5].double()) * float("inf"))
    assert torch.equal(r[:, 8].double(), torch.sign(g[:, 6].double()) * -float("inf"))
    rest = [i for i in range(K) if i not in (7, 8)]
    assert torch.equal(r[:, rest], plain["x"][:, rest])
    xi[2, 4] = float("inf")
    r = moe.linear_backward(g, xi, w, want=("w",))["w"]
    assert torch.equal(r[:, 4].double(), torch.sign(g[2].double()) * float("inf"))
    rest = [i for i in range(K) if i != 4]
    assert torch.equal(r[:, rest], plain["w"][:, rest])
    for bad in (float("inf"), float("-inf"), float("nan")):
        gb = g.clone()
        gb[4, 9] = bad
        w1, x1 = torch.where(w == 0, 1.0, w), torch.where(x == 0, 1.0, x)
        plain1, r = moe.linear_backward(g, x1, w1), moe.linear_backward(gb, x1, w1)
        rows = [i for i in range(T) if i != 4]
        assert torch.equal(r["x"][rows], plain1["x"][rows]) and bool((~torch.isfinite(r["x"][4])).all())
        rows = [i for i in range(N) if i != 9]
        assert torch.equal(r["w"][rows], plain1["w"][rows]) and bool((~torch.isfinite(r["w"][9])).all())
        if bad == bad:
            assert torch.equal(r["x"][4].double(), torch.sign(w1[9].double()) * bad)


def test_the_largest_floats():
    """Between bf16's largest value and fp32's a gradient keeps its value."""
    x, w = operands(41, 9, 64, 24, "bf16", 1e-9, 1e-9)
    g = rand(42, 9, 24)
    g[3] = 3.4e38 * g[3].sign()
    g[5] = 2.0 ** -140 * g[5].sign()
    check(g, x, w)
