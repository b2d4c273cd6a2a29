"""Dense products with their epilogues, and the gradients, against 64 bits (bounds: linear_ref64)."""
import math

import pytest
import torch

import linear_ref64 as ref
import mixture_experts_router_amd as moe

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "sigmoid", "swiglu")


def rand(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def make(seed, T, K, N, dtype="bf16"):
    dt = TYPES[dtype]
    return rand(seed, T, K).to(dt), (rand(seed + 1, N, K) / math.sqrt(K)).to(dt)


def near(got, want, bound, what=""):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), (what, float((off / bound).max()), float(off.max()))


def check(seed, T, K, N, dtype="bf16", act="none", bias=None, residual=False, row_scale=False, out=None, keep=False):
    x, w = make(seed, T, K, N, dtype)
    C = N // 2 if act == "swiglu" else N
    odt = TYPES[out] if out else x.dtype
    b = None if bias is None else (0.3 * rand(seed + 2, N)).to(TYPES[bias])
    r = rand(seed + 3, T, C).to(odt) if residual else None
    s = rand(seed + 4, T) if row_scale else None
    kw = dict(act=act, residual=r, row_scale=s, out_dtype=odt)
    got = moe.linear(x, w, b, want_preact=keep, **kw)
    again = moe.linear(x, w, b, want_preact=keep, **kw)
    if keep:
        got, z = got
        again, z2 = again
        assert z.shape == (T, N) and z.dtype == x.dtype and torch.equal(z, z2)
    assert got.shape == (T, C) and got.dtype == odt and torch.equal(got, again)
    want, bound, wz, zb = ref.forward(x, w, b, act, r, s, odt)
    near(got, want, bound, "out")
    if keep:
        near(z, wz, zb, "preact")


def check_grad(seed, T, K, N, dtype="bf16", act="none", row_scale=False, grad=None, bias=True):
    x, w = make(seed, T, K, N, dtype)
    C = N // 2 if act == "swiglu" else N
    g = rand(seed + 3, T, C).to(TYPES[grad] if grad else x.dtype)
    z = (1.5 * rand(seed + 5, T, N)).to(x.dtype) if act != "none" or row_scale else None
    s = rand(seed + 4, T) if row_scale else None
    want = ("x", "w") + (("bias",) if bias else ()) + (("row_scale",) if row_scale else ())
    r = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=s, want=want)
    assert set(r) == set(want)
    exact = ref.backward(g, x, w, act, z, s)
    for n, v in r.items():
        assert v.dtype == (x.dtype if n in ("x", "w") else torch.float32)
        near(v, *exact[n], n)
    again = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=s, want=want)
    assert all(torch.equal(r[n], again[n]) for n in r)
    for n in want:  # each alone gives the same
        assert torch.equal(moe.linear_backward(g, x, w, act=act, preact=z, row_scale=s, want=(n,))[n], r[n])


SHAPES = [(1, 64, 64), (1, 8, 1), (2, 4096, 16), (3, 72, 33), (15, 136, 250), (16, 256, 256), (17, 1000, 130),
          (33, 64, 999), (64, 2816, 512), (65, 520, 65), (100, 4096, 64), (127, 128, 127), (128, 64, 128),
          (129, 200, 129), (255, 1408, 96), (257, 312, 514), (300, 8, 300), (777, 1024, 320), (1500, 24, 700),
          (2048, 512, 2048)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_products(T, K, N, dtype):
    check(T + N, T, K, N, dtype)
    check(T + N + 50, T, K, N, dtype, out="f32")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (5, 264, 70), (40, 1024, 192), (130, 520, 322), (300, 4096, 64),
                                   (600, 328, 1026)])
def test_epilogues(T, K, N, act):
    check(1, T, K, N, "bf16", act, "f32", True, True, None, True)
    check(2, T, K, N, "f16", act, "f16", True, False, "f32", False)
    check(3, T, K, N, "bf16", act, None, False, True, "f32", True)
    check(4, T, K, N, "bf16", act, "bf16", False, False, None, False)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_gradients_of_products(T, K, N, dtype):
    check_grad(T + N, T, K, N, dtype)
    check_grad(T + N + 50, T, K, N, dtype, grad="f32", bias=False)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (5, 264, 70), (40, 1024, 192), (130, 520, 322), (300, 4096, 64),
                                   (600, 328, 1026), (17000, 64, 48)])
def test_gradients_of_epilogues(T, K, N, act):
    check_grad(1, T, K, N, "bf16", act, True)
    check_grad(2, T, K, N, "f16", act, False, "f32")
    check_grad(3, T, K, N, "bf16", act, True, "f32", False)


def test_more_columns_than_a_workgroup_sums():
    check_grad(1, 20, 64, 6000, "bf16", "silu", True)
    check_grad(2, 9, 64, 8200, "bf16", "swiglu", True, "f32")


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_rows_inside_wider_tensors(act):
    T, K, N = 150, 264, 200
    C = N // 2 if act == "swiglu" else N
    x, w = make(1, T, K, N)
    r = rand(5, T, C).to(x.dtype)
    plain, z = moe.linear(x, w, act=act, residual=r, want_preact=True)
    for pad, at in ((24, 8), (13, 5)):  # operands as they are, and copied; aligned outputs, and not
        wide = lambda t: torch.nn.functional.pad(t, (at, pad - at), value=float("nan"))  # noqa: E731
        cut = lambda t, n: t[:, at:at + n]  # noqa: E731
        wx, ww, wr = wide(x), wide(w), wide(r)
        out = torch.full((T, C + pad), 7.0, dtype=x.dtype, device="cuda")
        assert torch.equal(moe.linear(cut(wx, K), cut(ww, K), act=act, residual=cut(wr, C), out=cut(out, C)),
                           plain)
        assert torch.equal(cut(out, C), plain)
        cut(out, C)[:] = 7.0
        assert torch.all(out == 7.0)
        mine = cut(wr.clone(), C)
        assert moe.linear(x, w, act=act, residual=mine, out=mine) is mine and torch.equal(mine, plain)  # in place
        g = rand(6, T, C).to(x.dtype)
        a = moe.linear_backward(g, x, w, act=act, preact=z, want=("x", "w", "bias"))
        b = moe.linear_backward(cut(wide(g), C), cut(wx, K), cut(ww, K), act=act, preact=cut(wide(z), N),
                                want=("x", "w", "bias"))
        assert all(torch.equal(a[n], b[n]) for n in a)
    # orders other than rows
    assert torch.equal(moe.linear(x.t().contiguous().t(), w.t().contiguous().t(), act=act, residual=r), plain)
    assert torch.equal(moe.linear(x[:1], w, act=act)[0], moe.linear(x[:1].clone(), w, act=act)[0])


def test_offsets_past_32_bits():
    """Rows 2^22 elements apart: 260 of them are more than 2^31 bytes."""
    T, ld, K, N = 600, 1 << 22, 64, 40
    x, w = make(2, T, K, N)
    wide = torch.empty((T, ld), dtype=x.dtype, device="cuda")  # 5 GB
    wide[:, :K] = x
    wide[:, K:K + 8] = float("nan")
    assert torch.equal(moe.linear(wide[:, :K], w), moe.linear(x, w))
    g = rand(3, T, N).to(x.dtype)
    a, b = moe.linear_backward(g, wide[:, :K], w), moe.linear_backward(g, x, w)
    assert all(torch.equal(a[n], b[n]) for n in a)
    wide[:, 128:128 + N] = g
    out = wide[:, 256:256 + N]
    moe.linear(x, w, residual=wide[:, 128:128 + N], out=out)
    assert torch.equal(out, moe.linear(x, w, residual=g))
    b = moe.linear_backward(wide[:, 128:128 + N], x, w, want=("x", "w", "bias"))
    assert torch.equal(b["x"], a["x"]) and torch.equal(b["w"], a["w"])


def test_infinities_and_nan_stay_in_their_rows():
    for T in (3, 40, 300):
        x, w = make(4, T, 200, 96)
        want = moe.linear(x, w)
        x2 = x.clone()
        x2[1, 7], x2[T - 1, 199] = float("nan"), float("inf")
        got = moe.linear(x2, w)
        other = torch.ones(T, dtype=torch.bool, device="cuda")
        other[1] = other[T - 1] = False
        assert torch.equal(got[other], want[other]) and bool(got[1].isnan().all())
        assert bool((got[T - 1].isinf() | got[T - 1].isnan()).all())
        # the neighbour in memory of a row's end is not read: K is no multiple of the steps
        wide = torch.full((T, 208), float("inf"), dtype=x.dtype, device="cuda")
        wide[:, :200] = x
        assert torch.equal(moe.linear(wide[:, :200], w), want)
        big = torch.full((T, 96), 3e38, device="cuda")
        assert bool(torch.isfinite(moe.linear(x, w, residual=big, out_dtype=torch.float32)).all())


def test_saturated_activations():
    """Far values: the activation's limits, and slopes that vanish instead of NaN."""
    z = torch.tensor([[-1e4, -200.0, -90.0, -30.0, 0.0, 30.0, 90.0, 1e4]], device="cuda")
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    for act, f in (("relu", torch.relu), ("silu", torch.nn.functional.silu), ("sigmoid", torch.sigmoid),
                   ("gelu", torch.nn.functional.gelu)):
        got = moe.linear(x, w, z[0].contiguous(), act=act, out_dtype=torch.float32)
        assert torch.allclose(got, f(z.double()).float(), rtol=1e-6, atol=1e-12), act
        g = moe.linear_backward(torch.ones_like(got), x, w, act=act, preact=z.bfloat16(), want=("bias",))["bias"]
        assert bool(torch.isfinite(g).all()), act
        leaf = z.bfloat16().double().requires_grad_()
        f(leaf).sum().backward()
        assert torch.allclose(g, leaf.grad[0].float(), rtol=1e-5, atol=1e-6), act


def test_no_tokens():
    x, w = make(5, 0, 64, 24)
    assert moe.linear(x, w, act="swiglu").shape == (0, 12)
    r = moe.linear_backward(torch.zeros(0, 24, device="cuda"), x, w, want=("x", "w", "bias"))
    assert r["x"].shape == (0, 64) and bool((r["w"] == 0).all()) and bool((r["bias"] == 0).all())


def test_a_token_alone_gives_what_a_batch_gives_to_rounding():
    x, w = make(6, 64, 4096, 256)
    batch, bound, *_ = ref.forward(x, w)
    near(torch.cat([moe.linear(x[i:i + 1], w) for i in range(64)]), batch, bound)


@pytest.mark.parametrize("act", ACTS)
def test_autograd(act):
    T, K, N = 50, 72, 44
    C = N // 2 if act == "swiglu" else N
    x, w = make(7, T, K, N)
    b, r, s = 0.3 * rand(8, N), rand(9, T, C).to(x.dtype), rand(10, T)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r, s)]
    out = moe.linear(leaves[0], leaves[1], leaves[2], act=act, residual=leaves[3], row_scale=leaves[4])
    plain, z = moe.linear(x, w, b, act=act, residual=r, row_scale=s, want_preact=True)
    assert torch.equal(out, plain)
    g = rand(11, T, C).to(x.dtype)
    out.backward(g)
    want = moe.linear_backward(g, x, w, act=act, preact=z, row_scale=s, want=("x", "w", "bias", "row_scale"))
    for leaf, n in zip(leaves, ("x", "w", "bias", None, "row_scale")):
        assert torch.equal(leaf.grad, g if n is None else want[n].to(leaf.dtype))
    # only some of them, an expanded gradient, a bias in 16 bits
    one, b16 = w.clone().requires_grad_(), b.to(x.dtype).requires_grad_()
    moe.linear(x, one, b16, act=act).sum().backward()
    assert one.grad.shape == w.shape and b16.grad.dtype == x.dtype
    (gx,) = torch.autograd.grad((moe.linear(leaves[0], w, act=act).float() ** 2).sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        gx.sum().backward()
    with pytest.raises(RuntimeError, match="require"):
        moe.linear(leaves[0], w, out=torch.empty_like(plain))
    with torch.no_grad():
        assert not moe.linear(leaves[0], w).requires_grad


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    """Central differences in 64 bits of the definition, at the preactivations that the kernels are given: h^2 times a
    third derivative (below 2 in sum), and the rounding of dz and of the result."""
    T, K, N = 4, 8, 6
    x, w = make(12, T, K, N)
    x, w = x * 0.5, w * 0.5
    z0 = (x.double() @ w.double().t()).to(x.dtype)
    C = N // 2 if act == "swiglu" else N
    g = rand(13, T, C).to(x.dtype)
    r = moe.linear_backward(g, x, w, act=act, preact=z0, want=("x", "w"))

    def loss(x, w):  # around the rounded preactivation
        z = z0.double() + (x @ w.t() - x0 @ w0.t())
        return (ref.act(act, z)[0] * g.double()).sum()

    x0, w0, h = x.double(), w.double(), 1e-4
    if act == "relu":
        assert bool((z0.double().abs() > 1e-3).all())
    for n, base in (("x", x0), ("w", w0)):
        want = torch.zeros_like(base)
        for i in range(base.shape[0]):
            for j in range(base.shape[1]):
                d = torch.zeros_like(base)
                d[i, j] = h
                hi = loss(x0 + d, w0) if n == "x" else loss(x0, w0 + d)
                lo = loss(x0 - d, w0) if n == "x" else loss(x0, w0 - d)
                want[i, j] = (hi - lo) / (2 * h)
        near(r[n], want, ref.backward(g, x, w, act, z0)[n][1] + 1e-6, n)


def test_refusals():
    x, w = make(14, 10, 64, 24)
    f32, odd = torch.zeros(10, 24, device="cuda"), torch.zeros(10, 60, dtype=x.dtype, device="cuda")
    for call, err in (
            (lambda: moe.linear(x.float(), w), TypeError), (lambda: moe.linear(x, w.half()), TypeError),
            (lambda: moe.linear(x, w[:, :56]), ValueError), (lambda: moe.linear(x, w, act="tanh"), ValueError),
            (lambda: moe.linear(x, w, out_dtype=torch.float16), TypeError),
            (lambda: moe.linear(x, w, torch.zeros(24, dtype=torch.float16, device="cuda")), TypeError),
            (lambda: moe.linear(x, w, torch.zeros(23, device="cuda")), ValueError),
            (lambda: moe.linear(x, w, residual=f32), TypeError),
            (lambda: moe.linear(x, w, residual=f32.bfloat16()[:9]), ValueError),
            (lambda: moe.linear(x, w, row_scale=torch.zeros(9, device="cuda")), ValueError),
            (lambda: moe.linear(x, w, out=f32), TypeError), (lambda: moe.linear(x, w.cpu()), ValueError),
            (lambda: moe.linear(x, w[:23], act="swiglu"), moe.MoeError),
            (lambda: moe.linear(odd, odd), moe.MoeError),  # K = 60
            (lambda: moe.linear_backward(f32.half(), x, w), TypeError),
            (lambda: moe.linear_backward(f32[:9], x, w), ValueError),
            (lambda: moe.linear_backward(f32, x, w, act="silu"), ValueError),
            (lambda: moe.linear_backward(f32, x, w, want=("row_scale",)), ValueError),
            (lambda: moe.linear_backward(f32, x, w, want=("y",)), ValueError),
            (lambda: moe.linear_backward(f32, x, w, act="silu", preact=f32), TypeError)):
        with pytest.raises(err):
            call()


def test_streams_and_graphs():
    T, K, N = 200, 1024, 96
    x, w = make(15, T, K, N)
    g = rand(16, T, N // 2).to(x.dtype)
    want, z = moe.linear(x, w, act="swiglu", want_preact=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.linear(x, w, act="swiglu", stream=side)
    grads = moe.linear_backward(g, x, w, act="swiglu", preact=z, want=("x", "w", "bias"), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    plain = moe.linear_backward(g, x, w, act="swiglu", preact=z, want=("x", "w", "bias"))
    assert all(torch.equal(grads[n], plain[n]) for n in plain)
    lx, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
    eager = moe.linear(lx, lw, act="swiglu")  # an eager graph of the leaves that stays alive
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same calls, replayed in turn: each has its own workspaces
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(RuntimeError, match="captured"):
                moe.linear(lx, lw)
            with torch.no_grad():
                o, zz = moe.linear(lx, lw, act="swiglu", want_preact=True)
                r = moe.linear_backward(g, lx, lw, act="swiglu", preact=zz, want=("x", "w", "bias"))
        graphs.append((graph, o, zz, r))
    for i in range(4):
        x2, w2 = make(30 + i, T, K, N)
        with torch.no_grad():
            lx.copy_(x2)
            lw.copy_(w2)
        for graph, *_ in graphs:
            graph.replay()
        want, z = moe.linear(x2, w2, act="swiglu", want_preact=True)
        plain = moe.linear_backward(g, x2, w2, act="swiglu", preact=z, want=("x", "w", "bias"))
        for _, o, zz, r in graphs:
            assert torch.equal(o, want) and torch.equal(zz, z) and all(torch.equal(r[n], plain[n]) for n in plain)
        torch.cuda.synchronize()
    del eager
