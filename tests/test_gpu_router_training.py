"""The balance loss and the dense products as they are used together: a training step of a router, an expert that every
token takes beside the routed ones, and calls that share a device."""
import numpy as np
import pytest
import torch

import balance_ref64
import linear_ref64 as ref
import mixture_experts_router_amd as moe
import moe_inputs as mi
from gpu_util import Dev

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,K,E,k", [(300, 256, 32, 4), (1030, 512, 64, 2)])
def test_a_training_step_of_a_router(T, K, E, k, score):
    """Logits by linear, the gate, the balance loss of padded sequences; one backward pass through all of them against
    autograd in 64 bits of the same routing."""
    x, w = rand(1, T, K).bfloat16(), (rand(2, E, K) / K ** 0.5).bfloat16()
    b = 0.1 * rand(3, E)
    up = rand(4, T, k)  # what the weights' gradient would be
    offsets = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[T // 3 - 7:T // 3] = False
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    logits = moe.linear(*leaves, out_dtype=torch.float32)
    gate = moe.gate_from_logits(logits, k, score=score, scale=2.0)
    bal = moe.balance_loss(logits, gate["idx"], score=score, offsets=offsets, mask=mask)
    loss = (gate["w"] * up).sum() + 3.0 * bal["loss"].sum()
    if score == "softmax":
        loss = loss + 0.5 * bal["z"].sum()
    loss.backward()

    # the same in 64 bits
    l = (x.double() @ w.double().t() + b.double()).requires_grad_()
    at = gate["idx"].long()
    if score == "softmax":
        p, wts = torch.softmax(l, 1), 2.0 * torch.softmax(l.gather(1, at), 1)
    else:
        s = torch.sigmoid(l)
        p, sel = s / (s.sum(1, keepdim=True) + 1e-20), s.gather(1, at)
        wts = 2.0 * sel / (sel.sum(1, keepdim=True) + 1e-20)
    total = (wts * up.double()).sum()
    for q in range(3):
        rows = torch.arange(int(offsets[q]), int(offsets[q + 1]), device="cuda")
        rows = rows[mask[rows]]
        n = len(rows)
        assert int(bal["tokens"][q]) == n
        if not n:
            assert bal["loss"][q] == 0
            continue
        c = torch.bincount(at[rows].reshape(-1), minlength=E)
        assert torch.equal(bal["counts"][q].long(), c)
        one = E / (k * n) * (c.double() * p[rows].mean(0)).sum()
        assert abs(float(bal["loss"][q]) - float(one)) <= 1e-4 * float(one)
        total = total + 3.0 * one
        if score == "softmax":
            total = total + 0.5 * (torch.logsumexp(l[rows], 1) ** 2).mean()
    total.backward()
    # fp32 logits of 2^-24 (K / 16 + 96) 2 |x| |w| below 1e-3 and gradients below 10: the slopes are smooth, so 1e-2 of
    # bf16 dz and results (a step is 2^-8) covers every element by its row's or column's sum of absolute products
    dl = l.grad
    want, bound = ref.backward(dl, x, w)["x"]
    assert bool(((leaves[0].grad.double() - want).abs() <= bound + 2e-3 * (dl.abs() @ w.double().abs())).all())
    want, bound = ref.backward(dl, x, w)["w"]
    assert bool(((leaves[1].grad.double() - want).abs() <= bound + 2e-3 * (dl.abs().t() @ x.double().abs())).all())
    assert bool(((leaves[2].grad.double() - dl.sum(0)).abs() <= 2e-3 * dl.abs().sum(0)).all())


@pytest.mark.parametrize("name", ["tiny", "mid"])
def test_a_shared_expert_beside_the_routed_ones(name):
    """out = routed + sigmoid(x . g) * W_down swiglu(W_gate_up x): three products, the last in place on the layer's
    output."""
    inp = mi.make_inputs("tiny") if name == "tiny" else mi.make_inputs("tiny", T=70)
    d = Dev(inp)
    T, H = d.x.shape
    I = 96
    wgu, wd, g = ((rand(i, *s) / s[-1] ** 0.5).to(d.x.dtype) for i, s in ((5, (2 * I, H)), (6, (H, I)), (7, (1, H))))
    y = moe.layer_forward(d.x, d.wr, inp.k, d.down, gate_up=d.gate_up)
    routed = y.clone()
    s = moe.linear(d.x, g, act="sigmoid", out_dtype=torch.float32).view(T)
    h = moe.linear(d.x, wgu, act="swiglu")
    out = moe.linear(h, wd, residual=y, row_scale=s, out=y)
    assert out is y
    vs, bs, *_ = ref.forward(d.x, g, None, "sigmoid", None, None, torch.float32)
    vh, bh, *_ = ref.forward(d.x, wgu, None, "swiglu")
    assert bool(((s.double() - vs[:, 0]).abs() <= bs[:, 0]).all())
    assert bool(((h.double() - vh).abs() <= bh).all())
    want, bound, *_ = ref.forward(h, wd, None, "none", routed, s)
    assert bool(((out.double() - want).abs() <= bound).all())


def test_the_same_expert_twice_and_every_pair_dropped():
    l = rand(8, 40, 16)
    idx = torch.full((40, 3), 5, dtype=torch.int32, device="cuda")
    r = moe.balance_loss(l, idx)
    assert r["counts"][0, 5] == 120 and int(r["counts"].sum()) == 120
    want, bound = balance_ref64.balance(l.cpu().numpy(), idx.cpu().numpy(), "softmax")
    assert abs(float(r["loss"][0]) - want["loss"][0]) <= bound["loss"][0]
    r = moe.balance_loss(l, torch.full_like(idx, -1))
    assert r["loss"][0] == 0 and int(r["counts"].sum()) == 0 and int(r["tokens"][0]) == 40
    g = moe.balance_loss_backward(l, r["counts"], r["tokens"], torch.ones(1, device="cuda"), 3)
    assert bool((g == 0).all())


def test_calls_on_two_streams_at_once():
    """Every call has its own workspace: results are those of the calls alone."""
    cases = [(900, 4096, 64), (64, 2816, 512), (130, 1024, 700)]
    data = [((rand(10 + i, T, K)).bfloat16(), (rand(20 + i, N, K) / K ** 0.5).bfloat16()) for i, (T, K, N) in
            enumerate(cases)]
    lg = rand(30, 5000, 64)
    idx = torch.topk(lg, 4).indices.to(torch.int32)
    alone = [(moe.linear(x, w), moe.linear_backward(rand(40, len(x), len(w)), x, w, want=("x", "w", "bias")))
             for x, w in data]
    bal = moe.balance_loss(lg, idx)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):
        st = streams[turn % 2]
        x, w = data[turn % 3]
        g = rand(40, len(x), len(w))
        torch.cuda.synchronize() if turn == 0 else None
        st.wait_stream(torch.cuda.current_stream())
        got.append((turn % 3, moe.linear(x, w, stream=st),
                    moe.linear_backward(g, x, w, want=("x", "w", "bias"), stream=st),
                    moe.balance_loss(lg, idx, stream=st), g))
    torch.cuda.synchronize()
    for i, out, grads, b, _ in got:
        assert torch.equal(out, alone[i][0]) and all(torch.equal(grads[n], alone[i][1][n]) for n in grads)
        assert all(torch.equal(b[n], bal[n]) for n in bal)


def test_a_captured_training_step():
    """The whole step by the explicit calls in one graph, replayed on new inputs with eager work between."""
    T, K, E, k = 700, 256, 64, 4
    x, w = rand(50, T, K).bfloat16(), (rand(51, E, K) / K ** 0.5).bfloat16()
    up, one = rand(52, T, k), torch.ones(1, device="cuda")

    def step(x, w):
        logits = moe.linear(x, w, out_dtype=torch.float32)
        gate = moe.gate_from_logits(logits, k)
        bal = moe.balance_loss(logits, gate["idx"])
        dl = moe.gate_backward(logits, gate["idx"], up)
        dl = dl + moe.balance_loss_backward(logits, bal["counts"], bal["tokens"], one, k, grad_z=one)
        r = moe.linear_backward(dl, x, w, want=("x", "w", "bias"))
        return [logits, bal["loss"], bal["z"], bal["counts"], r["x"], r["w"], r["bias"]]

    step(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, w)
    for i in range(4):
        x.copy_(rand(60 + i, T, K).bfloat16())
        w.copy_((rand(70 + i, E, K) / K ** 0.5).bfloat16())
        graph.replay()
        want = step(x, w)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        torch.cuda.synchronize()


def test_autograd_of_no_tokens():
    w = rand(80, 24, 64).bfloat16().requires_grad_()
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    b = torch.zeros(24, device="cuda", requires_grad=True)
    moe.linear(x, w, b, act="silu").sum().backward()
    assert x.grad.shape == (0, 64) and bool((w.grad == 0).all()) and bool((b.grad == 0).all())
    l = torch.zeros(0, 8, device="cuda", requires_grad=True)
    r = moe.balance_loss(l, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    (r["loss"].sum() + r["z"].sum()).backward()
    assert l.grad.shape == (0, 8)
