"""Tensors that a call writes through `out`: autograd learns of it."""
import pytest
import torch

import mixture_experts_router_amd as moe
import moe_inputs as mi
from gpu_util import Dev

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def data():
    x, w = rand(1, 20, 64).bfloat16(), rand(2, 16, 64).bfloat16()
    l = rand(3, 20, 16)
    idx = torch.topk(l, 2).indices.to(torch.int32)
    return x, w, l, idx


def writers():
    x, w, l, idx = data()
    bal = moe.balance_loss(l, idx)
    one, gw = torch.ones(1, device="cuda"), rand(7, 20, 2)
    a, b = rand(8, 3, 8, 64).bfloat16(), rand(9, 3, 16, 8).bfloat16()
    ids = torch.zeros(20, dtype=torch.int32, device="cuda")
    base = rand(5, 20, 16).bfloat16()
    w2 = lambda out: (idx.clone(), out)  # noqa: E731
    return {
        "linear": (lambda out: moe.linear(x, w, out=out), base),
        "linear in place": (lambda out: moe.linear(x, w, residual=out, out=out), base),
        "balance_loss_backward": (lambda out: moe.balance_loss_backward(l, bal["counts"], bal["tokens"], one, 2, out=out),
                                  l),
        "gate_from_logits": (lambda out: moe.gate_from_logits(l, 2, out=w2(out)), gw),
        "gate": (lambda out: moe.gate(x, w, 2, out=w2(out)), gw),
        "gate_backward": (lambda out: moe.gate_backward(l, idx, gw, out=out), l),
        "lora_add": (lambda out: moe.lora_add(x, base, ids, a, b, out=out), base),
        "lora_add in place": (lambda out: moe.lora_add(x, out, ids, a, b, out=out), base),
    }


NAMES = ["linear", "linear in place", "balance_loss_backward", "gate_from_logits", "gate", "gate_backward", "lora_add",
         "lora_add in place"]


@pytest.mark.parametrize("name", NAMES)
def test_autograd_sees_what_out_overwrites(name):
    """A tensor that a graph has saved: its backward pass refuses the changed value, as after any in-place operation."""
    call, like = writers()[name]
    out = like.clone()
    leaf = rand(11, *out.shape).to(out.dtype).requires_grad_()
    y = (leaf * out).sum()
    call(out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    view = like.clone()
    part = view[:, :]
    y = (leaf * view).sum()
    call(part)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("name", NAMES)
def test_an_out_that_requires_grad(name):
    """Writing over it would leave a graph that belongs to another value."""
    call, like = writers()[name]
    leaf = like.clone().requires_grad_()
    node = leaf * 1.0
    for out in (leaf, node):
        with pytest.raises(RuntimeError, match="require"):
            call(out)
        with torch.no_grad():
            call(out)


@pytest.mark.parametrize("name", NAMES)
def test_inference_mode(name):
    """Tensors of inference mode have no version: written as ever."""
    with torch.inference_mode():
        call, like = writers()[name]
        call(like.clone())


def test_out_inside_a_captured_graph():
    x, w, l, idx = data()
    out = torch.zeros(20, 16, dtype=torch.bfloat16, device="cuda")
    want = moe.linear(x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear(x, w, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_layers():
    inp = mi.make_inputs("tiny")
    d = Dev(inp)
    for call in (lambda out: moe.layer_forward(d.x, d.wr, inp.k, d.down, gate_up=d.gate_up, out=out),
                 lambda out: moe.layer_forward_noalloc(d.x, d.wr, inp.k, d.down, gate_up=d.gate_up, out=out),
                 lambda out: moe.layer_forward_gated(d.x, d.wr, inp.k, d.down, gate_up=d.gate_up, out=out)):
        out = torch.ones_like(d.x)
        leaf = torch.ones_like(out, requires_grad=True)
        y = (leaf * out).sum()
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
