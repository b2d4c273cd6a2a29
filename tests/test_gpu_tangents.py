"""Forward-mode derivatives: no call has one, and an input with a tangent is refused."""
import pytest
import torch
from torch.autograd import forward_ad as fwd

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


def test_tangents_are_refused():
    x, w, l, idx = data()
    b, res, s = rand(4, 16), rand(5, 20, 16).bfloat16(), rand(6, 20)
    bal = moe.balance_loss(l, idx)
    one, gw = torch.ones(1, device="cuda"), rand(7, 20, 2)
    a, lb = rand(8, 3, 8, 64).bfloat16(), rand(9, 3, 16, 8).bfloat16()
    ids = torch.zeros(20, dtype=torch.int32, device="cuda")
    calls = [
        (lambda t: moe.linear(t, w), x), (lambda t: moe.linear(x, t), w), (lambda t: moe.linear(x, w, t), b),
        (lambda t: moe.linear(x, w, residual=t), res), (lambda t: moe.linear(x, w, row_scale=t), s),
        (lambda t: moe.linear_backward(t, x, w), res), (lambda t: moe.balance_loss(t, idx), l),
        (lambda t: moe.balance_loss_backward(t, bal["counts"], bal["tokens"], one, 2), l),
        (lambda t: moe.balance_loss_backward(l, bal["counts"], bal["tokens"], t, 2), one),
        (lambda t: moe.gate_from_logits(t, 2), l), (lambda t: moe.gate(t, w, 2), x), (lambda t: moe.gate(x, t, 2), w),
        (lambda t: moe.gate_backward(t, idx, gw), l), (lambda t: moe.gate_backward(l, idx, t), gw),
        (lambda t: moe.lora_add(t, res, ids, a, lb), x), (lambda t: moe.lora_add(x, t, ids, a, lb), res),
        (lambda t: moe.lora_add(x, res, ids, t, lb), a), (lambda t: moe.lora_add(x, res, ids, a, t), lb)]
    for call, t in calls:
        call(t)
        with fwd.dual_level():
            with pytest.raises(RuntimeError, match="tangent"):
                call(fwd.make_dual(t, torch.ones_like(t)))
            call(t)  # no tangent, no refusal
        leaf = t.clone().requires_grad_()  # also where reverse mode follows it
        with fwd.dual_level(), pytest.raises(RuntimeError):
            call(fwd.make_dual(leaf, torch.ones_like(t)))


def test_the_gated_layer():
    inp = mi.make_inputs("tiny")
    d = Dev(inp)
    call = lambda x: moe.layer_forward_gated(x, d.wr, inp.k, d.down, gate_up=d.gate_up)  # noqa: E731
    want = call(d.x)
    with fwd.dual_level():
        with pytest.raises(RuntimeError, match="tangent"):
            call(fwd.make_dual(d.x, torch.ones_like(d.x)))
        assert torch.equal(call(d.x), want)
