"""Inputs that require grad: the gate's weights carry gate_backward's graph, and the calls without a backward pass
refuse them instead of returning results that lost it."""
import pytest
import torch

import mixture_experts_router_amd as moe
import moe_inputs as mi
from gpu_util import Dev
from test_gpu_gate import logits_of
from test_gpu_lora import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_weights_carry_the_gradient(score, renorm, dtype):
    l = logits_of(1, 37, 64, dtype).cuda()
    bias = torch.linspace(-0.1, 0.1, 64).cuda()
    kw = dict(score=score, renorm=renorm, scale=2.5)
    sel = dict(bias=bias, groups=8, group_k=4, group_best=2)
    plain = moe.gate_from_logits(l, 6, **kw, **sel)
    leaf = l.clone().requires_grad_()
    r = moe.gate_from_logits(leaf, 6, **kw, **sel)
    assert torch.equal(r["idx"], plain["idx"]) and torch.equal(r["w"], plain["w"])
    assert r["w"].requires_grad and not r["idx"].requires_grad and not plain["w"].requires_grad
    dw = torch.randn(37, 6, device="cuda")
    want = moe.gate_backward(l, plain["idx"], dw, **kw)
    (r["w"] * dw).sum().backward()
    assert leaf.grad.dtype == l.dtype and torch.equal(leaf.grad, want)
    # an expanded gradient, logits inside a wider tensor, a graph of other operations in front, another stream
    wide = torch.zeros(37, 80, dtype=l.dtype, device="cuda")
    wide[:, 8:72] = l
    wide.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = moe.gate_from_logits((wide * 1)[:, 8:72], 6, stream=side, **kw, **sel)
    torch.cuda.current_stream().wait_stream(side)
    r["w"].sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(wide.grad[:, 8:72], moe.gate_backward(l, plain["idx"], torch.ones_like(dw), **kw))
    assert torch.all(wide.grad[:, :8] == 0) and torch.all(wide.grad[:, 72:] == 0)


def test_modes_without_a_graph():
    leaf = logits_of(2, 9, 32).cuda().requires_grad_()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert not moe.gate_from_logits(leaf, 4)["w"].requires_grad
    out = (torch.empty(9, 4, dtype=torch.int32, device="cuda"), torch.empty(9, 4, device="cuda"))
    with pytest.raises(RuntimeError, match="require grad"):
        moe.gate_from_logits(leaf, 4, out=out)
    w = moe.gate_from_logits(leaf, 4)["w"]
    (g,) = torch.autograd.grad((w * w).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    empty = torch.zeros(0, 32, device="cuda", requires_grad=True)
    moe.gate_from_logits(empty, 4)["w"].sum().backward()
    assert empty.grad.shape == (0, 32)


def test_a_captured_step_calls_the_gradient_itself():
    """Logits that require grad are refused during capture, before anything is enqueued; the two calls under no_grad
    are what a captured step records."""
    leaf = logits_of(3, 50, 64).cuda().requires_grad_()
    eager = moe.gate_from_logits(leaf, 4, score="sigmoid")  # a graph of the same leaf that stays alive
    dw, count = torch.randn(50, 4, device="cuda"), torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        count += 1
        with pytest.raises(RuntimeError, match="captured"):
            moe.gate_from_logits(leaf, 4, score="sigmoid")
        with torch.no_grad():
            r = moe.gate_from_logits(leaf, 4, score="sigmoid")
            grad = moe.gate_backward(leaf, r["idx"], dw, score="sigmoid")
    for i in range(3):
        with torch.no_grad():
            leaf.copy_(logits_of(10 + i, 50, 64))
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            now = moe.gate_from_logits(leaf, 4, score="sigmoid")
        assert torch.equal(r["idx"], now["idx"]) and torch.equal(r["w"], now["w"])
        assert torch.equal(grad, moe.gate_backward(leaf, now["idx"], dw, score="sigmoid"))
    assert int(count) == 3 and eager["w"].requires_grad


def test_calls_without_a_backward_pass_refuse():
    c = {n: t.cuda() for n, t in make(3, 12, 64, 32, 3, 8).items()}
    c["scale"] = torch.ones(3, device="cuda")
    for n in ("x", "base", "a", "b", "scale"):
        d = {**c, n: c[n].clone().requires_grad_()}
        with pytest.raises(RuntimeError, match="no backward"):
            moe.lora_add(**d)
        with torch.no_grad():
            assert not moe.lora_add(**d).requires_grad
    inp = mi.make_inputs("decode_b1", T=2, H=512, E=16, I=256)
    dev = Dev(inp)
    wr = dev.wr.clone().requires_grad_()
    logits = torch.randn(2, 16, device="cuda", requires_grad=True)
    for call in (lambda: moe.gate(dev.x, wr, 4),
                 lambda: moe.layer_forward_gated(dev.x, wr, inp.k, dev.down, gate_up=dev.gate_up),
                 lambda: moe.layer_forward_gated(dev.x, None, inp.k, dev.down, gate_up=dev.gate_up, logits=logits)):
        with pytest.raises(RuntimeError, match="no backward"):
            call()
        with torch.no_grad():
            call()
    torch.cuda.synchronize()
