"""Refusals of the gate and adapter entry points, on the host: addresses are fake
and every call returns before the first HIP call (or, valid without a GPU, at
the device check)."""
import ctypes

import pytest
import torch

import mixture_experts_router_amd as moe

P = 0x100000


def opts(score=0, bias=None, groups=0, group_k=0, group_best=1, renorm=1, scale=1.0, capacity=0):
    return moe.CGateOpts(score, bias, groups, group_k, group_best, renorm, scale, capacity)


def from_logits(o=None, logits=P, lt=moe.MOE_F32, ld=None, T=4, E=32, k=4, idx=P, w=P):
    return moe.lib().moe_gate_from_logits(logits, lt, E if ld is None else ld, T, E, k, o, idx, w, None)


def backward(o=None, logits=P, lt=moe.MOE_F32, ld=None, T=4, E=32, k=4, idx=P, dw=P, out=P, ldo=None):
    return moe.lib().moe_gate_backward(logits, lt, E if ld is None else ld, T, E, k, o, idx, dw, out,
                                       E if ldo is None else ldo, None)


BAD_SIZES = [
    (dict(lt=4), "MOE_ERR_DTYPE"), (dict(lt=0), "MOE_ERR_DTYPE"),
    (dict(T=-1), "MOE_ERR_SHAPE"), (dict(T=(1 << 25) + 1), "MOE_ERR_SHAPE"), (dict(E=0, k=1), "MOE_ERR_SHAPE"),
    (dict(E=257), "MOE_ERR_SHAPE"), (dict(ld=31), "MOE_ERR_SHAPE"), (dict(ld=0), "MOE_ERR_SHAPE"),
    (dict(k=0), "MOE_ERR_K"), (dict(k=9), "MOE_ERR_K"), (dict(E=3, k=4), "MOE_ERR_K"), (dict(k=-1), "MOE_ERR_K"),
    (dict(logits=None), "MOE_ERR_NULL"), (dict(idx=None), "MOE_ERR_NULL"),
    (dict(logits=P + 2), "MOE_ERR_ALIGN"), (dict(logits=P + 1, lt=moe.MOE_BF16), "MOE_ERR_ALIGN"),
    (dict(idx=P + 2), "MOE_ERR_ALIGN"),
]
BAD_OPTS = [
    (dict(score=2), "MOE_ERR_OPTION"), (dict(score=-1), "MOE_ERR_OPTION"), (dict(renorm=2), "MOE_ERR_OPTION"),
    (dict(scale=float("nan")), "MOE_ERR_OPTION"), (dict(scale=float("inf")), "MOE_ERR_OPTION"),
    (dict(bias=P + 2), "MOE_ERR_ALIGN"), (dict(groups=-1), "MOE_ERR_OPTION"),
    (dict(groups=5, group_k=2), "MOE_ERR_OPTION"),  # does not divide 32
    (dict(groups=8, group_k=0), "MOE_ERR_OPTION"), (dict(groups=8, group_k=9), "MOE_ERR_OPTION"),
    (dict(groups=16, group_k=1), "MOE_ERR_OPTION"),  # two experts cannot give four
    (dict(groups=8, group_k=2, group_best=0), "MOE_ERR_OPTION"),
    (dict(groups=8, group_k=2, group_best=3), "MOE_ERR_OPTION"),
    (dict(groups=32, group_k=8, group_best=2), "MOE_ERR_OPTION"),  # groups of one expert
    (dict(capacity=4), "MOE_ERR_OPTION"), (dict(capacity=-1), "MOE_ERR_OPTION"),
]


@pytest.mark.parametrize("kw,status", BAD_SIZES + [(dict(w=None), "MOE_ERR_NULL"), (dict(w=P + 1), "MOE_ERR_ALIGN")])
def test_gate_refuses_sizes(kw, status):
    assert moe.STATUS[from_logits(**kw)] == status


@pytest.mark.parametrize("kw,status", BAD_SIZES + [
    (dict(dw=None), "MOE_ERR_NULL"), (dict(out=None), "MOE_ERR_NULL"), (dict(ldo=31), "MOE_ERR_SHAPE"),
    (dict(out=P + 2), "MOE_ERR_ALIGN"), (dict(dw=P + 2), "MOE_ERR_ALIGN")])
def test_backward_refuses_sizes(kw, status):
    assert moe.STATUS[backward(**kw)] == status


@pytest.mark.parametrize("kw,status", BAD_OPTS)
def test_options_are_refused_by_every_entry_point(kw, status):
    o = opts(**kw)
    assert moe.STATUS[from_logits(o)] == status
    assert moe.STATUS[backward(o)] == status
    L = moe.lib()
    assert moe.STATUS[L.moe_gate(P, 1, 4, 64, P, 32, 4, o, P, P, P, None, 0, None)] == status


def test_groups_beyond_the_limit():
    o = opts(groups=128, group_k=128)
    assert moe.STATUS[from_logits(o, E=256)] == "MOE_ERR_OPTION"


def test_gate_refuses_what_the_router_refuses():
    L = moe.lib()
    g = lambda **kw: moe.STATUS[L.moe_gate(*[{**dict(x=P, dt=1, T=4, H=64, wr=P, E=32, k=4, o=None, idx=P, w=P,  # noqa: E731
                                                     lo=P, ws=None, n=0), **kw}[n] for n in
                                              ("x", "dt", "T", "H", "wr", "E", "k", "o", "idx", "w", "lo", "ws", "n")],
                                           None)]
    assert g(x=None) == "MOE_ERR_NULL" and g(wr=None) == "MOE_ERR_NULL" and g(idx=None) == "MOE_ERR_NULL"
    assert g(dt=3) == "MOE_ERR_DTYPE" and g(H=60) == "MOE_ERR_SHAPE" and g(k=moe.MOE_K_ENTROPY) == "MOE_ERR_K"
    assert g(lo=None) == "MOE_ERR_WORKSPACE"
    need = L.moe_gate_workspace_size(4, 32)
    assert need >= 4 * 32 * 4
    assert g(lo=None, ws=P, n=need - 1) == "MOE_ERR_WORKSPACE"
    assert g(lo=None, ws=P + 4, n=need) == "MOE_ERR_ALIGN"
    assert g(T=0, x=None, idx=None, w=None, lo=None) == "MOE_OK"


def test_zero_tokens_are_a_noop():
    assert from_logits(T=0, logits=None, idx=None, w=None) == 0
    assert backward(T=0, logits=None, idx=None, dw=None, out=None) == 0
    assert moe.STATUS[from_logits(opts(score=7), T=0)] == "MOE_ERR_OPTION"  # options are checked all the same


def W(E, N, K):
    return moe.CWeights(P, P, P, E, N, K, 4, 64, N, None)


def gated(wr=P, logits=None, o=None, T=4, E=8, k=2, x=P, y=P, ws=P, nbytes=None, dt=1):
    L = moe.lib()
    n = L.moe_layer_workspace_size(T, 256, E, k, 128, 0) if nbytes is None else nbytes
    return moe.STATUS[L.moe_layer_forward_gated(x, dt, T, 256, wr, logits, E, k, o, W(E, 256, 256), None, None,
                                                W(E, 256, 128), y, 0, None, ws, n, None)]


def test_gated_layer_refusals():
    assert gated(wr=P, logits=P) == "MOE_ERR_OPTION"
    assert gated(wr=None) == "MOE_ERR_NULL"
    assert gated(wr=None, logits=P + 2) == "MOE_ERR_ALIGN"
    assert gated(k=moe.MOE_K_ENTROPY) == "MOE_ERR_K"
    assert gated(o=opts(score=3)) == "MOE_ERR_OPTION"
    assert gated(o=opts(capacity=-1)) == "MOE_ERR_OPTION"
    assert gated(ws=None) == "MOE_ERR_WORKSPACE" and gated(nbytes=64) == "MOE_ERR_WORKSPACE"
    assert gated(T=0, x=None, y=None, ws=None, wr=None) == "MOE_OK"
    assert gated(T=0, x=None, y=None, ws=None, wr=None, logits=P + 4) == "MOE_OK"
    assert gated(dt=3) == "MOE_ERR_DTYPE"


def lora(x=P, dt=1, ldx=None, T=4, a=P, b=P, scale=None, ranks=None, L=3, R=16, K=64, N=48, ids=P, base=P, ldb=None,
         out=P + (1 << 16), ldo=None, odt=1):
    lib = moe.lib()
    return moe.STATUS[lib.moe_lora_add(x, dt, K if ldx is None else ldx, T, moe.CLora(a, b, scale, ranks, L, R, K, N),
                                       ids, base, N if ldb is None else ldb, out, N if ldo is None else ldo, odt,
                                       None)]


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), "MOE_ERR_NULL"), (dict(b=None), "MOE_ERR_NULL"), (dict(x=None), "MOE_ERR_NULL"),
    (dict(ids=None), "MOE_ERR_NULL"), (dict(base=None), "MOE_ERR_NULL"), (dict(out=None), "MOE_ERR_NULL"),
    (dict(dt=3), "MOE_ERR_DTYPE"), (dict(odt=2), "MOE_ERR_DTYPE"), (dict(odt=0), "MOE_ERR_DTYPE"),
    (dict(T=-1), "MOE_ERR_SHAPE"), (dict(L=0), "MOE_ERR_SHAPE"), (dict(K=60), "MOE_ERR_SHAPE"),
    (dict(K=0), "MOE_ERR_SHAPE"), (dict(N=0), "MOE_ERR_SHAPE"), (dict(R=12), "MOE_ERR_SHAPE"),
    (dict(R=0), "MOE_ERR_SHAPE"), (dict(R=136), "MOE_ERR_SHAPE"), (dict(ldx=56), "MOE_ERR_SHAPE"),
    (dict(ldx=68), "MOE_ERR_SHAPE"), (dict(ldb=47), "MOE_ERR_SHAPE"), (dict(ldo=0), "MOE_ERR_SHAPE"),
    (dict(out=P, ldo=56), "MOE_ERR_SHAPE"), (dict(x=P + 8), "MOE_ERR_ALIGN"), (dict(a=P + 8), "MOE_ERR_ALIGN"),
    (dict(b=P + 2), "MOE_ERR_ALIGN"), (dict(scale=P + 2), "MOE_ERR_ALIGN"), (dict(ranks=P + 1), "MOE_ERR_ALIGN"),
    (dict(ids=P + 2), "MOE_ERR_ALIGN"), (dict(base=P + 1), "MOE_ERR_ALIGN"), (dict(out=P + 1), "MOE_ERR_ALIGN"),
    (dict(odt=3, out=P + 2), "MOE_ERR_ALIGN"), (dict(ldx=(1 << 22) + 8), "MOE_ERR_SHAPE"),
    (dict(ldb=(1 << 22) + 1), "MOE_ERR_SHAPE"), (dict(K=(1 << 22) + 8), "MOE_ERR_SHAPE"),
    (dict(N=(1 << 22) + 8), "MOE_ERR_SHAPE"), (dict(T=(1 << 25) + 1), "MOE_ERR_SHAPE"),
])
def test_lora_refusals(kw, status):
    assert lora(**kw) == status


def test_lora_zero_tokens():
    assert lora(T=0, x=None, ids=None, base=None, out=None) == "MOE_OK"


@pytest.mark.skipif(torch.cuda.is_available(), reason="the device check passes on a GPU")
def test_valid_calls_reach_the_device_check():
    for st in (moe.STATUS[from_logits()], moe.STATUS[backward()], lora(), gated(), gated(wr=None, logits=P),
               moe.STATUS[from_logits(opts(1, P, 8, 4, 2), E=256, k=8)]):
        assert st == "MOE_ERR_DEVICE"


def test_binding_refuses_before_the_library():
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        moe.gate_from_logits(l, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.gate_backward(l, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        moe.lora_add(l.half(), l.half(), torch.zeros(4, dtype=torch.int32), l.half()[None], l.half()[None])


def test_structs_match_the_header_layout():
    assert ctypes.sizeof(moe.CGateOpts) == 40 and moe.CGateOpts.bias.offset == 8 and moe.CGateOpts.scale.offset == 32
    assert ctypes.sizeof(moe.CLora) == 48 and moe.CLora.L.offset == 32
