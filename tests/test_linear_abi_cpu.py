"""Refusals of the balance loss and the dense products, on the host: addresses are fake and every call returns before
the first HIP call (or, valid without a GPU, at the device check)."""
import pytest
import torch

import mixture_experts_router_amd as moe

P = 0x100000
F16, BF16, F32 = moe.MOE_F16, moe.MOE_BF16, moe.MOE_F32
BIG = 1 << 40


def bopts(score=0, seqs=1, offsets=None, mask=None):
    return moe.CBalanceOpts(score, seqs, offsets, mask)


def balance(o=None, logits=P, lt=F32, ld=None, T=4, E=32, k=4, idx=P, loss=P, z=None, prob=P, counts=P, tokens=P,
            ws=P, n=BIG):
    return moe.lib().moe_balance_loss(logits, lt, E if ld is None else ld, T, E, k, idx, o, loss, z, prob, counts,
                                      tokens, ws, n, None)


def balance_grad(o=None, logits=P, lt=F32, ld=None, T=4, E=32, k=4, counts=P, tokens=P, gl=P, gz=None, out=P,
                 ldo=None):
    return moe.lib().moe_balance_loss_backward(logits, lt, E if ld is None else ld, T, E, k, o, counts, tokens, gl, gz,
                                               out, E if ldo is None else ldo, None)


BOTH = [
    (dict(lt=4), "MOE_ERR_DTYPE"), (dict(T=-1), "MOE_ERR_SHAPE"), (dict(T=(1 << 25) + 1), "MOE_ERR_SHAPE"),
    (dict(E=0, k=1), "MOE_ERR_SHAPE"), (dict(E=257), "MOE_ERR_SHAPE"), (dict(ld=31), "MOE_ERR_SHAPE"),
    (dict(k=0), "MOE_ERR_K"), (dict(k=9), "MOE_ERR_K"), (dict(E=3, k=4), "MOE_ERR_K"),
    (dict(logits=None), "MOE_ERR_NULL"), (dict(counts=None), "MOE_ERR_NULL"), (dict(tokens=None), "MOE_ERR_NULL"),
    (dict(logits=P + 2), "MOE_ERR_ALIGN"), (dict(logits=P + 1, lt=BF16), "MOE_ERR_ALIGN"),
    (dict(counts=P + 2), "MOE_ERR_ALIGN"), (dict(tokens=P + 1), "MOE_ERR_ALIGN"),
    (dict(o=bopts(score=2)), "MOE_ERR_OPTION"), (dict(o=bopts(seqs=0)), "MOE_ERR_OPTION"),
    (dict(o=bopts(seqs=2)), "MOE_ERR_OPTION"),  # several sequences without offsets
    (dict(o=bopts(seqs=(1 << 20) + 1, offsets=P)), "MOE_ERR_OPTION"), (dict(o=bopts(offsets=P + 2)), "MOE_ERR_ALIGN"),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(idx=None), "MOE_ERR_NULL"), (dict(loss=None), "MOE_ERR_NULL"), (dict(idx=P + 2), "MOE_ERR_ALIGN"),
    (dict(loss=P + 2), "MOE_ERR_ALIGN"), (dict(z=P + 2), "MOE_ERR_ALIGN"), (dict(prob=P + 2), "MOE_ERR_ALIGN"),
    (dict(o=bopts(score=1), z=P), "MOE_ERR_OPTION"), (dict(T=3000, ws=None), "MOE_ERR_WORKSPACE"),
    (dict(T=3000, n=0), "MOE_ERR_WORKSPACE"), (dict(T=3000, ws=P + 8), "MOE_ERR_ALIGN")])
def test_balance_loss_refuses(kw, status):
    assert moe.STATUS[balance(**kw)] == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(ldo=31), "MOE_ERR_SHAPE"), (dict(out=None), "MOE_ERR_NULL"), (dict(out=P + 2), "MOE_ERR_ALIGN"),
    (dict(gl=P + 2), "MOE_ERR_ALIGN"), (dict(gz=P + 2), "MOE_ERR_ALIGN"), (dict(o=bopts(score=1), gz=P),
                                                                          "MOE_ERR_OPTION")])
def test_balance_gradient_refuses(kw, status):
    assert moe.STATUS[balance_grad(**kw)] == status


def test_balance_workspace():
    size = moe.lib().moe_balance_workspace_size
    assert size(0, 32, 1) == 0 and size(-1, 32, 1) == 0 and size(4, 0, 1) == 0 and size(4, 257, 1) == 0
    assert size(4, 32, 0) == 0
    need = size(3000, 32, 5)
    assert moe.STATUS[balance(T=3000, o=bopts(seqs=5, offsets=P), n=need - 1)] == "MOE_ERR_WORKSPACE"
    assert moe.STATUS[balance(T=3000, o=bopts(seqs=5, offsets=P), n=need)] == "MOE_ERR_DEVICE"
    # about a thousand chunks at most
    assert size(1 << 25, 256, 1) <= 1100 * (2 * 256 + 4) * 4


def linear(x=P, dt=BF16, ldx=None, T=4, w=P, ldw=None, bias=None, bias_dt=F32, N=24, K=64, act=0, res=None, ldr=None,
           rs=None, pre=None, ldp=None, out=P, ldo=None, odt=BF16, ws=P, n=BIG, null=False):
    C = N // 2 if act == 5 else N
    d = None if null else moe.CDense(w, K if ldw is None else ldw, bias, bias_dt, N, K, act)
    return moe.lib().moe_linear(x, dt, K if ldx is None else ldx, T, d, res, C if ldr is None else ldr, rs, pre,
                                N if ldp is None else ldp, out, C if ldo is None else ldo, odt, ws, n, None)


def linear_grad(g=P, gdt=BF16, ldg=None, x=P, dt=BF16, ldx=None, T=4, w=P, ldw=None, N=24, K=64, act=0, pre=P,
                ldp=None, rs=None, gx=P, ldgx=None, gw=P, ldgw=None, gb=P, grs=None, ws=P, n=BIG, null=False):
    C = N // 2 if act == 5 else N
    d = None if null else moe.CDense(w, K if ldw is None else ldw, None, 0, N, K, act)
    return moe.lib().moe_linear_backward(g, gdt, C if ldg is None else ldg, x, dt, K if ldx is None else ldx, T, d, pre,
                                         N if ldp is None else ldp, rs, gx, K if ldgx is None else ldgx, gw,
                                         K if ldgw is None else ldgw, gb, grs, ws, n, None)


MAXC = 1 << 22
DENSE = [
    (dict(null=True), "MOE_ERR_NULL"), (dict(dt=F32), "MOE_ERR_DTYPE"), (dict(dt=0), "MOE_ERR_DTYPE"),
    (dict(T=-1), "MOE_ERR_SHAPE"), (dict(T=(1 << 25) + 1), "MOE_ERR_SHAPE"), (dict(K=0), "MOE_ERR_SHAPE"),
    (dict(K=4), "MOE_ERR_SHAPE"), (dict(K=12), "MOE_ERR_SHAPE"), (dict(K=MAXC + 8), "MOE_ERR_SHAPE"),
    (dict(N=0), "MOE_ERR_SHAPE"), (dict(N=MAXC + 1), "MOE_ERR_SHAPE"), (dict(N=25, act=5), "MOE_ERR_SHAPE"),
    (dict(act=6), "MOE_ERR_OPTION"), (dict(act=-1), "MOE_ERR_OPTION"),
    (dict(T=1 << 25, N=MAXC), "MOE_ERR_SHAPE"), (dict(T=1 << 25, K=MAXC), "MOE_ERR_SHAPE"),
    (dict(w=None), "MOE_ERR_NULL"), (dict(w=P + 8), "MOE_ERR_ALIGN"), (dict(ldw=56), "MOE_ERR_SHAPE"),
    (dict(ldw=68), "MOE_ERR_SHAPE"), (dict(ldw=MAXC + 8), "MOE_ERR_SHAPE"), (dict(x=None), "MOE_ERR_NULL"),
    (dict(x=P + 8), "MOE_ERR_ALIGN"), (dict(ldx=56), "MOE_ERR_SHAPE"), (dict(ldx=68), "MOE_ERR_SHAPE"),
    (dict(ldx=MAXC + 8), "MOE_ERR_SHAPE"), (dict(rs=P + 2), "MOE_ERR_ALIGN"), (dict(pre=P + 1), "MOE_ERR_ALIGN"),
    (dict(pre=P, ldp=23), "MOE_ERR_SHAPE"), (dict(pre=P, ldp=MAXC + 1), "MOE_ERR_SHAPE"),
]


@pytest.mark.parametrize("kw,status", DENSE + [
    (dict(odt=F16), "MOE_ERR_DTYPE"), (dict(bias=P, bias_dt=F16), "MOE_ERR_DTYPE"),
    (dict(bias=P + 2), "MOE_ERR_ALIGN"), (dict(bias=P + 1, bias_dt=BF16), "MOE_ERR_ALIGN"),
    (dict(out=None), "MOE_ERR_NULL"), (dict(out=P + 1), "MOE_ERR_ALIGN"), (dict(out=P + 2, odt=F32), "MOE_ERR_ALIGN"),
    (dict(ldo=23), "MOE_ERR_SHAPE"), (dict(ldo=11, act=5), "MOE_ERR_SHAPE"), (dict(ldo=MAXC + 1), "MOE_ERR_SHAPE"),
    (dict(res=P + 1), "MOE_ERR_ALIGN"), (dict(res=2 * P, ldr=23), "MOE_ERR_SHAPE"),
    (dict(res=P, ldr=32), "MOE_ERR_SHAPE")])  # in place, other rows
def test_linear_refuses(kw, status):
    assert moe.STATUS[linear(**kw)] == status


@pytest.mark.parametrize("kw,status", DENSE + [
    (dict(gdt=F16), "MOE_ERR_DTYPE"), (dict(g=None), "MOE_ERR_NULL"), (dict(g=P + 1), "MOE_ERR_ALIGN"),
    (dict(g=P + 2, gdt=F32), "MOE_ERR_ALIGN"), (dict(ldg=23), "MOE_ERR_SHAPE"), (dict(ldg=MAXC + 1), "MOE_ERR_SHAPE"),
    (dict(pre=None, act=2), "MOE_ERR_NULL"), (dict(pre=None, grs=P), "MOE_ERR_NULL"),
    (dict(gx=P + 1), "MOE_ERR_ALIGN"), (dict(ldgx=63), "MOE_ERR_SHAPE"), (dict(gw=P + 1), "MOE_ERR_ALIGN"),
    (dict(ldgw=63), "MOE_ERR_SHAPE"), (dict(gb=P + 2), "MOE_ERR_ALIGN"), (dict(grs=P + 2), "MOE_ERR_ALIGN"),
    (dict(ws=None), "MOE_ERR_WORKSPACE"), (dict(n=0), "MOE_ERR_WORKSPACE"), (dict(ws=P + 8), "MOE_ERR_ALIGN")])
def test_linear_gradient_refuses(kw, status):
    assert moe.STATUS[linear_grad(**kw)] == status


def test_what_is_not_read_may_be_missing():
    ok = "MOE_ERR_DEVICE"
    assert moe.STATUS[linear()] == ok and moe.STATUS[linear_grad()] == ok
    assert moe.STATUS[linear(res=P)] == ok  # in place
    assert moe.STATUS[linear(bias=P, bias_dt=BF16, odt=F32)] == ok
    assert moe.STATUS[linear(T=0, x=None, out=None, ws=None, n=0)] == "MOE_OK"
    assert moe.STATUS[linear_grad(gx=None, w=None)] == ok
    assert moe.STATUS[linear_grad(gw=None, x=None)] == ok
    assert moe.STATUS[linear_grad(pre=None)] == ok
    assert moe.STATUS[linear_grad(T=0, g=None, x=None, gx=None, pre=None)] == ok  # grad_w and grad_bias are written
    assert moe.STATUS[balance(T=0, logits=None, idx=None, ws=None, n=0)] == ok
    assert moe.STATUS[balance_grad(T=0, logits=None, counts=None, tokens=None, out=None)] == "MOE_OK"


def test_linear_workspaces():
    L = moe.lib()
    assert L.moe_linear_workspace_size(-1, 8, 8) == 0 and L.moe_linear_workspace_size(4, 0, 8) == 0
    need = L.moe_linear_backward_workspace_size(100, 24, 64)
    assert need >= 100 * 24 * 2
    assert moe.STATUS[linear_grad(T=100, n=need - 1)] == "MOE_ERR_WORKSPACE"
    assert moe.STATUS[linear_grad(T=100, n=need)] == "MOE_ERR_DEVICE"
    for T, N, K in ((64, 64, 4096), (777, 64, 4096), (1, 22016, 4096)):
        n = L.moe_linear_workspace_size(T, N, K)
        if n:
            assert moe.STATUS[linear(T=T, N=N, K=K, n=n - 1)] == "MOE_ERR_WORKSPACE"
        assert moe.STATUS[linear(T=T, N=N, K=K, n=n)] == "MOE_ERR_DEVICE"


def test_the_binding_refuses_tensors_on_the_host():
    x, w, l = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 8)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: moe.linear(x, w), lambda: moe.linear_backward(torch.zeros(4, 8), x, w),
                 lambda: moe.balance_loss(l, idx),
                 lambda: moe.balance_loss_backward(l, torch.zeros(1, 8, dtype=torch.int32), idx[:1, 0], None, 2)):
        with pytest.raises(ValueError, match="GPU"):
            call()
