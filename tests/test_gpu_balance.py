"""The balance loss, the experts' counts and their gradient against 64 bits (bounds: balance_ref64)."""
import numpy as np
import pytest
import torch

import balance_ref64 as ref
import mixture_experts_router_amd as moe

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(seed, T, E, k, dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * 1.5 + 0.5 * torch.randn(E, generator=g)).to(TYPES[dtype])
    return l, torch.topk(l.float(), k, dim=1).indices.to(torch.int32)


def cuda(t):
    return None if t is None else t.cuda()


def check(l, idx, score, dtype="f32", offsets=None, mask=None, seed=0, dev=None):
    """Forward and backward of one input against 64 bits, and twice alike."""
    T, E = l.shape
    k = idx.shape[1]
    host = [None if t is None else t.numpy() for t in (offsets, mask)]
    want, bound = ref.balance(l.double().numpy(), idx.numpy(), score, *host)
    dl = l.cuda() if dev is None else dev
    kw = dict(score=score, offsets=cuda(offsets), mask=cuda(mask))
    got = moe.balance_loss(dl, idx.cuda(), **kw)
    assert set(got) == {"loss", "prob", "counts", "tokens"} | ({"z"} if score == "softmax" else set())
    for n, v in got.items():
        v = v.cpu().numpy()
        assert v.shape == want[n].shape
        if n in ("counts", "tokens"):
            assert v.dtype == np.int32 and np.array_equal(v, want[n]), n
            continue
        with np.errstate(over="ignore"):
            stored = want[n].astype(np.float32)  # beyond the type's largest value: infinite
        fine = np.isfinite(stored)
        assert np.array_equal(np.isnan(v), np.isnan(stored)), n
        assert np.array_equal(np.isinf(v), np.isinf(stored)), n
        assert np.all(np.abs(v - want[n])[fine] <= bound[n][fine]), (n, np.abs(v - want[n]).max())
    S = len(want["loss"])
    rng = np.random.default_rng(seed)
    scale = 1024.0 if dtype == "f16" else 1.0  # loss scaling
    gl = (rng.standard_normal(S) * scale).astype(np.float32)
    gz = (rng.standard_normal(S) * scale).astype(np.float32) if score == "softmax" else None
    t = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    grad = moe.balance_loss_backward(dl, got["counts"], got["tokens"], t(gl), k, grad_z=t(gz), **kw)
    assert grad.dtype == l.dtype
    wg, wb = ref.gradient(l.double().numpy(), want["counts"], want["tokens"], gl.astype(np.float64),
                          None if gz is None else gz.astype(np.float64), k, score, dtype, *host)
    g = grad.double().cpu().numpy()
    fine = np.isfinite(wg)
    assert np.array_equal(np.isnan(g), np.isnan(wg))
    off = np.abs(g - np.where(fine, wg, 0))
    assert np.all(off[fine] <= wb[fine]), (off[fine] / wb[fine]).max()
    again = moe.balance_loss(dl, idx.cuda(), **kw)
    assert all(torch.equal(again[n].nan_to_num(7.0), got[n].nan_to_num(7.0)) for n in got)
    return got, grad


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, "f32"), (1, 64, 4, "f32"), (2, 256, 8, "bf16"), (31, 5, 2, "f16"), (32, 65, 3, "f32"),
    (33, 128, 8, "bf16"), (512, 32, 2, "f32"), (777, 129, 6, "f16"), (1237, 160, 6, "bf16"), (1025, 255, 7, "f32"),
    (5000, 64, 4, "bf16"), (70001, 66, 2, "f32"), (40000, 256, 8, "f16")])
def test_one_sequence(T, E, k, dtype, score):
    l, idx = make(T + E, T, E, k, dtype)
    check(l, idx, score, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("borders", [
    [0, 300], [0, 0, 300], [0, 300, 300], [0, 1, 2, 3, 300], [5, 32, 64, 65, 290], [0, 31, 32, 33, 63, 64, 100, 300],
    [7, 7, 7, 7], [0, 0, 0, 150, 150, 150, 151, 151, 300], [299, 300], [300, 300, 300], list(range(301)),
    [0] * 90 + [10] * 70 + [200] * 80])
def test_sequences(borders, score):
    l, idx = make(len(borders), 300, 48, 4)
    check(l, idx, score, offsets=torch.tensor(borders, dtype=torch.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,S", [(4096, 3), (20000, 40), (65536, 16), (50001, 700)])
def test_long_ragged_batches(T, S, score):
    g = torch.Generator().manual_seed(T)
    border = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g)).values.to(torch.int32)
    mask = torch.rand(T, generator=g) < 0.8
    l, idx = make(S, T, 32, 2)
    check(l, idx, score, offsets=border, mask=mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_what_is_masked_is_not_looked_at(score):
    """Padding of NaN, infinities and wild indices; a sequence that is padding throughout."""
    l, idx = make(5, 200, 40, 4)
    mask = torch.zeros(200, dtype=torch.uint8)
    mask[:50] = 1
    mask[120:150] = 3  # any value but 0
    offsets = torch.tensor([0, 60, 110, 180], dtype=torch.int32)  # the second is not live at all
    for bad in (float("nan"), float("inf"), torch.finfo(torch.float32).min):
        l2, i2 = l.clone(), idx.clone()
        l2[mask == 0] = bad
        i2[mask == 0] = 1 << 30
        l2[180:], i2[180:] = bad, -5  # rows behind the last sequence
        got, grad = check(l2, i2, score, offsets=offsets, mask=mask)
        assert got["tokens"].tolist() == [50, 0, 30] and got["loss"][1] == 0 and torch.all(got["prob"][1] == 0)
        dead = mask == 0
        assert torch.all(grad[dead.cuda()] == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_experts_and_lost_rows(score, dtype):
    l, idx = make(6, 130, 50, 4, dtype)
    l[:, 7] = -np.inf  # an expert that no token may take
    l[3] = -np.inf  # a token that may take none
    l[9, 5:] = -np.inf
    idx[11, 1], idx[12, 0], idx[13, 2] = -1, 50, 1 << 30  # dropped pairs
    got, grad = check(l, idx, score, dtype)
    assert torch.all(grad[3] == 0) and torch.all(grad[:, 7] == 0) and got["prob"][0, 7] == 0
    assert int(got["counts"].sum()) == 130 * 4 - 3
    # the type's lowest value is a number, not a mask
    low = torch.finfo(TYPES[dtype]).min
    l2, i2 = make(7, 20, 12, 2, dtype)
    l2[:, 3] = low
    r = moe.balance_loss(l2.cuda(), i2.cuda(), score=score)
    assert bool(torch.isfinite(r["loss"]).all()) and r["prob"][0, 3] == 0
    l2[4] = low
    r = moe.balance_loss(l2.cuda(), i2.cuda(), score=score)
    assert bool(torch.isfinite(r["prob"]).all())


def test_nan_and_infinity_stay_in_their_sequence():
    l, idx = make(8, 90, 16, 2)
    l[10, 3], l[50, 2] = np.nan, np.inf
    l[10, 4] = -np.inf
    offsets = torch.tensor([0, 30, 60, 90], dtype=torch.int32)
    r = moe.balance_loss(l.cuda(), idx.cuda(), offsets=offsets.cuda())
    assert r["loss"].isnan().tolist() == [True, True, False]
    g = moe.balance_loss_backward(l.cuda(), r["counts"], r["tokens"], torch.ones(3, device="cuda"), 2,
                                  offsets=offsets.cuda())
    rows = g.isnan().any(1).nonzero().flatten().tolist()
    assert rows == [10, 50] and g[10, 4] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [40, 700])
def test_nan_reaches_every_expert_of_its_row_but_the_masked(T, score):
    """Also those whose exponential vanishes beside the row's maximum, or whose sigmoid is 0; compared element by
    element (sums, gradients and where they are NaN) with the formula."""
    l, idx = make(80, T, 70, 4)
    l[3, 5], l[3, 60] = np.inf, -np.inf
    l[9, 0], l[9, 8], l[9, 69] = np.nan, 3e38, -np.inf
    l[20] = -3e38
    l[20, 33] = 3e38
    if score == "softmax":
        l[21, 2] = 200.0  # the others vanish: 0, not NaN
    offsets = torch.tensor([0, 8, 15, T], dtype=torch.int32)
    got, grad = check(l, idx, score, offsets=offsets)
    inf = 69 if score == "softmax" else 0  # the sigmoid of +inf is 1
    assert [int(got["prob"][s].isnan().sum()) for s in range(3)] == [inf, 69, 0]
    assert [int(grad[t].isnan().sum()) for t in (3, 9, 20)] == [inf, 69, 0]


def test_rows_of_a_wider_tensor_and_outputs_in_place():
    l, idx = make(9, 300, 48, 4)
    for cols, at in ((64, 8), (61, 5)):  # aligned, and not
        wide = torch.full((300, cols), float("nan"), device="cuda")
        wide[:, at:at + 48] = l.cuda()
        got, grad = check(l, idx, "softmax", dev=wide[:, at:at + 48])
        out = torch.full((300, cols), 7.0, device="cuda")
        gl = torch.ones(1, device="cuda")
        plain = moe.balance_loss_backward(l.cuda(), got["counts"], got["tokens"], gl, 4)
        moe.balance_loss_backward(wide[:, at:at + 48], got["counts"], got["tokens"], gl, 4, out=out[:, at:at + 48])
        assert torch.equal(out[:, at:at + 48], plain)
        out[:, at:at + 48] = 7.0
        assert torch.all(out == 7.0)
    check(l.t().contiguous().t(), idx, "sigmoid")  # columns side by side: copied


def test_offsets_past_32_bits():
    T, ld = 40000, 120000  # 4.8e9 elements apart in all
    l, idx = make(10, T, 16, 2, "bf16")
    wide = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    wide[:, :16] = l.cuda()
    check(l, idx, "softmax", "bf16", dev=wide[:, :16])


def test_no_tokens():
    l, idx = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    for offsets in (None, torch.zeros(4, dtype=torch.int32, device="cuda")):
        r = moe.balance_loss(l, idx, offsets=offsets)
        assert all(bool((v == 0).all()) for v in r.values()) and r["loss"].numel() == (1 if offsets is None else 3)
    assert moe.balance_loss_backward(l, r["counts"], r["tokens"], r["loss"], 2, offsets=offsets).shape == (0, 8)


def test_offsets_out_of_order_stay_in_bounds():
    """Values are unspecified; the call and its neighbours in memory are not harmed."""
    l, idx = make(11, 500, 32, 2)
    for o in ([0, 400, 100, 500], [-9, 600, 200], [1 << 30, -(1 << 30), 77], [500, 0], [-5, -1, 900]):
        offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
        r = moe.balance_loss(l.cuda(), idx.cuda(), offsets=offsets)
        moe.balance_loss_backward(l.cuda(), r["counts"], r["tokens"], torch.ones(len(o) - 1, device="cuda"), 2,
                                  offsets=offsets)
    torch.cuda.synchronize()
    check(l, idx, "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """Central differences of the 64-bit loss: h^2 / 6 times a third derivative below 1, and 2^-52 |loss| / h."""
    l, idx = make(12, 6, 9, 2)
    leaf = l.cuda().requires_grad_()
    r = moe.balance_loss(leaf, idx.cuda(), score=score)
    total = r["loss"].sum() + (0.3 * r["z"].sum() if score == "softmax" else 0.0)
    total.backward()
    base, h = l.double().numpy(), 1e-4
    want = np.zeros((6, 9))
    for t in range(6):
        for e in range(9):
            v = []
            for d in (h, -h):
                m = base.copy()
                m[t, e] += d
                q, _ = ref.balance(m, idx.numpy(), score)
                v.append(q["loss"][0] + (0.3 * q["z"][0] if score == "softmax" else 0.0))
            want[t, e] = (v[0] - v[1]) / (2 * h)
    assert np.abs(leaf.grad.cpu().numpy() - want).max() < 1e-6


def test_autograd():
    l, idx = make(13, 64, 32, 4)
    offsets = torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
    plain = moe.balance_loss(l.cuda(), idx.cuda(), offsets=offsets)
    assert not plain["loss"].requires_grad
    leaf = l.cuda().requires_grad_()
    r = moe.balance_loss(leaf, idx.cuda(), offsets=offsets)
    assert all(torch.equal(r[n], plain[n]) for n in plain)
    assert r["loss"].requires_grad and r["z"].requires_grad and not r["prob"].requires_grad
    (r["loss"].mean() + 0.1 * r["z"].sum()).backward()
    half, tenth = torch.full((2,), 0.5, device="cuda"), torch.full((2,), 0.1, device="cuda")
    assert torch.equal(leaf.grad, moe.balance_loss_backward(l.cuda(), r["counts"], r["tokens"], half, 4, grad_z=tenth,
                                                            offsets=offsets))
    leaf.grad = None
    moe.balance_loss(leaf, idx.cuda(), score="sigmoid")["loss"].sum().backward()  # z has no part
    assert bool(torch.isfinite(leaf.grad).all())
    r = moe.balance_loss(leaf, idx.cuda())
    (g,) = torch.autograd.grad((r["loss"] ** 2).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    with torch.no_grad():
        assert not moe.balance_loss(leaf, idx.cuda())["loss"].requires_grad


def test_refusals():
    l, idx = (t.cuda() for t in make(14, 10, 16, 2))
    for bad, err in ((dict(score="tanh"), ValueError), (dict(offsets=torch.zeros(3, device="cuda")), TypeError),
                     (dict(offsets=torch.zeros(1, dtype=torch.int32, device="cuda")), ValueError),
                     (dict(offsets=torch.zeros(3, dtype=torch.int32)), ValueError),
                     (dict(mask=torch.ones(10, device="cuda")), TypeError),
                     (dict(mask=torch.ones(9, dtype=torch.bool, device="cuda")), ValueError)):
        with pytest.raises(err):
            moe.balance_loss(l, idx, **bad)
    with pytest.raises(ValueError):
        moe.balance_loss(l, idx[:9])
    with pytest.raises(TypeError):
        moe.balance_loss(l, idx.long())
    with pytest.raises(TypeError):
        moe.balance_loss(l.double(), idx)
    r = moe.balance_loss(l, idx)
    one = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        moe.balance_loss_backward(l, r["counts"][:, :8], r["tokens"], one, 2)
    with pytest.raises(moe.MoeError, match="MOE_ERR_OPTION"):
        moe.balance_loss_backward(l, r["counts"], r["tokens"], one, 2, grad_z=one, score="sigmoid")
    with pytest.raises(moe.MoeError, match="MOE_ERR_K"):
        moe.balance_loss_backward(l, r["counts"], r["tokens"], one, 9)


def test_streams_and_graphs():
    l, idx = make(15, 3000, 64, 4)
    side = torch.cuda.Stream()
    dl, di = l.cuda(), idx.cuda()
    one = torch.ones(1, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    r = moe.balance_loss(dl, di, stream=side)
    g = moe.balance_loss_backward(dl, r["counts"], r["tokens"], one, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = moe.balance_loss(dl, di)
    assert torch.equal(r["loss"], want["loss"])
    assert torch.equal(g, moe.balance_loss_backward(dl, want["counts"], want["tokens"], one, 4))
    leaf = dl.clone().requires_grad_()
    eager = moe.balance_loss(leaf, di)  # an eager graph of the leaf that stays alive
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            moe.balance_loss(leaf, di)
        with torch.no_grad():
            r = moe.balance_loss(leaf, di)
            g = moe.balance_loss_backward(leaf, r["counts"], r["tokens"], one, 4)
    for i in range(4):
        l2, i2 = make(20 + i, 3000, 64, 4)
        with torch.no_grad():
            leaf.copy_(l2)
        di.copy_(i2)
        graph.replay()
        want = moe.balance_loss(l2.cuda(), i2.cuda())
        assert all(torch.equal(r[n], want[n]) for n in want)
        assert torch.equal(g, moe.balance_loss_backward(l2.cuda(), want["counts"], want["tokens"], one, 4))
        torch.cuda.synchronize()
    del eager


def test_very_many_tokens_and_sequences():
    T = (1 << 24) + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    l = torch.randn(T, 4, generator=g, device="cuda")
    idx = torch.randint(0, 4, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    r = moe.balance_loss(l, idx)
    p = torch.softmax(l.double(), 1)
    counts = torch.bincount(idx.reshape(-1), minlength=4)
    prob, z = p.mean(0), (torch.logsumexp(l.double(), 1) ** 2).mean()
    # chunks of T / 512 tokens, 32 at a time: T / 16384 + 300 additions of positive terms, and 128 of a probability
    steps = (T / 16384 + 428) * ref.U
    assert torch.equal(r["counts"][0].long(), counts) and int(r["tokens"][0]) == T
    assert bool(((r["prob"][0].double() - prob).abs() <= steps * prob).all())
    assert abs(float(r["loss"][0]) - float(4 / (2 * T) * (counts.double() * prob).sum())) <= steps * 2
    assert abs(float(r["z"][0]) - float(z)) <= (steps + 300 * ref.U) * float(z) + 300 * ref.U
    one = torch.ones(1, device="cuda")
    d = moe.balance_loss_backward(l, r["counts"], r["tokens"], one, 2)
    slope = 4 / (2.0 * T * T) * counts.double()
    want = p * (slope - (p * slope).sum(1, keepdim=True))  # (a library product of so many rows is wrong at its end)
    assert bool(((d.double() - want).abs() <= 300 * ref.U * p * 2 * slope.max()).all())
    # a sequence for every token
    l, idx = make(16, 20000, 8, 2)
    check(l, idx, "softmax", offsets=torch.arange(20001, dtype=torch.int32))
