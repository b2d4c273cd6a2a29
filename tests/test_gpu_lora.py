"""Per-request low-rank adapters on the GPU against 64-bit numpy, and the run of
adapters on the router, gate and experts.

u = 2^-24.  Bounds, against the sums over absolute values `mag` (of products)
and `vmag` (of B times the ranks' values): x A^T adds K exact products in fp32
(K u mag, and two roundings for partial sums and scale each split), v reaches
the matrix cores with 2^-17 (bf16 adapters, 16-bit output) or 2^-21 (fp16, or
fp32 output) of its value left out, and the second product adds at most
3 R + 2 terms; the output is rounded once.
"""
import numpy as np
import pytest
import torch

import mixture_experts_router_amd as moe
import moe_inputs as mi
import oracle
from gate_ref64 import lora64, select64, weights64
from gpu_util import Dev, assert_within_tolerance, host_bits

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(seed, T, K, N, L, R, dtype="bf16", out="same"):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=n(T, K).to(dt), base=n(T, N).to(dt if out == "same" else TYPES[out]),
                ids=torch.randint(-1, L, (T,), generator=g, dtype=torch.int32), a=(n(L, R, K) / K ** 0.5).to(dt),
                b=(n(L, N, R) / R ** 0.5).to(dt))


def call(c, **kw):
    return moe.lora_add(*(c[n].cuda() for n in ("x", "base", "ids", "a", "b")),
                        **{k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()})


def check(c, scale=None, ranks=None, got=None):
    got = call(c, scale=scale, ranks=ranks) if got is None else got
    torch.cuda.synchronize()
    K, R, dt = c["x"].shape[1], c["a"].shape[1], c["base"].dtype
    assert got.dtype == dt
    want, mag, vmag = lora64(f64(c["x"]), f64(c["base"]), c["ids"].numpy(), f64(c["a"]), f64(c["b"]),
                             None if scale is None else f64(scale), None if ranks is None else ranks.numpy())
    left = 2.0 ** -17 if c["x"].dtype == torch.bfloat16 and dt != torch.float32 else 2.0 ** -21
    tol = (K + 3 * R + 64) * 2.0 ** -24 * (mag + np.abs(want)) + left * vmag
    if dt != torch.float32:
        tol += torch.finfo(dt).eps / 2 * (np.abs(want) + tol)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol + 1e-37), float((err - tol).max())
    same = (c["ids"] < 0) | (c["ids"] >= c["a"].shape[0])
    assert torch.equal(got.cpu()[same], c["base"][same])
    return got


@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 64, 65, 200])
@pytest.mark.parametrize("K,N,L,R", [(64, 32, 1, 8), (8, 1, 3, 16), (520, 33, 5, 24), (1000, 100, 7, 32),
                                     (256, 264, 2, 64), (192, 77, 4, 128), (1024, 512, 70, 16), (128, 40, 3, 40),
                                     (136, 48, 2, 104)])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("f16", "same"), ("bf16", "f32"), ("f16", "f32")])
def test_sizes(T, K, N, L, R, dtype, out):
    check(make(T + K, T, K, N, L, R, dtype, out))


@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_whole_numbers_are_exact(dtype, out, R):
    """Small whole numbers: every product and sum is exact (|v| <= 3 K < 2^16, two parts of 8 bits hold it; the results
    are whole and a 16-bit output rounds each once), so any lane, row or column that is misplaced shows."""
    T, K, N, L = 150, 200, 72, 6
    g = torch.Generator().manual_seed(R)
    i = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()  # noqa: E731
    dt = TYPES[dtype]
    c = dict(x=i(-1, 1, T, K).to(dt), base=i(-9, 9, T, N).to(dt if out == "same" else TYPES[out]),
             ids=torch.randint(-1, L, (T,), generator=g, dtype=torch.int32), a=i(-3, 3, L, R, K).to(dt),
             b=i(-2, 2, L, N, R).to(dt))
    got = call(c)
    want, _, _ = lora64(f64(c["x"]), f64(c["base"]), c["ids"].numpy(), f64(c["a"]), f64(c["b"]))
    assert np.array_equal(f64(got), f64(torch.from_numpy(want).to(c["base"].dtype)))


@pytest.mark.parametrize("ids", [[5] * 130, list(range(64)) + list(range(64)), [0] * 63 + [1] + [2] * 66,
                                 [-1] * 130, [-7, 64, 1 << 30, 3] * 40, [1, 0] * 65, [9]])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_orders_of_adapters(ids, dtype):
    c = make(len(ids), len(ids), 320, 96, 64, 16, dtype)
    c["ids"] = torch.tensor(ids, dtype=torch.int32)
    check(c, scale=torch.linspace(0.25, 2.0, 64))


@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("f16", "same"), ("bf16", "f32")])
def test_ranks_leave_the_rest_unread(R, dtype, out):
    """Rows and columns from the rank on hold NaN and infinities; rank 0 adds nothing; ranks are taken into [0, R]."""
    L = 9
    c = make(R, 90, 144, 50, L, R, dtype, out)
    ranks = torch.tensor([0, 1, 3, R // 2, R - 1, R, R + 5, -4, 7], dtype=torch.int32)
    for i in range(L):
        r = min(max(int(ranks[i]), 0), R)
        c["a"][i, r:] = torch.nan
        c["b"][i, :, r:] = torch.inf
    check(c, ranks=ranks)


def test_nan_in_one_row_stays_there():
    c = make(3, 100, 128, 64, 3, 16)
    c["x"][10] = torch.nan
    c["base"][20] = torch.inf
    clean = make(3, 100, 128, 64, 3, 16)
    got, want = call(c).cpu(), call(clean).cpu()
    keep = torch.ones(100, dtype=torch.bool)
    keep[[10, 20]] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("R", [8, 16, 24, 40, 128])
@pytest.mark.parametrize("dtype,out", [("bf16", "same"), ("f16", "same"), ("bf16", "f32"), ("f16", "f32")])
def test_infinities_are_not_spread_by_unused_ranks(R, dtype, out):
    """With positive adapters an infinite x gives an infinite row, whatever the tile's unused ranks hold; an adapter of
    rank 0 adds nothing to it, and nothing of an infinite scale."""
    c = make(8, 20, 72, 40, 3, R, dtype, out)
    c["a"], c["b"] = c["a"].abs() + 0.125, c["b"].abs() + 0.125
    c["ids"] = torch.arange(20, dtype=torch.int32) % 3
    c["x"][3, 5], c["x"][7, 71], c["x"][5, 0] = torch.inf, -torch.inf, torch.inf
    got = call(c, ranks=torch.tensor([R, R - 3, 0], dtype=torch.int32), scale=torch.tensor([1.0, 2.0, torch.inf])).cpu()
    assert torch.all(got[3] == torch.inf) and torch.all(got[7] == -torch.inf)
    none = c["ids"] == 2
    assert torch.equal(got[none], c["base"][none])
    rest = ~none
    rest[[3, 7]] = False
    assert torch.all(torch.isfinite(got[rest]))


@pytest.mark.parametrize("power", [-30, 14])
def test_fp16_values_beyond_its_range(power):
    """x A^T outside fp16's range (and far below it) still reaches the fp32 output."""
    c = make(4, 40, 64, 48, 2, 16, "f16", "f32")
    c["x"] = (c["x"].float().clamp(-3, 3) * 2.0 ** min(power, 0)).to(torch.float16) if power < 0 else c["x"]
    scale = torch.tensor([2.0 ** power, 2.0 ** power])
    c["base"].zero_()
    check(c, scale=scale)


def test_strides_offsets_and_in_place():
    g = make(7, 70, 128, 64, 4, 16)
    x, base, ids, a, b = (g[n].cuda() for n in ("x", "base", "ids", "a", "b"))
    want = moe.lora_add(x, base, ids, a, b)
    wide = torch.zeros(70, 200, dtype=x.dtype, device="cuda")
    for off in (0, 8, 3):  # 3: not aligned, copied
        wide[:, off:off + 128] = x
        assert torch.equal(moe.lora_add(wide[:, off:off + 128], base, ids, a, b), want)
    for ld, off in ((72, 0), (75, 1), (80, 8)):
        buf = torch.full((70, ld), 5.0, dtype=x.dtype, device="cuda")
        out = buf[:, off:off + 64]
        moe.lora_add(x, base, ids, a, b, out=out)
        assert torch.equal(out, want) and torch.all(buf[:, :off] == 5) and torch.all(buf[:, off + 64:] == 5)
        buf[:, off:off + 64] = base
        assert moe.lora_add(x, out, ids, a, b, out=out) is out
        assert torch.equal(out, want) and torch.all(buf[:, :off] == 5) and torch.all(buf[:, off + 64:] == 5)
    t = torch.empty(64, 70, dtype=x.dtype, device="cuda").t()
    t.copy_(base)
    assert torch.equal(moe.lora_add(x, t, ids, a, b), want)
    assert moe.lora_add(x[:0], base[:0], ids[:0], a, b).shape == (0, 64)


def test_rows_without_an_adapter_are_left_alone_in_place():
    g = make(9, 40, 64, 32, 3, 8)
    g["ids"][::3] = -1
    base = g["base"].clone()
    base[::3] = torch.nan
    dev = base.cuda()
    bits = dev.view(torch.int16).clone()
    moe.lora_add(g["x"].cuda(), dev, g["ids"].cuda(), g["a"].cuda(), g["b"].cuda(), out=dev)
    assert torch.equal(dev.view(torch.int16)[::3], bits[::3])


def test_long_batches_and_repeats_are_identical():
    c = make(1, 5000, 256, 128, 6, 32)
    c["ids"] = torch.repeat_interleave(torch.tensor([4, -1, 0, 5, 2], dtype=torch.int32), 1000)
    first = check(c)
    for _ in range(3):
        assert torch.equal(call(c), first)


def test_streams_and_graph_replays():
    c = make(5, 96, 512, 256, 8, 32)
    d = {n: c[n].cuda() for n in c}
    want = moe.lora_add(**d)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:  # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        got.append(moe.lora_add(**d, stream=s))
    for s in sides:
        s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.lora_add(**d, out=out)
    for i in range(4):
        n = make(50 + i, 96, 512, 256, 8, 32)
        d["x"].copy_(n["x"])
        d["ids"].copy_(n["ids"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, moe.lora_add(**d))


def test_argument_errors():
    c = {n: t.cuda() for n, t in make(2, 6, 64, 32, 3, 8).items()}
    for change, err in (
        (dict(x=c["x"].float()), TypeError), (dict(base=c["base"].half()), TypeError), (dict(a=c["a"].half()), TypeError),
        (dict(b=c["b"][:, :31]), ValueError), (dict(a=c["a"][:2]), None), (dict(ids=c["ids"].long()), TypeError),
        (dict(ids=c["ids"][:5]), ValueError), (dict(ids=c["ids"].cpu()), ValueError), (dict(base=c["base"][:5]), ValueError),
        (dict(scale=torch.zeros(2, device="cuda")), ValueError), (dict(ranks=torch.zeros(3, device="cuda")), TypeError),
        (dict(out=c["base"].float()), TypeError), (dict(out=c["base"][:, :31]), ValueError),
        (dict(a=c["a"][:, :4], b=c["b"][:, :, :4]), ValueError),
        (dict(a=c["a"][:, :4].contiguous(), b=c["b"][:, :, :4].contiguous()), moe.MoeError),
    ):
        with pytest.raises(ValueError if err is None else err):
            moe.lora_add(**{**c, **change})


def test_rows_past_32_bit_offsets():
    """Rows 2^22 elements apart (the widest), 1100 of them, and an output 2^23 apart: byte offsets to 2^34; what lies
    between x's rows is NaN and what lies between out's stays."""
    T, K, N = 1100, 64, 40
    c = make(12, T, K, N, 4, 16)
    want = call(c)
    x = torch.full((T, 1 << 22), torch.nan, dtype=torch.bfloat16, device="cuda")[:, 8:8 + K]
    x.copy_(c["x"])
    out = torch.full((T, 1 << 23), 3.0, dtype=torch.bfloat16, device="cuda")
    ids, a, b = (c[n].cuda() for n in ("ids", "a", "b"))
    moe.lora_add(x, c["base"].cuda(), ids, a, b, out=out[:, 1:1 + N])
    assert torch.equal(out[:, 1:1 + N], want)
    assert torch.all(out[:, 0] == 3) and torch.all(out[:, 1 + N:1 + 2 * N] == 3)


def test_adapters_past_32_bit_offsets():
    """The last of 2100 adapters lies 2^32 bytes from the first."""
    L, K, N, R = 2100, 8192, 8192, 128
    a = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    c = make(13, 20, K, N, 1, R)
    a[L - 1].copy_(c["a"][0])
    b[L - 1].copy_(c["b"][0])
    last = torch.full((20,), L - 1, dtype=torch.int32, device="cuda")
    c["ids"] = torch.zeros(20, dtype=torch.int32)
    assert torch.equal(moe.lora_add(c["x"].cuda(), c["base"].cuda(), last, a, b), call(c))


def test_sixteen_bit_rows_of_a_long_batch():
    """20000 tokens (313 chunks, one workgroup each) in runs, every 64 of them the same as alone."""
    n, times = 64, 313
    c = make(14, n, 128, 96, 5, 32)
    one = call(c)
    d = {m: c[m].cuda() for m in c}
    many = moe.lora_add(d["x"].repeat(times, 1), d["base"].repeat(times, 1), d["ids"].repeat(times), d["a"], d["b"])
    assert torch.all(many.view(times, n, 96) == one)


def test_views_of_one_buffer_add_in_place():
    """base and out as two views of the same rows are the in-place form."""
    c = {n: t.cuda() for n, t in make(15, 33, 64, 24, 3, 8).items()}
    want = moe.lora_add(**c)
    buf = torch.zeros(33, 40, dtype=torch.bfloat16, device="cuda")
    buf[:, 8:32] = c["base"]
    c["base"] = buf[:, 8:32]
    moe.lora_add(**c, out=buf[:, 8:32])
    assert torch.equal(buf[:, 8:32], want) and torch.all(buf[:, :8] == 0) and torch.all(buf[:, 32:] == 0)


# ------------------------------------- adapters on the router, gate, experts


@pytest.mark.parametrize("recipe,kw,flags,capacity", [
    ("decode_b1", dict(T=3, H=1024, E=16, I=704), 0, 0),
    ("decode_b1", dict(T=2, H=512, E=32, I=256), moe.FLAG_UNFUSED, 0),
    ("prefill", dict(T=150, H=512, E=16, I=192), moe.FLAG_FORCE_MFMA, 0),
    ("prefill", dict(T=150, H=512, E=64, I=192), 0, 24),
    ("batched_decode", dict(T=40, H=512, E=32, I=256), 0, 0),
])
def test_adapted_router_gate_and_layer(recipe, kw, flags, capacity):
    """Per-request adapters on the shared router's logits, the gate with groups and a bias, and the experts: each
    step against its reference on the step before, the layer against the oracle under the gate's routing."""
    inp = mi.make_inputs(recipe, **kw)
    dev = Dev(inp)
    T, E, H, k = inp.T, inp.E, inp.H, inp.k
    c = make(3, T, H, E, 4, 8, inp.dtype, "f32")
    bias = torch.linspace(-0.2, 0.2, E).cuda()
    opts = dict(score="sigmoid", groups=8, group_k=4, group_best=2, scale=1.5)
    r = moe.gate(dev.x, dev.wr, k, bias=bias, want_logits=True, **opts)
    c["x"], c["base"] = dev.x.cpu(), r["logits"].cpu()
    logits = check(c)
    taps = moe.make_taps(T, E, k, inp.I, "cuda")
    y = moe.layer_forward_gated(dev.x, None, k, dev.down, gate_up=dev.gate_up, logits=logits, bias=bias, flags=flags,
                                taps=taps, capacity=capacity, **opts)
    torch.cuda.synchronize()
    assert ("gate" in moe.last_plan()) and ("router_logits" not in moe.last_plan())
    idx, w = taps["topk_idx"].cpu().numpy(), taps["topk_w"].cpu().numpy()
    want = select64(f64(logits), k, bias=f64(bias), **opts)
    assert np.array_equal(idx, want)
    assert np.allclose(w, weights64(f64(logits), want, **opts), rtol=2.0 ** -17, atol=0)
    assert torch.equal(taps["logits"], logits) and int(taps["k_used"]) == k
    gate_up = oracle.fuse_gate_up(inp.gate, inp.up)
    wk = w.copy()
    if capacity:
        seen = {}
        for p, e in enumerate(idx.ravel()):
            seen[e] = seen.get(e, 0) + 1
            if seen[e] > capacity:
                wk.ravel()[p] = 0.0
        assert (wk == 0).any()
    ref = oracle.tokens_forward(inp.x, inp.dtype, np.arange(T), idx, wk, k, gate_up, inp.down)
    assert_within_tolerance(host_bits(y), ref, inp.dtype, recipe)
    # the same layer with the router inside: the gate's own routing of the plain logits
    y2 = moe.layer_forward_gated(dev.x, dev.wr, k, dev.down, gate_up=dev.gate_up, bias=bias, flags=flags, taps=taps,
                                 capacity=capacity, **opts)
    assert torch.equal(taps["topk_idx"], r["idx"]) and torch.equal(taps["topk_w"], r["w"])
    y3 = moe.layer_forward_gated(dev.x, None, k, dev.down, gate_up=dev.gate_up, logits=r["logits"], bias=bias,
                                 flags=flags, capacity=capacity, **opts)
    assert np.array_equal(host_bits(y2), host_bits(y3))


def test_gated_layer_in_its_default_form_is_the_layer():
    """No options: the static top-k's experts, weights up to the order in which eight of them are summed."""
    inp = mi.make_inputs("prefill", T=90, H=512, E=16, I=192)
    dev = Dev(inp)
    a, b = (moe.make_taps(90, inp.E, inp.k, inp.I, "cuda", names=("topk_idx", "topk_w", "counts", "perm"))
            for _ in range(2))
    y = moe.layer_forward_gated(dev.x, dev.wr, inp.k, dev.down, gate_up=dev.gate_up, taps=a)
    z = moe.layer_forward(dev.x, dev.wr, inp.k, dev.down, gate_up=dev.gate_up, taps=b)
    for n in ("topk_idx", "counts", "perm"):
        assert torch.equal(a[n], b[n])
    assert torch.allclose(a["topk_w"], b["topk_w"], rtol=16 * 2.0 ** -24, atol=0)
    # weights within 2^-20: y differs by that and at most one rounding step of the output
    assert torch.all((y.float() - z.float()).abs() <= 2.0 ** -7 * z.float().abs() + 1e-6)


def test_gated_layer_replays_in_a_graph():
    inp = mi.make_inputs("prefill", T=60, H=512, E=16, I=192)
    dev = Dev(inp)
    need = moe.layer_workspace_size(60, 512, 16, inp.k, 192)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    logits = torch.randn(60, 16, device="cuda")
    out = torch.empty_like(dev.x)
    opts = dict(score="sigmoid", groups=4, group_k=2, group_best=1)
    run = lambda y, w: moe.layer_forward_gated(dev.x, None, inp.k, dev.down, gate_up=dev.gate_up, logits=logits, out=y,  # noqa: E731
                                               workspace=w, **opts)
    run(out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, ws)
    for i in range(4):
        logits.copy_(torch.randn(60, 16, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = host_bits(out)
        assert np.array_equal(got, host_bits(run(None, ws)))  # an eager call on the same workspace in between


def test_threads_calling_at_once():
    """Four host threads, each on a stream of its own: the calls share no state."""
    import threading
    c = {n: t.cuda() for n, t in make(21, 40, 256, 96, 5, 32, "bf16", "f32").items()}
    opts = dict(score="sigmoid", groups=8, group_k=4, group_best=2)
    want = moe.lora_add(**c)
    gate = moe.gate_from_logits(want, 6, **opts)
    grad = moe.gate_backward(want, gate["idx"], gate["w"], score="sigmoid")
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(40):
            y = moe.lora_add(**c, stream=s)
            r = moe.gate_from_logits(y, 6, stream=s, **opts)
            g = moe.gate_backward(y, r["idx"], r["w"], score="sigmoid", stream=s)
            s.synchronize()
            if not (torch.equal(y, want) and torch.equal(r["idx"], gate["idx"]) and torch.equal(g, grad)):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
