"""Cases that time the router's balance loss, dense products with fused epilogues, and their gradients.

Four operators of this package, each beside its plain form in elementary torch operations:

  balance           per sequence, the routed pairs of every expert (whole numbers), the mean routing probability of
                    every expert, loss = E / (k n) * sum_e counts_e * prob_e over the sequence's n tokens and, with
                    softmax scores, the mean squared logsumexp of its logits
  balance_backward  the gradient of both losses with respect to the logits, at fixed counts
  linear            out = residual + row_scale * act(x W^T + bias): the products of an expert that every token takes,
                    of a router with a bias, of a projection beside the layer; act may be the gated silu(g) * u
  linear_backward   the gradients of x, W and bias
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-20  # added to the sum of a token's sigmoid scores before it divides


def balance_case(name, op, T, E, k, score, dtype="f32", seqs=1, kind="one"):
    """kind: "one" sequence, sequences "packed" one after another with rows left over, or "padded" to one length."""
    return dict(name=name, op=op, T=T, E=E, k=k, score=score, dtype=dtype, seqs=seqs, kind=kind)


def linear_case(name, op, T, K, N, dtype, act="none", bias=False, residual=False, row_scale=False, out="same",
                train=False):
    """N: rows of W (the gated act gives N / 2 columns).  train: the forward pass also keeps x W^T + bias."""
    return dict(name=name, op=op, T=T, K=K, N=N, dtype=dtype, act=act, bias=bias, residual=residual,
                row_scale=row_scale, out=out, train=train)


def listed():
    return [
        # router fine-tuning on a small batch of a 32-expert layer: only latency counts
        balance_case("balance_512x32", "balance", 512, 32, 2, "softmax"),
        # a packed batch of ragged sequences over 160 experts, bf16 logits, with the squared logsumexp
        balance_case("balance_1237x160_packed", "balance", 1237, 160, 6, "softmax", "bf16", 9, "packed"),
        # a training step's tokens over 256 experts: 16 sequences padded to 4096 tokens, sigmoid scores
        balance_case("balance_65536x256_padded", "balance", 65536, 256, 8, "sigmoid", "f32", 16, "padded"),
        # the gradients of the first, and of a step's packed tokens
        balance_case("balance_grad_512x32", "balance_backward", 512, 32, 2, "softmax"),
        balance_case("balance_grad_65536x256", "balance_backward", 65536, 256, 8, "softmax", "f32", 16,
                     "packed"),
        # one new token through the gate and up projections of an expert that every token takes
        linear_case("linear_1x4096_swiglu", "linear", 1, 4096, 2 * 11008, "f16", "swiglu"),
        # a decode batch's down projection: each token's own weight, added to what its routed experts gave
        linear_case("linear_64x2816_down", "linear", 64, 2816, 4096, "bf16", residual=True, row_scale=True),
        # a ragged prompt through a projection with a bias
        linear_case("linear_777x4096_gelu", "linear", 777, 4096, 2816, "bf16", "gelu", bias=True),
        # a training step's gate and up projections, keeping what the gradient needs
        linear_case("linear_4096x4096_swiglu", "linear", 4096, 4096, 2 * 1408, "bf16", "swiglu", train=True),
        # a prefill's down projection added to the residual stream
        linear_case("linear_4096x11008_down", "linear", 4096, 11008, 4096, "bf16", residual=True),
        # router training: fp32 gradients of 64 logits a token
        linear_case("linear_grad_4096x64_router", "linear_backward", 4096, 4096, 64, "bf16", bias=True, out="f32"),
        # the gradients of the training step's gate and up projections
        linear_case("linear_grad_4096x4096_swiglu", "linear_backward", 4096, 4096, 2 * 1408, "bf16", "swiglu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("balance", "balance_backward", "linear", "linear", "linear_backward"))
    if op.startswith("balance"):
        T, E = _log_int(rng, 1, 65536), rng.randint(4, 256)
        kind = rng.choice(("one", "packed", "padded"))
        seqs = 1 if kind == "one" else _log_int(rng, 1, max(1, min(64, T // 2)))
        if kind == "padded":
            T = max(1, T // seqs) * seqs
        c = balance_case(None, op, T, E, rng.randint(1, min(8, E)), rng.choice(("softmax", "sigmoid")),
                         rng.choice(("f32", "f32", "f16", "bf16")), seqs, kind)
    else:
        act = rng.choice(("none", "none", "relu", "silu", "gelu", "sigmoid", "swiglu"))
        T, K = _log_int(rng, 1, 4096), 8 * _log_int(rng, 8, 512)
        N = 2 * _log_int(rng, 8, 2048) if act == "swiglu" else _log_int(rng, 16, 4096)
        c = linear_case(None, op, T, K, N, rng.choice(("f16", "bf16", "bf16")), act, rng.random() < 0.5,
                        op == "linear" and rng.random() < 0.5, rng.random() < 0.3, rng.choice(("same", "same", "f32")),
                        op == "linear" and rng.random() < 0.3)
    del c["name"]
    return c


def _columns(case):
    return case["N"] // 2 if case["act"] == "swiglu" else case["N"]


def _out_type(case):
    return case["dtype"] if case["out"] == "same" else case["out"]


def prepare(case, seed):
    """What a user's program holds before the call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DTYPES[case["dtype"]]
    if case["op"].startswith("balance"):
        return _prepare_balance(case, g, rand, dt)
    T, K, N, C = case["T"], case["K"], case["N"], _columns(case)
    odt = DTYPES[_out_type(case)]
    s = dict(case=case, x=rand(T, K).to(dt), w=(rand(N, K) / math.sqrt(K)).to(dt),
             bias=0.1 * rand(N) if case["bias"] else None,
             row_scale=torch.rand(T, generator=g, device="cuda") if case["row_scale"] else None)
    if case["op"] == "linear":
        s["residual"] = rand(T, C).to(odt) if case["residual"] else None
        return s
    s["grad"] = rand(T, C).to(odt)
    # what the forward pass kept; of a plain product nothing is needed but with row_scale
    z = s["x"].float() @ s["w"].float().T
    z = z if s["bias"] is None else z + s["bias"]
    s["preact"] = z.to(dt) if case["act"] != "none" or case["row_scale"] else None
    return s


def _prepare_balance(case, g, rand, dt):
    T, E, S = case["T"], case["E"], case["seqs"]
    logits = (rand(T, E) * 1.5 + rand(E) * 0.5).to(dt)
    s = dict(case=case, logits=logits, offsets=None, mask=None)
    s["idx"] = torch.topk(logits.float() + 0.1 * rand(E), case["k"], dim=1).indices.to(torch.int32)
    if case["kind"] == "packed":  # borders fall anywhere; the batch's last rows belong to no sequence
        end = T - T // 16
        border = torch.sort(torch.randint(0, end + 1, (S - 1,), generator=g, device="cuda")).values
        ends = torch.tensor([0, end], device="cuda")
        s["offsets"] = torch.cat((ends[:1], border, ends[1:])).to(torch.int32)
    elif case["kind"] == "padded":
        n = T // S
        s["offsets"] = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
        length = torch.randint((n + 1) // 2, n + 1, (S,), generator=g, device="cuda")
        s["mask"] = (torch.arange(n, device="cuda")[None, :] < length[:, None]).reshape(T)
    if case["op"] == "balance_backward":
        seq, live = _sequences(s)
        s["counts"], s["tokens"] = _counts(s, seq, live), _tokens(case, seq, live)
        # a coefficient of the loss, and the loss scaling that 16-bit floats of so small an exponent need
        scale = (65536.0 if case["dtype"] == "f16" else 1.0) / S
        s["grad_loss"] = 0.01 * scale * (0.5 + torch.rand(S, generator=g, device="cuda"))
        softmax = case["score"] == "softmax"
        s["grad_z"] = 0.001 * scale * (0.5 + torch.rand(S, generator=g, device="cuda")) if softmax else None
    return s


# ------------------------------------------------------------ plain forms


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _erf_gelu(v):
    return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))


def _sequences(state):
    """The sequence of every token (S for none), and whether it takes part."""
    T, S = state["case"]["T"], state["case"]["seqs"]
    t = torch.arange(T, device=state["logits"].device)
    if state["offsets"] is None:
        return torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    seq = torch.searchsorted(state["offsets"].long(), t, right=True) - 1
    live = (seq >= 0) & (seq < S)
    if state["mask"] is not None:
        live &= state["mask"]
    return torch.where(live, seq, S), live


def _tokens(case, seq, live):
    tokens = torch.zeros(case["seqs"] + 1, dtype=torch.int32, device=seq.device)
    return tokens.index_add_(0, seq, live.to(torch.int32))[:-1]


def _counts(state, seq, live):
    S, E = state["case"]["seqs"], state["case"]["E"]
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=seq.device)
    at = seq[:, None] * E + state["idx"].long()
    counts.index_add_(0, at.reshape(-1), live[:, None].expand_as(at).reshape(-1).to(torch.int32))
    return counts.view(S + 1, E)[:-1]


def _scores(state):
    """Routing probabilities of every token, with what their gradient needs."""
    l = state["logits"].float()
    if state["case"]["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - m)
        z = e.sum(1, keepdim=True)
        return e / z, (m + torch.log(z))[:, 0]
    s = _sigmoid(l)
    total = s.sum(1, keepdim=True) + EPS
    return s / total, _sigmoid(-l)


def _balance(state):
    case = state["case"]
    S, E = case["seqs"], case["E"]
    seq, live = _sequences(state)
    p, lse = _scores(state)
    counts, tokens = _counts(state, seq, live), _tokens(case, seq, live)
    member = (seq[None, :] == torch.arange(S, device=seq.device)[:, None]).float()
    n = tokens.clamp(min=1).float()
    prob = member @ p / n[:, None]
    r = dict(loss=(counts.float() * prob).sum(1) * E / (case["k"] * n), prob=prob, counts=counts, tokens=tokens)
    if case["score"] == "softmax":
        r["z"] = (member @ (lse * lse)[:, None])[:, 0] / n
    return r


def _balance_backward(state):
    case = state["case"]
    seq, live = _sequences(state)
    p, more = _scores(state)
    n = state["tokens"].clamp(min=1).float()
    slope = state["counts"].float() * (state["grad_loss"] * case["E"] / (case["k"] * n * n))[:, None]
    at = seq.clamp(max=case["seqs"] - 1)
    g = slope[at]
    grad = p * (g - (g * p).sum(1, keepdim=True))
    if case["score"] == "sigmoid":
        grad = grad * more
    else:
        grad = grad + p * ((state["grad_z"] / n)[at] * 2.0 * more)[:, None]
    return torch.where(live[:, None], grad, 0.0).to(state["logits"].dtype)


def _act(act, z):
    """The activation of z, its slope, and (gated) the slope of the second half."""
    if act == "none":
        return z, None, None
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).float(), None
    if act == "sigmoid":
        s = _sigmoid(z)
        return s, s * _sigmoid(-z), None
    if act == "silu":
        s = _sigmoid(z)
        return z * s, s * (1.0 + z * _sigmoid(-z)), None
    if act == "gelu":
        slope = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return _erf_gelu(z), slope, None
    a, b = z.chunk(2, dim=1)
    s = _sigmoid(a)
    return a * s * b, s * (1.0 + a * _sigmoid(-a)) * b, a * s


def _linear(state):
    case, dt = state["case"], state["x"].dtype
    z = state["x"].float() @ state["w"].float().T
    if state["bias"] is not None:
        z = z + state["bias"]
    out = _act(case["act"], z)[0]
    if state["row_scale"] is not None:
        out = out * state["row_scale"][:, None]
    if state["residual"] is not None:
        out = out + state["residual"].float()
    out = out.to(DTYPES[_out_type(case)])
    return dict(out=out, preact=z.to(dt)) if case["train"] else dict(out=out)


def _linear_backward(state):
    case, dt, g = state["case"], state["x"].dtype, state["grad"].float()
    a = slope = gated = None
    if state["preact"] is not None:
        a, slope, gated = _act(case["act"], state["preact"].float())
    r = {}
    if state["row_scale"] is not None:
        r["row_scale"] = (g * a).sum(1)
        g = g * state["row_scale"][:, None]
    dz = g if slope is None else g * slope if gated is None else torch.cat((g * slope, g * gated), 1)
    r["x"] = (dz @ state["w"].float()).to(dt)
    r["w"] = (dz.T @ state["x"].float()).to(dt)
    if case["bias"]:
        r["bias"] = dz.sum(0)
    return r


def run(state):
    case = state["case"]
    if own:
        import mixture_experts_router_amd as moe
        if case["op"] == "balance":
            return moe.balance_loss(state["logits"], state["idx"], score=case["score"], offsets=state["offsets"],
                                    mask=state["mask"])
        if case["op"] == "balance_backward":
            return moe.balance_loss_backward(state["logits"], state["counts"], state["tokens"], state["grad_loss"],
                                             case["k"], grad_z=state["grad_z"], score=case["score"],
                                             offsets=state["offsets"], mask=state["mask"])
        if case["op"] == "linear":
            r = moe.linear(state["x"], state["w"], state["bias"], act=case["act"], residual=state["residual"],
                           row_scale=state["row_scale"], out_dtype=DTYPES[_out_type(case)],
                           want_preact=case["train"])
            return dict(out=r[0], preact=r[1]) if case["train"] else dict(out=r)
        want = ("x", "w") + (("bias",) if case["bias"] else ()) + (("row_scale",) if case["row_scale"] else ())
        return moe.linear_backward(state["grad"], state["x"], state["w"], act=case["act"], preact=state["preact"],
                                   row_scale=state["row_scale"], want=want)
    if case["op"] == "balance":
        return _balance(state)
    if case["op"] == "balance_backward":
        return _balance_backward(state)
    return _linear(state) if case["op"] == "linear" else _linear_backward(state)


def work(case):
    T, size = case["T"], BYTES[case["dtype"]]
    if case["op"].startswith("balance"):
        E, k, S = case["E"], case["k"], case["seqs"]
        read = T * E * size + (T if case["kind"] == "padded" else 0)
        if case["op"] == "balance":
            return dict(bytes=read + 4 * T * k + 8 * S * E, flops=5.0 * T * E)
        return dict(bytes=read + T * E * size + 4 * S * E, flops=8.0 * T * E)
    K, N, C, osize = case["K"], case["N"], _columns(case), BYTES[_out_type(case)]
    operands = T * K * size + N * K * size
    if case["op"] == "linear":
        kept = T * N * size if case["train"] else 0
        return dict(bytes=operands + T * C * osize * (2 if case["residual"] else 1) + kept, flops=2.0 * T * K * N)
    kept = T * N * size if case["act"] != "none" or case["row_scale"] else 0
    return dict(bytes=2 * operands + T * C * osize + kept, flops=4.0 * T * K * N)


# ---------------------------------------------------- definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    n = {key: v.double() for key, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    return _exact_balance(case, s, n) if case["op"].startswith("balance") else _exact_linear(case, s, n)


def _exact_balance(case, s, n):
    """Sequence by sequence, straight from the definition."""
    T, E, k, S, l = case["T"], case["E"], case["k"], case["seqs"], n["logits"]
    softmax = case["score"] == "softmax"
    border = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=l.device)  # noqa: E731
    loss, z, prob, grad = zeros(S), zeros(S), zeros(S, E), zeros(T, E)
    counts = torch.zeros(S, E, dtype=torch.int32, device=l.device)
    tokens = torch.zeros(S, dtype=torch.int32, device=l.device)
    for q in range(S):
        rows = torch.arange(border[q], border[q + 1], device=l.device)
        if s["mask"] is not None:
            rows = rows[s["mask"][rows]]
        m = int(rows.numel())
        if m == 0:
            continue
        v = l[rows]
        score = torch.softmax(v, 1) if softmax else torch.sigmoid(v)
        total = score.sum(1, keepdim=True) + (0.0 if softmax else EPS)
        p, lse = score / total, torch.logsumexp(v, 1)
        counts[q] = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=E).to(torch.int32)
        tokens[q], prob[q], z[q] = m, p.mean(0), (lse * lse).mean()
        loss[q] = E / (k * m) * torch.dot(counts[q].double(), prob[q])
        if case["op"] == "balance_backward":
            f = n["grad_loss"][q] * E / (k * m * m) * counts[q].double()
            d = f[None, :] - (p @ f)[:, None]
            grad[rows] = p * d if softmax else p * (1.0 - score) * d
            if softmax:
                grad[rows] += n["grad_z"][q] * 2.0 / m * lse[:, None] * p
    if case["op"] == "balance_backward":
        return grad
    r = dict(loss=loss, prob=prob, counts=counts, tokens=tokens)
    return dict(r, z=z) if softmax else r


def _exact_linear(case, s, n):
    act = {"none": lambda v: v, "relu": torch.relu, "sigmoid": torch.sigmoid, "gelu": torch.nn.functional.gelu,
           "silu": torch.nn.functional.silu,
           "swiglu": lambda v: torch.nn.functional.silu(v[:, ::2]) * v[:, 1::2]}[case["act"]]
    N, gated = case["N"], case["act"] == "swiglu"
    # pairs of gate and up columns side by side
    order = torch.arange(N, device="cuda").view(2, N // 2).T.reshape(-1) if gated else torch.arange(N, device="cuda")
    back = torch.argsort(order)
    x, w = n["x"], n["w"]
    rs = n["row_scale"][:, None] if s["row_scale"] is not None else 1.0
    if case["op"] == "linear":
        z = x.matmul(w.t())
        if s["bias"] is not None:
            z += n["bias"]
        out = rs * act(z[:, order])
        if s["residual"] is not None:
            out = out + n["residual"]
        return dict(out=out, preact=z) if case["train"] else dict(out=out)
    r, dz = {}, rs * n["grad"]
    if s["preact"] is not None:
        with torch.enable_grad():
            z = n["preact"][:, order].requires_grad_(True)
            a = act(z)
            if s["row_scale"] is not None:
                r["row_scale"] = (n["grad"] * a).sum(1).detach()
            dz = torch.autograd.grad(a, z, rs * n["grad"])[0][:, back]
    r["x"], r["w"] = dz.matmul(w), dz.t().matmul(x)
    if case["bias"]:
        r["bias"] = dz.sum(0)
    return r
