"""Cases that time the routing gate, its gradient and the per-request low-rank adapters.

Three operators of this package, each beside its plain form in elementary torch operations:

  gate           experts of every token from router logits: softmax or sigmoid scores, a balancing bias that
                 only the selection sees, groups of experts, top-k, renormalised and scaled weights
  gate_backward  the gradient of the gate's weights with respect to the logits
  lora           out[t] = base[t] + scale_a * (x[t] A_a^T) B_a^T with a = ids[t]: the adapters of many
                 requests added to the output of a projection that all of them share
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-20  # added to the sum of the selected sigmoid scores before it divides


def gate_case(name, op, T, E, k, score, dtype="f32", bias=False, groups=0, group_k=0, group_best=1, renorm=True,
              scale=1.0):
    return dict(name=name, op=op, T=T, E=E, k=k, score=score, dtype=dtype, bias=bias, groups=groups, group_k=group_k,
                group_best=group_best, renorm=renorm, scale=scale)


def lora_case(name, T, K, N, L, R, dtype, out, ids, ragged):
    return dict(name=name, op="lora", T=T, K=K, N=N, L=L, R=R, dtype=dtype, out=out, ids=ids, ragged=ragged)


def listed():
    return [
        # one new token of a 64-expert layer: only latency counts
        gate_case("gate_1x64", "gate", 1, 64, 4, "softmax"),
        # a decode batch over 256 experts, balanced by a bias, in 8 groups of which a token keeps 4
        gate_case("gate_64x256_groups", "gate", 64, 256, 8, "sigmoid", bias=True, groups=8, group_k=4, group_best=2,
                  scale=2.5),
        # a ragged prompt over 160 experts with bf16 logits (many ties), the best expert ranking each group
        gate_case("gate_1237x160_bf16", "gate", 1237, 160, 6, "softmax", dtype="bf16", groups=8, group_k=3,
                  renorm=False, scale=16.0),
        # a prefill of the 64-expert layer, balanced by a bias
        gate_case("gate_4096x64_bias", "gate", 4096, 64, 4, "sigmoid", bias=True),
        # a training step's tokens over 256 experts in groups
        gate_case("gate_65536x256_groups", "gate", 65536, 256, 8, "sigmoid", bias=True, groups=8, group_k=4,
                  group_best=2, scale=2.5),
        # router fine-tuning on a small batch of a 32-expert layer
        gate_case("grad_512x32", "gate_backward", 512, 32, 2, "softmax"),
        # weights that are probabilities over all experts: a dense gradient
        gate_case("grad_4096x64_dense", "gate_backward", 4096, 64, 4, "softmax", renorm=False),
        # a training step's tokens over 256 experts, sigmoid scores
        gate_case("grad_65536x256", "gate_backward", 65536, 256, 8, "sigmoid", scale=2.5),
        # one request's next token through its adapter
        lora_case("lora_1x4096", 1, 4096, 4096, 8, 16, "f16", "f16", "mixed", False),
        # a decode batch of 64 requests, 48 adapters of different ranks in use, some requests without one
        lora_case("lora_64x4096_mixed", 64, 4096, 4096, 48, 32, "bf16", "bf16", "mixed", True),
        # fine-tuned routers: the adapters act on the fp32 logits of the shared router, a ragged prompt batch
        lora_case("lora_777x64_logits", 777, 4096, 64, 12, 8, "bf16", "f32", "runs", False),
        # a prefill of a few requests, each a run of tokens
        lora_case("lora_4096x4096_runs", 4096, 4096, 4096, 6, 64, "bf16", "bf16", "runs", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gate", "gate", "gate_backward", "lora", "lora"))
    if op == "lora":
        R = rng.choice((8, 16, 24, 32, 64))
        out = rng.choice(("same", "same", "f32"))
        dtype = rng.choice(("f16", "bf16"))
        return lora_case_of(rng, R, dtype, dtype if out == "same" else "f32")
    gs = rng.randint(2, 32)  # experts per group
    G = rng.randint(2, max(2, min(16, 256 // gs)))
    E = min(256, gs * G) if rng.random() < 0.5 else rng.randint(4, 256)
    k = rng.randint(1, min(8, E))
    score = rng.choice(("softmax", "sigmoid"))
    T = _log_int(rng, 1, 65536)
    renorm = k > 1 and rng.random() < 0.6  # the weight of a single renormalised expert is constant
    c = gate_case(None, op, T, E, k, score, dtype=rng.choice(("f32", "f32", "f16", "bf16")), renorm=renorm,
                  scale=rng.choice((1.0, 2.5, 16.0)))
    del c["name"]
    if op == "gate":
        c["bias"] = rng.random() < 0.5
        if E == gs * G and rng.random() < 0.7:
            c["groups"], c["group_best"] = G, rng.randint(1, 2)
            c["group_k"] = rng.randint(-(-k // gs), G)  # enough groups for k experts
    return c


def lora_case_of(rng, R, dtype, out):
    T = _log_int(rng, 1, 4096)
    K = 8 * _log_int(rng, 8, 512)
    N = _log_int(rng, 16, 512) if out == "f32" else 8 * _log_int(rng, 8, 512)
    L = _log_int(rng, 1, max(1, min(64, 4096 * 384 // (T * R))))
    c = lora_case(None, T, K, N, L, R, dtype, out, rng.choice(("mixed", "runs")), rng.random() < 0.5)
    del c["name"]
    return c


def ranks_of(case):
    """The rank of every adapter: R, or by turns smaller ones where they are ragged."""
    R = case["R"]
    return [max(1, R - (i % 4) * (R // 4) - (i % 3)) if case["ragged"] else R for i in range(case["L"])]


def prepare(case, seed):
    """What a user's program holds before the call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "lora":
        T, K, N, L, R = (case[n] for n in ("T", "K", "N", "L", "R"))
        dt = DTYPES[case["dtype"]]
        ranks = torch.tensor(ranks_of(case), dtype=torch.int32, device="cuda")
        live = torch.arange(R, device="cuda")[None, :] < ranks[:, None]
        a = rand(L, R, K).mul_(1 / math.sqrt(K)).mul_(live[:, :, None]).to(dt)
        b = rand(L, N, R).mul_(0.5 / math.sqrt(R)).mul_(live[:, None, :]).to(dt)
        if case["ids"] == "mixed":
            ids = torch.randint(0, L, (T,), generator=g, device="cuda")
            none = torch.rand(T, generator=g, device="cuda") < 0.1
        else:  # runs of tokens: the requests' borders fall anywhere
            runs = max(1, min(T, 2 * L))
            border = torch.sort(torch.randint(0, T, (runs - 1,), generator=g, device="cuda")).values
            of = torch.searchsorted(border, torch.arange(T, device="cuda"), right=True)
            ids = torch.randint(0, L, (runs,), generator=g, device="cuda")[of]
            none = (torch.rand(runs, generator=g, device="cuda") < 0.1)[of]
        if T > 1:
            ids = torch.where(none, -1, ids)  # requests without an adapter
        return dict(case=case, x=rand(T, K).to(dt), base=rand(T, N).to(DTYPES[case["out"]]), ids=ids.to(torch.int32),
                    a=a, b=b, scale=0.5 + torch.rand(L, generator=g, device="cuda"), ranks=ranks)
    T, E = case["T"], case["E"]
    logits = (rand(T, E) * 1.5 + rand(E) * 0.5).to(DTYPES[case["dtype"]])
    s = dict(case=case, logits=logits, bias=rand(E) * 0.1 if case["bias"] else None)
    if case["op"] == "gate_backward":
        s["idx"] = _select(s)
        s["grad_w"] = rand(T, case["k"])
    return s


# ------------------------------------------------------------ plain forms


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softmax(v):
    e = torch.exp(v - v.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _first(keys, n):
    """The n largest of every row, equal ones by the lower index."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :n]


def _select(state):
    """Experts of every token.  Scores next to each other decide, so the keys are in 64 bits; without a bias the
    logits themselves give the order."""
    case, l, bias = state["case"], state["logits"], state["bias"]
    T, E, G = case["T"], case["E"], case["groups"]
    by_score = bias is not None or (G > 1 and case["group_best"] == 2)
    if by_score:
        score = _softmax(l.double()) if case["score"] == "softmax" else _sigmoid(l.double())
        keys = score if bias is None else score + bias.double()
    else:
        keys = l.float()
    if G > 1:
        best = torch.topk(keys.view(T, G, E // G), case["group_best"], dim=2).values.sum(2)
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        kept.scatter_(1, _first(best, case["group_k"]), True)
        keys = keys.masked_fill(~kept.repeat_interleave(E // G, dim=1), -math.inf)
    return _first(keys, case["k"]).to(torch.int32)


def _gate(state):
    case, l = state["case"], state["logits"].float()
    idx = _select(state)
    at = idx.long()
    if case["score"] == "softmax":
        w = _softmax(l.gather(1, at)) if case["renorm"] else _softmax(l).gather(1, at)
    else:
        w = _sigmoid(l.gather(1, at))
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + EPS)
    return dict(idx=idx, w=w * case["scale"])


def _gate_backward(state):
    case, l, at = state["case"], state["logits"].float(), state["idx"].long()
    dw = state["grad_w"] * case["scale"]
    grad = torch.zeros_like(l)
    sel = l.gather(1, at)
    if case["score"] == "sigmoid":
        s = _sigmoid(sel)
        if case["renorm"]:
            total = s.sum(1, keepdim=True) + EPS
            dw = (dw - (dw * s).sum(1, keepdim=True) / total) / total
        grad.scatter_(1, at, dw * s * _sigmoid(-sel))
    elif case["renorm"]:
        p = _softmax(sel)
        grad.scatter_(1, at, p * (dw - (dw * p).sum(1, keepdim=True)))
    else:
        p = _softmax(l)
        dot = (dw * p.gather(1, at)).sum(1, keepdim=True)
        grad.scatter_(1, at, dw)
        grad = p * (grad - dot)
    return grad.to(state["logits"].dtype)


def _lora(state):
    case, x, base = state["case"], state["x"].float(), state["base"]
    T, K, N, L, R = (case[n] for n in ("T", "K", "N", "L", "R"))
    u = (x @ state["a"].float().view(L * R, K).T).view(T, L, R)
    mine = torch.arange(L, device=x.device)[None, :] == state["ids"][:, None]
    live = torch.arange(R, device=x.device)[None, :] < state["ranks"][:, None]
    v = torch.where(mine[:, :, None] & live[None], u * state["scale"][None, :, None], 0.0)
    delta = v.view(T, L * R) @ state["b"].float().transpose(1, 2).reshape(L * R, N)
    return (base.float() + delta).to(base.dtype)


def run(state):
    case = state["case"]
    if own:
        import mixture_experts_router_amd as moe
        if case["op"] == "lora":
            return moe.lora_add(state["x"], state["base"], state["ids"], state["a"], state["b"], scale=state["scale"],
                                ranks=state["ranks"])
        if case["op"] == "gate_backward":
            return moe.gate_backward(state["logits"], state["idx"], state["grad_w"], score=case["score"],
                                     renorm=case["renorm"], scale=case["scale"])
        r = moe.gate_from_logits(state["logits"], case["k"], score=case["score"], bias=state["bias"],
                                 groups=case["groups"], group_k=case["group_k"], group_best=case["group_best"],
                                 renorm=case["renorm"], scale=case["scale"])
        return dict(idx=r["idx"], w=r["w"])
    if case["op"] == "lora":
        return _lora(state)
    return _gate_backward(state) if case["op"] == "gate_backward" else _gate(state)


def work(case):
    T = case["T"]
    if case["op"] == "lora":
        K, N, R = case["K"], case["N"], case["R"]
        ranks = ranks_of(case)
        used = min(case["L"], T)  # adapters in use, at most one a token
        rank = sum(ranks) / len(ranks)
        size, osize = BYTES[case["dtype"]], BYTES[case["out"]]
        return dict(bytes=T * K * size + 2 * T * N * osize + used * rank * (K + N) * size + 4 * T,
                    flops=2.0 * T * rank * (K + N))
    E, k, size = case["E"], case["k"], BYTES[case["dtype"]]
    if case["op"] == "gate":
        return dict(bytes=T * E * size + 8 * T * k + (4 * E if case["bias"] else 0), flops=4.0 * T * E)
    read = E if case["score"] == "softmax" and not case["renorm"] else k  # only a dense gradient needs every logit
    return dict(bytes=T * E * size + T * read * size + 8 * T * k, flops=4.0 * T * read)


# ---------------------------------------------------- definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    n = {key: v.double().cpu().numpy() for key, v in s.items() if torch.is_tensor(v)}
    if case["op"] == "lora":
        out, ids = n["base"].copy(), n["ids"].astype(np.int64)
        for a in range(case["L"]):
            rows, r = np.flatnonzero(ids == a), int(n["ranks"][a])
            if rows.size:
                out[rows] += n["scale"][a] * ((n["x"][rows] @ n["a"][a, :r].T) @ n["b"][a, :, :r].T)
        return out
    l, c = n["logits"], case["scale"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    rows = np.arange(T)[:, None]
    softmax = case["score"] == "softmax"
    lse = (l.max(1) + np.log(np.exp(l - l.max(1, keepdims=True)).sum(1)))[:, None]
    log_s = l - lse if softmax else -np.logaddexp(0.0, -l)  # logarithms of the scores
    if case["op"] == "gate":
        by_score = case["bias"] or (G > 1 and case["group_best"] == 2)
        keys = (np.exp(log_s) + n.get("bias", 0.0)) if by_score else l
        if G > 1:
            best = -np.sort(-keys.reshape(T, G, -1), axis=2)[:, :, :case["group_best"]].sum(2)
            out_of = np.argsort(-best, axis=1, kind="stable")[:, case["group_k"]:]
            keys = keys.reshape(T, G, -1).copy()
            keys[rows, out_of] = -np.inf
            keys = keys.reshape(T, E)
        idx = np.argsort(-keys, axis=1, kind="stable")[:, :k]
    else:
        idx = n["idx"].astype(np.int64)
    s = np.exp(log_s[rows, idx])
    total = s.sum(1, keepdims=True) + (0.0 if softmax else EPS)
    w = c * (s / total if case["renorm"] else s)
    if case["op"] == "gate":
        return dict(idx=torch.from_numpy(idx.astype(np.int32)), w=w)
    # d w_r / d s_j at the selected experts, then d s / d l
    dw = n["grad_w"]
    ds = c * dw / total - (dw * w).sum(1, keepdims=True) / total if case["renorm"] else c * dw
    grad = np.zeros((T, E))
    if softmax:
        grad[rows, idx] = ds
        p = np.exp(log_s)
        grad = p * (grad - (ds * s).sum(1, keepdims=True))
    else:
        grad[rows, idx] = ds * s * np.exp(-np.logaddexp(0.0, l[rows, idx]))
    return grad
