"""Dense products with their epilogues and gradients in 64 bits, with bounds of the kernels' error.

U = 2^-24, h = half a step of the 16-bit type (bf16 2^-8, fp16 2^-11).  Products of two 16-bit floats are exact in
fp32.  A sum over K takes steps of 16 or 32 products in the matrix cores and joins at most 64 partial sums: every
addition is off by at most 2 U of the sum of the absolute products (the matrix cores need not round to nearest), at
most K / 16 + 96 of them on the way of one term.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def steps(K):
    return (K / 16 + 96) * 2 * U


def act(name, z):
    """(value, slope[, slope of the second half]) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    s = torch.sigmoid(z)
    if name == "sigmoid":
        return s, s * torch.sigmoid(-z)
    if name == "silu":
        return z * s, s * (1 + z * torch.sigmoid(-z))
    if name == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a, b = z.chunk(2, 1)
    s = torch.sigmoid(a)
    return a * s * b, s * (1 + a * torch.sigmoid(-a)) * b, a * s


def forward(x, w, bias=None, act_name="none", residual=None, row_scale=None, out_dtype=None):
    """(out, bound, z, bound of z) for tensors on the GPU."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    odt = x.dtype if out_dtype is None else out_dtype
    z = d(x) @ d(w).t()
    zb = steps(x.shape[1]) * (d(x).abs() @ d(w).abs().t())
    if bias is not None:
        z = z + d(bias)
        zb = zb + U * z.abs()
    a = act(act_name, z)
    if act_name == "swiglu":
        gate, up = z.chunk(2, 1)
        gb, ub = zb.chunk(2, 1)
        v, m = a[0], a[0].abs()
        # silu's slope is at most 1.1; gate and up errors, and eight roundings of the value
        b = 1.1 * gb * (up.abs() + ub) + a[2].abs() * ub + 8 * U * m
    else:
        v = a[0]
        b = 1.13 * zb + 8 * U * v.abs()  # no activation is steeper
    if act_name in ("silu", "gelu", "swiglu"):
        b = b + U  # the exponential's and erfc's own error where the value nearly vanishes
    if row_scale is not None:
        v = v * d(row_scale)[:, None]
        b = b * d(row_scale).abs()[:, None] + U * v.abs()
    if residual is not None:
        v = v + d(residual)
        b = b + U * v.abs()
    ob = b + HALF[odt] * (v.abs() + b) + TINY[odt]
    return v, ob, z, zb + HALF[x.dtype] * (z.abs() + zb) + TINY[x.dtype]


def backward(g, x, w, act_name="none", preact=None, row_scale=None):
    """dict of (gradient, bound) for x, w, bias and row_scale."""
    g, xd, wd = g.double(), x.double(), w.double()
    gr = g if row_scale is None else g * row_scale.double()[:, None]
    a = None
    dz, mag = gr, gr.abs()  # mag: what a slope's error of a few U multiplies
    if preact is not None:
        z = preact.double()
        a, *slopes = act(act_name, z)
        dz = torch.cat([gr * v for v in slopes], 1)
        if act_name == "swiglu":
            gate, up = z.chunk(2, 1)
            mag = torch.cat((mag * up.abs(), mag * gate.abs()), 1)
    # no activation's slope exceeds 1.2: its terms and roundings are off by at most 24 U
    fp32 = torch.zeros_like(dz) if preact is None and row_scale is None else 24 * U * (mag + dz.abs())
    rounded = fp32 + HALF[x.dtype] * (dz.abs() + fp32) + TINY[x.dtype]  # the operand of the products
    T, N = dz.shape

    def product(p, bound, q, n):
        v = p @ q
        b = bound @ q.abs()
        b = b + steps(n) * (p.abs() @ q.abs() + b)
        return v, b + HALF[x.dtype] * (v.abs() + b) + TINY[x.dtype]

    out = dict(x=product(dz, rounded, wd, N), w=product(dz.t(), rounded.t(), xd, T))
    # fp32 sums: T / 16 steps over blocks of rows, or the columns of a row, and at most 128 more
    out["bias"] = dz.sum(0), (fp32 + (T / 16 + 128) * U * (dz.abs() + fp32)).sum(0) + 2.0 ** -149
    if a is not None:
        out["row_scale"] = ((g * a).sum(1), (g.abs() * (24 * U * (a.abs() + 1) + (N / 16 + 128) * U * a.abs())).sum(1) +
                            2.0 ** -149)
    return out
