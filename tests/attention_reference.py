"""Plain 64-bit definitions of linear attention with a decay for each head and of
the heads' norm with rotation, in torch so that their gradients come from
automatic differentiation; and the tolerances of the tests.

Tolerances are relative 2-norms, counted in roundings of half a step.

fp32 (and the states, fp32 whatever the inputs): a product of the kernels is made
of parts of its factors, two of tf32 (2^-21 of the product is lost) or two of bf16
(2^-17, where the inputs are bf16).  An output is two products deep: a score and
a value, or a state's entry and a query; so is a gradient.  Decay factors and the
accumulation are fp32: eight roundings of 2^-24 a token, whose signs are independent,
so that n tokens add up like sqrt(n).  Sums with terms of both signs may be smaller
than their terms, for which a factor of four is left.

bf16 outputs take one rounding of 2^-8; before it, scores and states are rounded to
bf16 where they are multiplied: three of 2^-8 in all, the rest is far below.
"""
import math

import torch

from tests.layer_reference import HALF_STEP, rel, spans

F32, BF16 = torch.float32, torch.bfloat16


def tol(out_dtype, in_dtype, n):
    if out_dtype == BF16:
        return 3 * HALF_STEP[BF16]
    product = 2.0 ** -21 if in_dtype == F32 else 2.0 ** -17
    return 4 * (2 * product + 8 * math.sqrt(n) * 2.0 ** -24)


def close(got, want, in_dtype, n, what=""):
    err, bound = rel(got, want), tol(got.dtype, in_dtype, max(1, n))
    assert err <= bound, f"{what}: relative error {err:.3e} over {bound:.3e}"


def attention(q, k, v, g, h0, lens, scale):
    """q, k [M, H, K]; v [M, HV, V]; g [HV]; h0 [N, HV, K, V] -> o [M, HV, V], ht [N, HV, K, V]."""
    G = v.shape[1] // q.shape[1]
    f = torch.exp(g)[:, None, None]
    os, hts = [], []
    for n, i, j in spans(lens):
        s = h0[n]
        for t in range(i, j):
            s = f * s + k[t].repeat_interleave(G, 0)[:, :, None] * v[t][:, None]
            os.append((q[t].repeat_interleave(G, 0)[:, :, None] * s).sum(1) * scale)
        hts.append(s)
    return torch.stack(os) if os else v.new_zeros(v.shape), torch.stack(hts)


def attention_grads(q, k, v, g, h0, lens, scale, do, dht):
    """(dq, dk, dv, dh0) by automatic differentiation of the definition."""
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v, h0)]
    o, ht = attention(leaves[0], leaves[1], leaves[2], g, leaves[3], lens, scale)
    loss = (o * do).sum() + (ht * dht).sum()
    got = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(t) if d is None else d for t, d in zip(leaves, got)]


def heads(x, w, cos, sin, positions, interleaved, eps=1e-6):
    """x [M, heads, D], w [D], cos and sin [P, R] (None: no rotation); rows of negative positions are zero."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if cos is None:
        return n
    R, D = cos.shape[1], x.shape[-1]
    there = positions >= 0
    c, s = cos[positions.clamp(min=0)][:, None], sin[positions.clamp(min=0)][:, None]
    ia = torch.arange(R) * 2 if interleaved else torch.arange(R)
    ib = ia + (1 if interleaved else R)
    a, b = n[..., ia], n[..., ib]
    y = n.clone() if R < D // 2 or D % 2 else torch.empty_like(n)
    y = y.index_copy(-1, ia, a * c - b * s).index_copy(-1, ib, b * c + a * s)
    return torch.where(there[:, None, None], y, torch.zeros_like(y))


# -------------------------------------------------------------------------------------- inputs
def attention_inputs(lens, H, HV, K, V, dtype, seed=0, g=None):
    r = torch.Generator().manual_seed(seed)
    M, N = sum(lens), len(lens)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)  # noqa: E731
    if g is None:  # memories of a token and a half to two hundred
        g = -torch.exp2(-8.0 * torch.arange(1, HV + 1, dtype=torch.float64) / HV) * (0.5 + torch.rand(HV, generator=r))
    return dict(q=n(M, H, K).to(dtype), k=n(M, H, K).to(dtype), v=n(M, HV, V).to(dtype), g=g.float(),
                h0=n(N, HV, K, V).float(), do=n(M, HV, V).to(dtype), dht=n(N, HV, K, V).float())


def head_inputs(M, H, HK, D, R, dtype, seed=0, wdtype=None, table=64):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)  # noqa: E731
    wdtype = wdtype or dtype
    p = dict(q=n(M, H, D).to(dtype), k=n(M, HK, D).to(dtype) if HK else None, wq=(1 + 0.1 * n(D)).to(wdtype),
             wk=(1 + 0.1 * n(D)).to(wdtype) if HK else None, dyq=n(M, H, D).to(dtype),
             dyk=n(M, HK, D).to(dtype) if HK else None, cos=None, sin=None, positions=None)
    if R:
        angle = torch.arange(table, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(R) / R)
        p.update(cos=torch.cos(angle).float(), sin=torch.sin(angle).float(),
                 positions=torch.randint(0, table, (M,), generator=r))
    return p
