"""Plain 64-bit definitions of the operators around the recurrence (norm, short
convolution, selective scan), one token after the other, in torch so that their
gradients come from automatic differentiation; and the tolerances of the tests.

Tolerances are relative 2-norms, counted in roundings.  A value stored in fp32
is off by at most 2^-24 of itself, in bf16 by 2^-8.  An output takes one such
rounding.  Below it lie the fp32 roundings of the computation: an exponential is
off by up to 2^-22 (four of 2^-24) and each of a token's decay, product and sum
by 2^-24, seven in all, whose signs are independent, so that n tokens (or
summed rows) add up like sqrt(n); sums with terms of both signs may be smaller
than their terms, for which a factor of four is left.  32 more cover the
token's own operations (gate, softplus, filter, mean).
"""
import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def tol(dtype, n=1):
    return HALF_STEP[dtype] + (28 * math.sqrt(n) + 32) * 2.0 ** -24


def rel(got, want):
    assert tuple(got.shape) == tuple(want.shape), f"{tuple(got.shape)} != {tuple(want.shape)}"
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    if got.numel() == 0:
        return 0.0
    assert torch.isfinite(got).all(), "non-finite values in the output"
    den = float(want.norm())
    return float((got - want).norm()) / (den if den > 0 else 1.0)


def close(got, want, n=1, what=""):
    """got, in its own dtype, against the 64-bit value."""
    err, bound = rel(got, want), tol(got.dtype, n)
    assert err <= bound, f"{what}: relative error {err:.3e} over {bound:.3e}"


def spans(lens):
    at = 0
    for n, length in enumerate(lens):
        yield n, at, at + length
        at += length


def cu_of(lens, device="cpu"):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64, device=device)


def f64(t):
    return None if t is None else t.detach().double()


# --------------------------------------------------------------------------------------- norm
def norm(s, weight, eps):
    """y of rows s [M, E] (64-bit), with its gradient by automatic differentiation."""
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * weight


def stored_sum(x, residual):
    """x + residual as the residual stream holds it."""
    return (x.double() + residual.double()).to(residual.dtype)


# --------------------------------------------------------------------------------- convolution
def conv(x, weight, bias, s0, lens, silu=True):
    """x [M, E], s0 [N, W - 1, E] -> y [M, E], st [N, W - 1, E]."""
    W = weight.shape[1]
    ys, sts = [], []
    for n, i, j in spans(lens):
        full = torch.cat([s0[n], x[i:j]])
        pre = sum(full[k:k + j - i] * weight[:, k] for k in range(W))
        if bias is not None:
            pre = pre + bias
        ys.append(pre * torch.sigmoid(pre) if silu else pre)
        sts.append(full[full.shape[0] - (W - 1):])
    return torch.cat(ys), torch.stack(sts)


# ---------------------------------------------------------------------------------------- scan
def scan(x, dt, a, b, c, d, z, dt_bias, h0, lens, softplus=True):
    """x, dt, z [M, E]; b, c [M, G, S]; h0 [N, E, S] -> y [M, E], ht [N, E, S]."""
    E, G = x.shape[1], b.shape[1]
    raw = dt if dt_bias is None else dt + dt_bias
    delta = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    ys, hts = [], []
    for n, i, j in spans(lens):
        h = h0[n]
        for t in range(i, j):
            bt, ct = (v[t].repeat_interleave(E // G, 0) for v in (b, c))
            h = torch.exp(delta[t][:, None] * a) * h + (delta[t] * x[t])[:, None] * bt
            ys.append((h * ct).sum(1))
        hts.append(h)
    y = torch.stack(ys) if ys else x.new_zeros(x.shape)
    if d is not None:
        y = y + d * x
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    return y, torch.stack(hts)


def grads(fn, inputs, outputs_grads):
    """Gradients of sum(out * g) with respect to the inputs that are not None."""
    leaves = [None if t is None else t.detach().double().requires_grad_() for t in inputs]
    outs = fn(*leaves)
    loss = sum((o * g).sum() for o, g in zip(outs, outputs_grads) if g is not None)
    used = [t for t in leaves if t is not None]
    found = iter(torch.autograd.grad(loss, used, allow_unused=True))
    return [None if t is None else next(found) for t in leaves]


# -------------------------------------------------------------------------------------- inputs
def conv_inputs(lens, E, W, dtype, seed=0, bias=True, wdtype=None, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    M, N = sum(lens), len(lens)
    r = lambda *s, k=1.0: torch.randn(*s, generator=g, dtype=torch.float64) * k  # noqa: E731
    wdtype = wdtype or dtype
    p = dict(x=r(M, E).to(dtype), weight=r(E, W, k=W ** -0.5).to(wdtype), bias=r(E, k=0.1).to(wdtype) if bias else None,
             s0=r(N, W - 1, E).to(dtype), dy=r(M, E).to(dtype), dst=r(N, W - 1, E).to(dtype))
    return {k: None if v is None else v.to(device) for k, v in p.items()}


def scan_inputs(lens, E, S, G, dtype, seed=0, d=True, z=True, dt_bias=True, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    M, N = sum(lens), len(lens)
    r = lambda *s, k=1.0: torch.randn(*s, generator=g, dtype=torch.float64) * k  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, dtype=torch.float64)  # noqa: E731
    d0 = torch.exp(u(E) * math.log(100) + math.log(1e-3))  # delta at rest: log-uniform in [1e-3, 1e-1]
    p = dict(x=r(M, E).to(dtype), dt=r(M, E, k=0.5).to(dtype),
             a=(-torch.arange(1, S + 1, dtype=torch.float64) * (0.5 + u(E, S))).float(), b=r(M, G, S).to(dtype),
             c=r(M, G, S).to(dtype), d=r(E).float() if d else None, z=r(M, E).to(dtype) if z else None,
             dt_bias=(d0 + torch.log(-torch.expm1(-d0))).float() if dt_bias else None, h0=r(N, E, S, k=0.3).float(),
             dy=r(M, E).to(dtype), dht=r(N, E, S).float())
    return {k: None if v is None else v.to(device) for k, v in p.items()}
