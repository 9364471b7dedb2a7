"""Linear attention with a decay for each head, and the norm of its queries and keys.

    o, ht = la_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=1.0)
    dq, dk, dv, dh0 = la_bwd(q, k, v, g, do, h0=None, dht=None, cu_seqlens=None, scale=1.0)
    o = la_step(q, k, v, g, state, slots=None, scale=1.0)
    yq, yk = qk_norm_fwd(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False)
    dq, dk, dwq, dwk = qk_norm_bwd(dyq, dyk, q, k, wq, wk, ...)
    cos, sin = rotation_table(positions, channels, base=10000.0, device="cuda")

Argument marshalling only, like the rest of the binding; ``include/gdr.h``
states the formulas, layouts and error codes.  q, k, v and the gradients of
outputs may be slices of wider tensors: the heads of a token must be contiguous
and tokens evenly spaced.  Parameters, states, tables and ``cu_seqlens`` must be
contiguous; outputs are.  Activations are bf16 or fp32.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .layer_ops import _addr, _call, _device, _dtype_code, _new, _param_code, _rows, _whole


class GdrLaDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("HV", ctypes.c_int64),
                ("K", ctypes.c_int64), ("V", ctypes.c_int64), ("N", ctypes.c_int64), ("ld_q", ctypes.c_int64),
                ("ld_k", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("ld_do", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class GdrQkNormDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("H", ctypes.c_int64), ("HK", ctypes.c_int64), ("D", ctypes.c_int64),
                ("P", ctypes.c_int64), ("R", ctypes.c_int64), ("ld_q", ctypes.c_int64), ("ld_k", ctypes.c_int64),
                ("ld_dyq", ctypes.c_int64), ("ld_dyk", ctypes.c_int64), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


def _bind():
    P = ctypes.c_void_p
    for name, desc, pointers in (("gdr_la_fwd", GdrLaDesc, 9), ("gdr_la_bwd", GdrLaDesc, 13),
                                 ("gdr_la_step", GdrLaDesc, 8), ("gdr_qk_norm_fwd", GdrQkNormDesc, 10),
                                 ("gdr_qk_norm_bwd", GdrQkNormDesc, 14)):
        getattr(_lib, name).argtypes = [ctypes.POINTER(desc)] + [P] * pointers


_bind()


def _like(t):
    """An output of t's shape and dtype, contiguous (of a slice in one call, which q, k and v mostly are)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# ------------------------------------------------------------------------------------ linear attention
def _la_desc(q, k, v, g, scale, dev, B, T, N, ld_do=None):
    lead = q.shape[:-2]
    H, K = q.shape[-2:]
    HV, V = v.shape[-2:]
    if v.dim() != q.dim() or v.shape[:-2] != lead:
        raise ValueError(f"v must be {tuple(lead)} + (HV, V), got {tuple(v.shape)}")
    _whole(g, "g", dev, torch.float32, (HV,))
    code, dtype = _dtype_code(q, "q"), q.dtype
    return GdrLaDesc(B, T, H, HV, K, V, N, _rows(q, "q", dev, None, None, 2), _rows(k, "k", dev, dtype, q.shape, 2),
                     _rows(v, "v", dev, dtype, None, 2), HV * V if ld_do is None else ld_do, scale, code, 0)


def _la_sequences(q, cu_seqlens):
    """(device, B, T, N) of a batch."""
    if q.dim() != 4:
        raise ValueError("q and k must be [B, T, H, K], v [B, T, HV, V]")
    dev = _device(q, "q")
    B, T = q.shape[:2]
    if cu_seqlens is None:
        return dev, B, T, B
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    _whole(cu_seqlens, "cu_seqlens", dev, torch.int64, cu_seqlens.shape)
    return dev, B, T, cu_seqlens.numel() - 1


def la_fwd(q, k, v, g, h0=None, cu_seqlens=None, scale=1.0, output_final_state=True, stream=None):
    """Linear attention with a decay for each head, per sequence and value head:

    ``S_t = exp(g) S_{t-1} + k_t v_t^T``, ``o_t = scale S_t^T q_t``.

    q, k [B, T, H, K]; v [B, T, HV, V], HV a multiple of H; g [HV] fp32; h0
    [N, HV, K, V] fp32.  Returns ``(o, ht)`` (ht None unless requested).

    Sums and states are fp32.  For bf16 heads of up to 128 channels (multiples of
    8, aligned rows) scores and the state that o reads are rounded to bf16 where
    they are multiplied: o is off by 2.3e-3, of which 1.7e-3 are its own rounding,
    and the fp32 ht by 2.5e-6.  Other heads: 6e-7 before the output's rounding.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return la_fwd(q, k, v, g, h0, cu_seqlens, scale, output_final_state)
    dev, B, T, N = _la_sequences(q, cu_seqlens)
    desc = _la_desc(q, k, v, g, scale, dev, B, T, N)
    shape = (N, desc.HV, desc.K, desc.V)
    _whole(h0, "h0", dev, torch.float32, shape)
    o = _like(v)
    ht = _new(g, shape) if output_final_state else None
    _call(_lib.gdr_la_fwd, dev, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(h0),
          _addr(cu_seqlens), o.data_ptr(), _addr(ht))
    return o, ht


def la_bwd(q, k, v, g, do, h0=None, dht=None, cu_seqlens=None, scale=1.0, stream=None):
    """Backward of ``la_fwd`` for L = sum(o * do) + sum(ht * dht).

    Returns ``(dq, dk, dv, dh0)``: dq, dk, dv in the inputs' dtype, dh0 fp32
    (the gradient of the initial state, zero or not).  g is a constant of the
    layer and has no gradient.  Roundings are those of ``la_fwd``: dq, dk and dv
    are as o there, dh0 as ht.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return la_bwd(q, k, v, g, do, h0, dht, cu_seqlens, scale)
    dev, B, T, N = _la_sequences(q, cu_seqlens)
    desc = _la_desc(q, k, v, g, scale, dev, B, T, N, _rows(do, "do", dev, q.dtype, v.shape, 2))
    shape = (N, desc.HV, desc.K, desc.V)
    _whole(h0, "h0", dev, torch.float32, shape)
    _whole(dht, "dht", dev, torch.float32, shape)
    dq, dk, dv, dh0 = _like(q), _like(k), _like(v), _new(g, shape)
    _call(_lib.gdr_la_bwd, dev, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(h0),
          _addr(cu_seqlens), do.data_ptr(), _addr(dht), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dh0.data_ptr())
    return dq, dk, dv, dh0


def la_step(q, k, v, g, state, slots=None, scale=1.0, stream=None):
    """One token per row: q, k [R, H, K]; v [R, HV, V]; state [P, HV, K, V] fp32, updated in place.

    Row r uses ``state[slots[r]]`` (slots int32; None: slot r).  A negative slot
    is a padding row with a zero output.  Slots of one call must differ.  All of it
    is fp32 but the rounding of o to its type.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return la_step(q, k, v, g, state, slots, scale)
    if q.dim() != 3 or state.dim() != 4:
        raise ValueError("q and k must be [R, H, K], v [R, HV, V], state [P, HV, K, V]")
    dev = _device(q, "q")
    R, P = q.shape[0], state.shape[0]
    _whole(slots, "slots", dev, torch.int32, (R,))
    if slots is None and P < R:
        raise ValueError(f"state has {P} slots for {R} rows")
    desc = _la_desc(q, k, v, g, scale, dev, R, 1, P)
    _whole(state, "state", dev, torch.float32, (P, desc.HV, desc.K, desc.V))
    o = _like(v)
    _call(_lib.gdr_la_step, dev, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(slots),
          state.data_ptr(), o.data_ptr())
    return o


# ------------------------------------------------------------------------- norm of queries and keys
def rotation_table(positions, channels, base=10000.0, device="cuda"):
    """(cos, sin) [positions, channels / 2] fp32 of the angles p base^(-2 i / channels), worked out in 64 bits."""
    if channels < 2 or channels % 2:
        raise ValueError(f"channels must be even and at least 2, got {channels}")
    freq = base ** (-torch.arange(0, channels, 2, dtype=torch.float64) / channels)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cos(angle).float().to(device), torch.sin(angle).float().to(device)


def _qk_desc(q, k, wq, wk, cos, sin, positions, eps, interleaved):
    if q.dim() < 2:
        raise ValueError("q must be [..., H, D]")
    dev = _device(q, "q")
    code, lead = _dtype_code(q, "q"), q.shape[:-2]
    H, D = q.shape[-2:]
    M = lead[0] if len(lead) == 1 else lead.numel()
    _whole(wq, "wq", dev, None, (D,))
    HK, ld_k = 0, 0
    if k is not None:
        if k.dim() != q.dim() or k.shape[:-2] != lead or k.shape[-1] != D:
            raise ValueError(f"k must be {tuple(lead)} + (HK, {D}), got {tuple(k.shape)}")
        _whole(wk, "wk", dev, wq.dtype, (D,))
        HK, ld_k = k.shape[-2], _rows(k, "k", dev, q.dtype, None, 2)
    P = R = 0
    if cos is None:
        if sin is not None or positions is not None:
            raise ValueError("a rotation needs cos, sin and positions")
    else:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [P, R]")
        _whole(cos, "cos", dev, torch.float32, cos.shape)
        _whole(sin, "sin", dev, torch.float32, cos.shape)
        _whole(positions, "positions", dev, torch.int64, lead)
        P, R = cos.shape
    return dev, GdrQkNormDesc(M, H, HK, D, P, R, _rows(q, "q", dev, None, None, 2), ld_k, H * D, HK * D, eps, code,
                              _param_code(wq, q, "wq"), int(bool(interleaved)), 0)


def qk_norm_fwd(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Root-mean-square norm of each head of q [..., H, D] and k [..., HK, D], and the rotation by position.

    ``n = x / sqrt(mean(x^2) + eps) * w`` over a head's channels; then the pairs
    of its first ``2 R`` channels, R the width of cos and sin [P, R] fp32, are
    turned by the angles of the token's position (positions [...], int64):
    channels i and i + R, or 2 i and 2 i + 1 with ``interleaved``.  No tables: no
    rotation.  A negative position is a padding token with zero outputs.  k (and
    wk) may be None.  Returns ``(yq, yk)``.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return qk_norm_fwd(q, k, wq, wk, cos, sin, positions, eps, interleaved)
    dev, desc = _qk_desc(q, k, wq, wk, cos, sin, positions, eps, interleaved)
    yq, yk = _like(q), None if k is None else _like(k)
    _call(_lib.gdr_qk_norm_fwd, dev, desc, q.data_ptr(), _addr(k), wq.data_ptr(), _addr(wk), _addr(cos), _addr(sin),
          _addr(positions), yq.data_ptr(), _addr(yk))
    return yq, yk


def qk_norm_bwd(dyq, dyk, q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Backward of ``qk_norm_fwd`` for L = sum(yq * dyq) + sum(yk * dyk).

    Returns ``(dq, dk, dwq, dwk)``: dq, dk in the inputs' dtype, dwq, dwk [D] fp32.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return qk_norm_bwd(dyq, dyk, q, k, wq, wk, cos, sin, positions, eps, interleaved)
    dev, desc = _qk_desc(q, k, wq, wk, cos, sin, positions, eps, interleaved)
    desc.ld_dyq = _rows(dyq, "dyq", dev, q.dtype, q.shape, 2)
    dk = dwk = None
    if k is not None:
        desc.ld_dyk = _rows(dyk, "dyk", dev, q.dtype, k.shape, 2)
        dk, dwk = _like(k), _new(q, desc.D, torch.float32)
    dq, dwq = _like(q), _new(q, desc.D, torch.float32)
    _call(_lib.gdr_qk_norm_bwd, dev, desc, dyq.data_ptr(), None if k is None else dyk.data_ptr(), q.data_ptr(),
          _addr(k), wq.data_ptr(), _addr(wk), _addr(cos), _addr(sin), _addr(positions), dq.data_ptr(), _addr(dk),
          dwq.data_ptr(), _addr(dwk))
    return dq, dk, dwq, dwk
