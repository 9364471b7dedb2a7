"""Operators around the recurrence: norm, short convolution, selective scan.

    y, s = norm_fwd(x, weight, residual=None, eps=1e-6)
    y8, scale, s = norm_fwd(x, weight, residual, quant="row" | "group")
    dx, dres, dweight = norm_bwd(dy, s, weight, ds=None, eps=1e-6)
    y, st = conv_fwd(x, weight, bias=None, s0=None, cu_seqlens=None, activation="silu")
    dx, dweight, dbias, ds0 = conv_bwd(x, weight, dy, bias=None, s0=None, dst=None, cu_seqlens=None)
    y = conv_step(x, state, weight, bias=None, slots=None)
    y, ht = ssm_fwd(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, cu_seqlens=None)
    dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0 = ssm_bwd(x, dt, a, b, c, dy, ...)
    y = ssm_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, slots=None)

Argument marshalling only, like the rest of the binding; ``include/gdr.h``
states the formulas, layouts and error codes.  Token-major inputs (x, dt, z, b,
c, dy, residual, s, ds) may be slices of wider tensors: their rows must be
contiguous and evenly spaced.  Parameters, states and ``cu_seqlens`` must be
contiguous; outputs are.  Activations are bf16 or fp32.
"""
from __future__ import annotations

import ctypes

import torch

from . import (GDR_BF16, GDR_ERR_DTYPE, GDR_ERR_NULLPTR, GDR_ERR_SHAPE, GDR_F32, GdrError, _check, _lib, _ptr,
               _require, _stream_ptr)

_QUANTS = {None: 0, "row": 1, "group": 2}
_ACTIVATIONS = {None: 0, "silu": 1}
_DTYPES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}
GROUP_SIZE = 128
GDR_SSM_SOFTPLUS = 1


class GdrNormDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("E", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_res", ctypes.c_int64),
                ("ld_ds", ctypes.c_int64), ("dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("quant", ctypes.c_int32), ("eps", ctypes.c_float),
                ("flags", ctypes.c_int32)]


class GdrConvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("E", ctypes.c_int64), ("N", ctypes.c_int64),
                ("W", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_dy", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class GdrSsmDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("E", ctypes.c_int64), ("S", ctypes.c_int64),
                ("G", ctypes.c_int64), ("N", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_dt", ctypes.c_int64),
                ("ld_z", ctypes.c_int64), ("ld_b", ctypes.c_int64), ("ld_c", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


def _bind():
    P = ctypes.c_void_p
    for name, desc, pointers in (("gdr_norm_fwd", GdrNormDesc, 7), ("gdr_norm_bwd", GdrNormDesc, 8),
                                 ("gdr_conv_fwd", GdrConvDesc, 8), ("gdr_conv_bwd", GdrConvDesc, 12),
                                 ("gdr_conv_step", GdrConvDesc, 7), ("gdr_ssm_fwd", GdrSsmDesc, 13),
                                 ("gdr_ssm_bwd", GdrSsmDesc, 22), ("gdr_ssm_step", GdrSsmDesc, 12)):
        getattr(_lib, name).argtypes = [ctypes.POINTER(desc)] + [P] * pointers


_bind()


def _dtype_code(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise GdrError(GDR_ERR_DTYPE, f"{name}: unsupported dtype {t.dtype}")
    return code


def _param_code(t, x, name):
    """The dtype code of a parameter, which is fp32 or of x's dtype."""
    if t.dtype != x.dtype and t.dtype != torch.float32:
        raise GdrError(GDR_ERR_DTYPE, f"{name} must be {x.dtype} or torch.float32, got {t.dtype}")
    return _DTYPES[t.dtype]


def _on(t, ref, name):
    """t is on the GPU that ref is on."""
    if not t.is_cuda:
        raise GdrError(GDR_ERR_NULLPTR, f"{name} must be a CUDA tensor")
    if ref is not None and t.device != ref.device:
        raise GdrError(GDR_ERR_NULLPTR, f"{name} is on {t.device}, expected {ref.device}")


def _rows(t, name, ref=None, dtype=None, shape=None, row_dims=1):
    """Checks a token-major input; returns the distance between its rows in elements."""
    _on(t, ref, name)
    if dtype is not None and t.dtype != dtype:
        raise GdrError(GDR_ERR_DTYPE, f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    size, stride = t.shape, t.stride()
    width = 1
    for i in range(t.dim() - 1, t.dim() - 1 - row_dims, -1):
        if size[i] != 1 and stride[i] != width:
            raise GdrError(GDR_ERR_SHAPE, f"{name}: the elements of a row must be contiguous")
        width *= size[i]
    ld = None
    step = 1
    for i in range(t.dim() - 1 - row_dims, -1, -1):
        if size[i] != 1:
            if ld is None:
                if stride[i] < width:
                    raise GdrError(GDR_ERR_SHAPE, f"{name}: rows overlap")
                ld = stride[i]
            elif stride[i] != ld * step:
                if t.numel():
                    raise GdrError(GDR_ERR_SHAPE, f"{name}: rows must be evenly spaced; call contiguous()")
            step *= size[i]
    return width if ld is None else max(ld, width)


def _device_of(t, name):
    """The call runs on the current device, which must own the inputs."""
    _on(t, None, name)
    if t.device.index != torch.cuda.current_device():
        raise GdrError(GDR_ERR_NULLPTR, f"{name} is on {t.device}, but cuda:{torch.cuda.current_device()} is current")


class _outputs_on:
    """Outputs belong to the launching stream: memory is taken while it is current."""

    def __init__(self, stream):
        self.ctx = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


# ------------------------------------------------------------------------------------------------ norm
def _norm_shape(x, weight, name):
    if x.dim() < 1:
        raise ValueError(f"{name} must be [..., E]")
    E = x.shape[-1]
    _on(weight, x, "weight")
    _require(weight, "weight", None, (E,))
    return x.numel() // E if E else 0, E


def norm_fwd(x, weight, residual=None, eps=1e-6, quant=None, stream=None):
    """Root-mean-square norm over the last dimension, with the residual's addition.

    ``s = round(x + residual)`` in the residual's dtype (x's or fp32) and
    ``y = s / sqrt(mean(s^2) + eps) * weight``.  Returns ``(y, s)``, s None
    without a residual.  ``quant`` "row" or "group" (128 columns) returns
    ``(y8, scale, s)`` with y8 in float8_e4m3fn and ``y ~ y8 * scale``.
    """
    code = _dtype_code(x, "x")
    _device_of(x, "x")
    M, E = _norm_shape(x, weight, "x")
    if quant not in _QUANTS:
        raise ValueError(f"quant must be None, 'row' or 'group', got {quant!r}")
    ld_x, ld_r, rcode = _rows(x, "x"), E, code
    if residual is not None:
        rcode = _param_code(residual, x, "residual")
        ld_r = _rows(residual, "residual", x, None, x.shape)
    desc = GdrNormDesc(M, E, ld_x, ld_r, E, code, rcode, _param_code(weight, x, "weight"), _QUANTS[quant], eps, 0)
    with _outputs_on(stream):
        s = None if residual is None else torch.empty(x.shape, dtype=residual.dtype, device=x.device)
        scale = None
        if quant is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
            lead = x.shape[:-1]
            scale = torch.empty(lead if quant == "row" else (*lead, -(-E // GROUP_SIZE)), dtype=torch.float32,
                                device=x.device)
    _check(_lib.gdr_norm_fwd(ctypes.byref(desc), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y), _ptr(scale),
                             _ptr(s), _stream_ptr(stream)))
    return (y, s) if quant is None else (y, scale, s)


def norm_bwd(dy, s, weight, ds=None, eps=1e-6, stream=None):
    """Backward of ``norm_fwd`` for L = sum(y * dy) + sum(s * ds); s is x where there was no residual.

    Returns ``(dx, dres, dweight)``: dx in dy's dtype, dres in s's (the same
    tensor where the two agree), dweight fp32.
    """
    code = _dtype_code(dy, "dy")
    _device_of(dy, "dy")
    M, E = _norm_shape(dy, weight, "dy")
    rcode = _param_code(s, dy, "s")
    ld_s, ld_ds = _rows(s, "s", dy, None, dy.shape), E
    if ds is not None:
        ld_ds = _rows(ds, "ds", dy, s.dtype, dy.shape)
    desc = GdrNormDesc(M, E, _rows(dy, "dy"), ld_s, ld_ds, code, rcode, _param_code(weight, dy, "weight"), 0, eps, 0)
    with _outputs_on(stream):
        dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
        dres = dx if s.dtype == dy.dtype else torch.empty(dy.shape, dtype=s.dtype, device=dy.device)
        dweight = torch.empty(E, dtype=torch.float32, device=dy.device)
    _check(_lib.gdr_norm_bwd(ctypes.byref(desc), _ptr(dy), _ptr(s), _ptr(ds), _ptr(weight), _ptr(dx),
                             None if dres is dx else _ptr(dres), _ptr(dweight), _stream_ptr(stream)))
    return dx, dres, dweight


# ------------------------------------------------------------------------------------------ convolution
def _conv_desc(x, weight, bias, activation, B, T, N, ld_dy):
    code = _dtype_code(x, "x")
    E = x.shape[-1]
    _on(weight, x, "weight")
    if weight.dim() != 2 or weight.shape[0] != E:
        raise ValueError(f"weight must be [{E}, W], got {tuple(weight.shape)}")
    _require(weight, "weight")
    wcode = _param_code(weight, x, "weight")
    if bias is not None:
        _on(bias, x, "bias")
        _require(bias, "bias", weight.dtype, (E,))
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    return GdrConvDesc(B, T, E, N, weight.shape[1], _rows(x, "x"), ld_dy, code, wcode, _ACTIVATIONS[activation], 0)


def _sequences(x, cu_seqlens):
    if x.dim() != 3:
        raise ValueError("x must be [B, T, E]")
    B, T = x.shape[:2]
    if cu_seqlens is None:
        return B, T, B
    _on(cu_seqlens, x, "cu_seqlens")
    _require(cu_seqlens, "cu_seqlens", torch.int64)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    return B, T, cu_seqlens.numel() - 1


def _state(t, name, ref, dtype, shape):
    if t is not None:
        _on(t, ref, name)
        _require(t, name, dtype, shape)


def _slots(slots, x, R):
    if slots is not None:
        _on(slots, x, "slots")
        _require(slots, "slots", torch.int32, (R,))


def conv_fwd(x, weight, bias=None, s0=None, cu_seqlens=None, activation="silu", output_final_state=True,
             stream=None):
    """Causal convolution per channel, ``y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j})``.

    x [B, T, E]; weight [E, W], W in 2..4; s0 [N, W - 1, E] the inputs before
    each sequence (zero when None).  Returns ``(y, st)``, st the last W - 1
    inputs of each sequence (None unless requested).
    """
    B, T, N = _sequences(x, cu_seqlens)
    _device_of(x, "x")
    desc = _conv_desc(x, weight, bias, activation, B, T, N, x.shape[-1])
    shape = (N, desc.W - 1, desc.E)
    _state(s0, "s0", x, x.dtype, shape)
    with _outputs_on(stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        st = torch.empty(shape, dtype=x.dtype, device=x.device) if output_final_state and desc.W > 1 else None
    _check(_lib.gdr_conv_fwd(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(s0), _ptr(cu_seqlens),
                             _ptr(y), _ptr(st), _stream_ptr(stream)))
    return y, st


def conv_bwd(x, weight, dy, bias=None, s0=None, dst=None, cu_seqlens=None, activation="silu", stream=None):
    """Backward of ``conv_fwd`` for L = sum(y * dy) + sum(st * dst).

    Returns ``(dx, dweight, dbias, ds0)``: dx and ds0 in x's dtype, dweight and
    dbias fp32 (dbias None without a bias).
    """
    B, T, N = _sequences(x, cu_seqlens)
    _device_of(x, "x")
    desc = _conv_desc(x, weight, bias, activation, B, T, N, _rows(dy, "dy", x, x.dtype, x.shape))
    shape = (N, desc.W - 1, desc.E)
    _state(s0, "s0", x, x.dtype, shape)
    _state(dst, "dst", x, x.dtype, shape)
    with _outputs_on(stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dweight = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
        dbias = None if bias is None else torch.empty(desc.E, dtype=torch.float32, device=x.device)
        ds0 = torch.empty((N, max(0, desc.W - 1), desc.E), dtype=x.dtype, device=x.device)
    _check(_lib.gdr_conv_bwd(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(s0), _ptr(cu_seqlens),
                             _ptr(dy), _ptr(dst), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(ds0),
                             _stream_ptr(stream)))
    return dx, dweight, dbias, ds0


def conv_step(x, state, weight, bias=None, activation="silu", slots=None, stream=None):
    """One token per row, x [R, E]; state [P, W - 1, E] is updated in place.

    Row r uses ``state[slots[r]]`` (slots int32; None: slot r).  A negative slot
    is a padding row with a zero output.  Slots of one call must differ.
    """
    if x.dim() != 2:
        raise ValueError("x must be [R, E]")
    _device_of(x, "x")
    R = x.shape[0]
    desc = _conv_desc(x, weight, bias, activation, R, 1, state.shape[0], x.shape[1])
    _state(state, "state", x, x.dtype, (state.shape[0], desc.W - 1, desc.E))
    _slots(slots, x, R)
    if slots is None and state.shape[0] < R:
        raise ValueError(f"state has {state.shape[0]} slots for {R} rows")
    with _outputs_on(stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _check(_lib.gdr_conv_step(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(slots), _ptr(state),
                              _ptr(y), _stream_ptr(stream)))
    return y


# ------------------------------------------------------------------------------------------------ scan
def _ssm_desc(x, dt, a, b, c, d, z, dt_bias, B, T, N, softplus, ld_dy):
    code = _dtype_code(x, "x")
    lead, E = x.shape[:-1], x.shape[-1]
    if b.dim() != x.dim() + 1 or tuple(b.shape[:-2]) != tuple(lead):
        raise ValueError(f"b must be {tuple(lead)} + (G, S), got {tuple(b.shape)}")
    G, S = b.shape[-2:]
    _on(a, x, "a")
    _require(a, "a", torch.float32, (E, S))
    for t, name in ((d, "d"), (dt_bias, "dt_bias")):
        if t is not None:
            _on(t, x, name)
            _require(t, name, torch.float32, (E,))
    return GdrSsmDesc(B, T, E, S, G, N, _rows(x, "x"), _rows(dt, "dt", x, x.dtype, x.shape),
                      E if z is None else _rows(z, "z", x, x.dtype, x.shape),
                      _rows(b, "b", x, x.dtype, None, 2), _rows(c, "c", x, x.dtype, b.shape, 2), ld_dy, code,
                      GDR_SSM_SOFTPLUS if softplus else 0)


def ssm_fwd(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, dt_softplus=True,
            output_final_state=True, stream=None):
    """Selective state space scan, per channel e of group g:

    ``h_t = exp(delta_t a[e]) h_{t-1} + delta_t x_t b_t[g]``,
    ``y_t = (c_t[g] . h_t + d[e] x_t) silu(z_t)``, ``delta = softplus(dt + dt_bias)``.

    x, dt, z [B, T, E]; a [E, S] fp32; b, c [B, T, G, S]; h0 [N, E, S] fp32.
    Returns ``(y, ht)`` (ht None unless requested).
    """
    B, T, N = _sequences(x, cu_seqlens)
    _device_of(x, "x")
    desc = _ssm_desc(x, dt, a, b, c, d, z, dt_bias, B, T, N, dt_softplus, x.shape[-1])
    shape = (N, desc.E, desc.S)
    _state(h0, "h0", x, torch.float32, shape)
    with _outputs_on(stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ht = torch.empty(shape, dtype=torch.float32, device=x.device) if output_final_state else None
    _check(_lib.gdr_ssm_fwd(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(z),
                            _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), _ptr(y), _ptr(ht), _stream_ptr(stream)))
    return y, ht


def ssm_bwd(x, dt, a, b, c, dy, d=None, z=None, dt_bias=None, h0=None, dht=None, cu_seqlens=None, dt_softplus=True,
            stream=None):
    """Backward of ``ssm_fwd`` for L = sum(y * dy) + sum(ht * dht).

    Returns ``(dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0)``: dx, ddt, db, dc,
    dz in x's dtype, the others fp32; dd, dz and ddt_bias are None where d, z
    and dt_bias are.  The forward is recomputed inside the call.
    """
    B, T, N = _sequences(x, cu_seqlens)
    _device_of(x, "x")
    desc = _ssm_desc(x, dt, a, b, c, d, z, dt_bias, B, T, N, dt_softplus, _rows(dy, "dy", x, x.dtype, x.shape))
    shape = (N, desc.E, desc.S)
    _state(h0, "h0", x, torch.float32, shape)
    _state(dht, "dht", x, torch.float32, shape)
    like = dict(dtype=x.dtype, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    with _outputs_on(stream):
        dx, ddt = torch.empty(x.shape, **like), torch.empty(x.shape, **like)
        db, dc = torch.empty(b.shape, **like), torch.empty(b.shape, **like)
        dz = None if z is None else torch.empty(x.shape, **like)
        da = torch.empty(a.shape, **f32)
        dd = None if d is None else torch.empty(desc.E, **f32)
        ddt_bias = None if dt_bias is None else torch.empty(desc.E, **f32)
        dh0 = torch.empty(shape, **f32)
    _check(_lib.gdr_ssm_bwd(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(z),
                            _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), _ptr(dy), _ptr(dht), _ptr(dx), _ptr(ddt),
                            _ptr(da), _ptr(db), _ptr(dc), _ptr(dd), _ptr(dz), _ptr(ddt_bias), _ptr(dh0),
                            _stream_ptr(stream)))
    return dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0


def ssm_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, slots=None, dt_softplus=True, stream=None):
    """One token per row: x, dt, z [R, E]; b, c [R, G, S]; state [P, E, S] fp32, updated in place.

    ``slots`` as in ``conv_step``.
    """
    if x.dim() != 2:
        raise ValueError("x must be [R, E]")
    _device_of(x, "x")
    R = x.shape[0]
    desc = _ssm_desc(x, dt, a, b, c, d, z, dt_bias, R, 1, state.shape[0], dt_softplus, x.shape[1])
    _state(state, "state", x, torch.float32, (state.shape[0], desc.E, desc.S))
    _slots(slots, x, R)
    if slots is None and state.shape[0] < R:
        raise ValueError(f"state has {state.shape[0]} slots for {R} rows")
    with _outputs_on(stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _check(_lib.gdr_ssm_step(ctypes.byref(desc), _ptr(x), _ptr(dt), _ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(z),
                             _ptr(dt_bias), _ptr(slots), _ptr(state), _ptr(y), _stream_ptr(stream)))
    return y
