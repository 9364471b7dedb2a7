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

from . import GDR_BF16, GDR_ERR_DTYPE, GDR_ERR_NULLPTR, GDR_ERR_SHAPE, GDR_F32, GdrError, _check, _lib

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


# The smallest calls take less time on the GPU than here, so these checks read
# each attribute once and hand plain integers to ctypes.
def _addr(t):
    return None if t is None else t.data_ptr()


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


def _device(t, name):
    """The index of the current device, which must own the inputs."""
    dev = t.get_device()  # -1 on the CPU
    if dev < 0:
        raise GdrError(GDR_ERR_NULLPTR, f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise GdrError(GDR_ERR_NULLPTR, f"{name} is on {t.device}, but cuda:{torch.cuda.current_device()} is current")
    return dev


def _on(t, dev, name):
    """t is on the GPU that the call runs on."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise GdrError(GDR_ERR_NULLPTR, f"{name} must be a CUDA tensor")
        raise GdrError(GDR_ERR_NULLPTR, f"{name} is on {t.device}, expected cuda:{dev}")


def _whole(t, name, dev, dtype, shape):
    """Checks a contiguous tensor (None: nothing to check)."""
    if t is None:
        return
    _on(t, dev, name)
    if dtype is not None and t.dtype != dtype:
        raise GdrError(GDR_ERR_DTYPE, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise GdrError(GDR_ERR_SHAPE, f"{name} must be contiguous")


def _rows(t, name, dev, dtype=None, shape=None, row_dims=1):
    """Checks a token-major input; returns the distance between its rows in elements."""
    _on(t, dev, name)
    if dtype is not None and t.dtype != dtype:
        raise GdrError(GDR_ERR_DTYPE, f"{name} must be {dtype}, got {t.dtype}")
    size = t.shape
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(size)}")
    width = size[-1] if row_dims == 1 else size[-1] * size[-2]
    if t.is_contiguous():
        return width
    stride = t.stride()
    inner = 1
    for i in range(len(size) - 1, len(size) - 1 - row_dims, -1):
        if size[i] != 1 and stride[i] != inner:
            raise GdrError(GDR_ERR_SHAPE, f"{name}: the elements of a row must be contiguous")
        inner *= size[i]
    ld, step = None, 1
    for i in range(len(size) - 1 - row_dims, -1, -1):
        if size[i] != 1:
            if ld is None:
                ld = stride[i]
                if ld < width:
                    raise GdrError(GDR_ERR_SHAPE, f"{name}: rows overlap")
            elif stride[i] != ld * step:
                raise GdrError(GDR_ERR_SHAPE, f"{name}: rows must be evenly spaced; call contiguous()")
            step *= size[i]
    return width if ld is None else ld


def _like(t):
    """An output of t's shape and dtype, contiguous."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _new(t, shape, dtype=None):
    return torch.empty(shape, dtype=t.dtype if dtype is None else dtype, device=t.device)


def _call(fn, dev, desc, *args):
    rc = fn(desc, *args, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc)


# ------------------------------------------------------------------------------------------------ norm
def _norm_shape(x, weight, dev, name):
    if x.dim() < 1:
        raise ValueError(f"{name} must be [..., E]")
    E = x.shape[-1]
    _whole(weight, "weight", dev, None, (E,))
    return x.numel() // E if E else 0, E


def norm_fwd(x, weight, residual=None, eps=1e-6, quant=None, stream=None):
    """Root-mean-square norm over the last dimension, with the residual's addition.

    ``s = round(x + residual)`` in the residual's dtype (x's or fp32) and
    ``y = s / sqrt(mean(s^2) + eps) * weight``.  Returns ``(y, s)``, s None
    without a residual.  ``quant`` "row" or "group" (128 columns) returns
    ``(y8, scale, s)`` with y8 in float8_e4m3fn and ``y ~ y8 * scale``.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return norm_fwd(x, weight, residual, eps, quant)
    code = _dtype_code(x, "x")
    dev = _device(x, "x")
    M, E = _norm_shape(x, weight, dev, "x")
    if quant not in _QUANTS:
        raise ValueError(f"quant must be None, 'row' or 'group', got {quant!r}")
    ld_x, ld_r, rcode = _rows(x, "x", dev), E, code
    if residual is not None:
        rcode = _param_code(residual, x, "residual")
        ld_r = _rows(residual, "residual", dev, None, x.shape)
    desc = GdrNormDesc(M, E, ld_x, ld_r, E, code, rcode, _param_code(weight, x, "weight"), _QUANTS[quant], eps, 0)
    s = None if residual is None else _like(residual)
    scale = None
    if quant is None:
        y = _like(x)
    else:
        y = _new(x, x.shape, torch.float8_e4m3fn)
        lead = x.shape[:-1]
        scale = _new(x, lead if quant == "row" else (*lead, -(-E // GROUP_SIZE)), torch.float32)
    _call(_lib.gdr_norm_fwd, dev, desc, x.data_ptr(), _addr(residual), weight.data_ptr(), y.data_ptr(), _addr(scale),
          _addr(s))
    return (y, s) if quant is None else (y, scale, s)


def norm_bwd(dy, s, weight, ds=None, eps=1e-6, stream=None):
    """Backward of ``norm_fwd`` for L = sum(y * dy) + sum(s * ds); s is x where there was no residual.

    Returns ``(dx, dres, dweight)``: dx in dy's dtype, dres in s's (the same
    tensor where the two agree), dweight fp32.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return norm_bwd(dy, s, weight, ds, eps)
    code = _dtype_code(dy, "dy")
    dev = _device(dy, "dy")
    M, E = _norm_shape(dy, weight, dev, "dy")
    rcode = _param_code(s, dy, "s")
    ld_s, ld_ds = _rows(s, "s", dev, None, dy.shape), E
    if ds is not None:
        ld_ds = _rows(ds, "ds", dev, s.dtype, dy.shape)
    desc = GdrNormDesc(M, E, _rows(dy, "dy", dev), ld_s, ld_ds, code, rcode, _param_code(weight, dy, "weight"), 0, eps,
                       0)
    dx = _like(dy)
    dres = dx if s.dtype == dy.dtype else _new(s, dy.shape)
    dweight = _new(dy, E, torch.float32)
    _call(_lib.gdr_norm_bwd, dev, desc, dy.data_ptr(), s.data_ptr(), _addr(ds), weight.data_ptr(), dx.data_ptr(),
          None if dres is dx else dres.data_ptr(), dweight.data_ptr())
    return dx, dres, dweight


# ------------------------------------------------------------------------------------------ convolution
def _conv_desc(x, dev, weight, bias, activation, B, T, N, ld_dy):
    code = _dtype_code(x, "x")
    E = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != E:
        raise ValueError(f"weight must be [{E}, W], got {tuple(weight.shape)}")
    _whole(weight, "weight", dev, None, weight.shape)
    wcode = _param_code(weight, x, "weight")
    _whole(bias, "bias", dev, weight.dtype, (E,))
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise ValueError(f"weight must have 2 to 4 taps, got {W}")
    return GdrConvDesc(B, T, E, N, W, _rows(x, "x", dev), ld_dy, code, wcode, _ACTIVATIONS[activation], 0)


def _sequences(x, cu_seqlens):
    """(device, B, T, N) of a batch."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, E]")
    dev = _device(x, "x")
    B, T, _ = x.shape
    if cu_seqlens is None:
        return dev, B, T, B
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    _whole(cu_seqlens, "cu_seqlens", dev, torch.int64, cu_seqlens.shape)
    return dev, B, T, cu_seqlens.numel() - 1


def _step_rows(x, state, slots):
    """(device, rows, slots in the pool) of a single-token call."""
    if x.dim() != 2:
        raise ValueError("x must be [R, E]")
    dev = _device(x, "x")
    R, P = x.shape[0], state.shape[0]
    _whole(slots, "slots", dev, torch.int32, (R,))
    if slots is None and P < R:
        raise ValueError(f"state has {P} slots for {R} rows")
    return dev, R, P


def conv_fwd(x, weight, bias=None, s0=None, cu_seqlens=None, activation="silu", output_final_state=True,
             stream=None):
    """Causal convolution per channel, ``y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j})``.

    x [B, T, E]; weight [E, W], W in 2..4; s0 [N, W - 1, E] the inputs before
    each sequence (zero when None).  Returns ``(y, st)``, st the last W - 1
    inputs of each sequence (None unless requested).
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return conv_fwd(x, weight, bias, s0, cu_seqlens, activation, output_final_state)
    dev, B, T, N = _sequences(x, cu_seqlens)
    desc = _conv_desc(x, dev, weight, bias, activation, B, T, N, x.shape[-1])
    shape = (N, desc.W - 1, desc.E)
    _whole(s0, "s0", dev, x.dtype, shape)
    y = _like(x)
    st = _new(x, shape) if output_final_state else None
    _call(_lib.gdr_conv_fwd, dev, desc, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(s0), _addr(cu_seqlens),
          y.data_ptr(), _addr(st))
    return y, st


def conv_bwd(x, weight, dy, bias=None, s0=None, dst=None, cu_seqlens=None, activation="silu", stream=None):
    """Backward of ``conv_fwd`` for L = sum(y * dy) + sum(st * dst).

    Returns ``(dx, dweight, dbias, ds0)``: dx and ds0 in x's dtype, dweight and
    dbias fp32 (dbias None without a bias).
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return conv_bwd(x, weight, dy, bias, s0, dst, cu_seqlens, activation)
    dev, B, T, N = _sequences(x, cu_seqlens)
    desc = _conv_desc(x, dev, weight, bias, activation, B, T, N, _rows(dy, "dy", dev, x.dtype, x.shape))
    shape = (N, desc.W - 1, desc.E)
    _whole(s0, "s0", dev, x.dtype, shape)
    _whole(dst, "dst", dev, x.dtype, shape)
    dx, ds0 = _like(x), _new(x, shape)
    dweight = _new(x, weight.shape, torch.float32)
    dbias = None if bias is None else _new(x, desc.E, torch.float32)
    _call(_lib.gdr_conv_bwd, dev, desc, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(s0), _addr(cu_seqlens),
          dy.data_ptr(), _addr(dst), dx.data_ptr(), dweight.data_ptr(), _addr(dbias), ds0.data_ptr())
    return dx, dweight, dbias, ds0


def conv_step(x, state, weight, bias=None, activation="silu", slots=None, stream=None):
    """One token per row, x [R, E]; state [P, W - 1, E] is updated in place.

    Row r uses ``state[slots[r]]`` (slots int32; None: slot r).  A negative slot
    is a padding row with a zero output.  Slots of one call must differ.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return conv_step(x, state, weight, bias, activation, slots)
    dev, R, P = _step_rows(x, state, slots)
    desc = _conv_desc(x, dev, weight, bias, activation, R, 1, P, x.shape[1])
    _whole(state, "state", dev, x.dtype, (P, desc.W - 1, desc.E))
    y = _like(x)
    _call(_lib.gdr_conv_step, dev, desc, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(slots), state.data_ptr(),
          y.data_ptr())
    return y


# ------------------------------------------------------------------------------------------------ scan
def _ssm_desc(x, dev, dt, a, b, c, d, z, dt_bias, B, T, N, softplus, ld_dy):
    code = _dtype_code(x, "x")
    shape, dtype = x.shape, x.dtype
    E = shape[-1]
    if b.dim() != x.dim() + 1 or b.shape[:-2] != shape[:-1]:
        raise ValueError(f"b must be {tuple(shape[:-1])} + (G, S), got {tuple(b.shape)}")
    G, S = b.shape[-2:]
    _whole(a, "a", dev, torch.float32, (E, S))
    _whole(d, "d", dev, torch.float32, (E,))
    _whole(dt_bias, "dt_bias", dev, torch.float32, (E,))
    return GdrSsmDesc(B, T, E, S, G, N, _rows(x, "x", dev), _rows(dt, "dt", dev, dtype, shape),
                      E if z is None else _rows(z, "z", dev, dtype, shape), _rows(b, "b", dev, dtype, None, 2),
                      _rows(c, "c", dev, dtype, b.shape, 2), ld_dy, code, GDR_SSM_SOFTPLUS if softplus else 0)


def ssm_fwd(x, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, dt_softplus=True,
            output_final_state=True, stream=None):
    """Selective state space scan, per channel e of group g:

    ``h_t = exp(delta_t a[e]) h_{t-1} + delta_t x_t b_t[g]``,
    ``y_t = (c_t[g] . h_t + d[e] x_t) silu(z_t)``, ``delta = softplus(dt + dt_bias)``.

    x, dt, z [B, T, E]; a [E, S] fp32, S in 1..64; b, c [B, T, G, S]; h0
    [N, E, S] fp32.  Returns ``(y, ht)`` (ht None unless requested).
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return ssm_fwd(x, dt, a, b, c, d, z, dt_bias, h0, cu_seqlens, dt_softplus, output_final_state)
    dev, B, T, N = _sequences(x, cu_seqlens)
    desc = _ssm_desc(x, dev, dt, a, b, c, d, z, dt_bias, B, T, N, dt_softplus, x.shape[-1])
    shape = (N, desc.E, desc.S)
    _whole(h0, "h0", dev, torch.float32, shape)
    y = _like(x)
    ht = _new(a, shape) if output_final_state else None
    _call(_lib.gdr_ssm_fwd, dev, desc, x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _addr(d),
          _addr(z), _addr(dt_bias), _addr(h0), _addr(cu_seqlens), y.data_ptr(), _addr(ht))
    return y, ht


def ssm_bwd(x, dt, a, b, c, dy, d=None, z=None, dt_bias=None, h0=None, dht=None, cu_seqlens=None, dt_softplus=True,
            stream=None):
    """Backward of ``ssm_fwd`` for L = sum(y * dy) + sum(ht * dht).

    Returns ``(dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0)``: dx, ddt, db, dc,
    dz in x's dtype, the others fp32; dd, dz and ddt_bias are None where d, z
    and dt_bias are.  The forward is recomputed inside the call.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return ssm_bwd(x, dt, a, b, c, dy, d, z, dt_bias, h0, dht, cu_seqlens, dt_softplus)
    dev, B, T, N = _sequences(x, cu_seqlens)
    desc = _ssm_desc(x, dev, dt, a, b, c, d, z, dt_bias, B, T, N, dt_softplus, _rows(dy, "dy", dev, x.dtype, x.shape))
    shape = (N, desc.E, desc.S)
    _whole(h0, "h0", dev, torch.float32, shape)
    _whole(dht, "dht", dev, torch.float32, shape)
    dx, ddt = _like(x), _like(x)
    db, dc = _new(x, b.shape), _new(x, b.shape)
    dz = None if z is None else _like(x)
    da, dh0 = _like(a), _new(a, shape)
    dd = None if d is None else _new(a, desc.E)
    ddt_bias = None if dt_bias is None else _new(a, desc.E)
    _call(_lib.gdr_ssm_bwd, dev, desc, x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _addr(d),
          _addr(z), _addr(dt_bias), _addr(h0), _addr(cu_seqlens), dy.data_ptr(), _addr(dht), dx.data_ptr(),
          ddt.data_ptr(), da.data_ptr(), db.data_ptr(), dc.data_ptr(), _addr(dd), _addr(dz), _addr(ddt_bias),
          dh0.data_ptr())
    return dx, ddt, da, db, dc, dd, dz, ddt_bias, dh0


def ssm_step(x, dt, a, b, c, state, d=None, z=None, dt_bias=None, slots=None, dt_softplus=True, stream=None):
    """One token per row: x, dt, z [R, E]; b, c [R, G, S]; state [P, E, S] fp32, updated in place.

    ``slots`` as in ``conv_step``.
    """
    if stream is not None:  # outputs are taken while it is current, so that they belong to it
        with torch.cuda.stream(stream):
            return ssm_step(x, dt, a, b, c, state, d, z, dt_bias, slots, dt_softplus)
    dev, R, P = _step_rows(x, state, slots)
    desc = _ssm_desc(x, dev, dt, a, b, c, d, z, dt_bias, R, 1, P, dt_softplus, x.shape[1])
    _whole(state, "state", dev, torch.float32, (P, desc.E, desc.S))
    y = _like(x)
    _call(_lib.gdr_ssm_step, dev, desc, x.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _addr(d),
          _addr(z), _addr(dt_bias), _addr(slots), state.data_ptr(), y.data_ptr())
    return y
