"""What the layer operators refuse, checked on the host before anything is
launched: the C ABI's codes and the Python entry points' errors."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(16)  # never dereferenced: every call here is refused first


def norm_desc(m, **kw):
    return m.GdrNormDesc(**dict(dict(M=4, E=64, ld_x=64, ld_res=64, ld_ds=64, dtype=1, res_dtype=1, weight_dtype=1,
                                     quant=0, eps=1e-6, flags=0), **kw))


def conv_desc(m, **kw):
    return m.GdrConvDesc(**dict(dict(B=1, T=8, E=64, N=1, W=4, ld_x=64, ld_dy=64, dtype=1, weight_dtype=1,
                                     activation=1, flags=0), **kw))


def ssm_desc(m, **kw):
    return m.GdrSsmDesc(**dict(dict(B=1, T=8, E=64, S=16, G=1, N=1, ld_x=64, ld_dt=64, ld_z=64, ld_b=16, ld_c=16,
                                    ld_dy=64, dtype=1, flags=1), **kw))


def call(gdr, name, desc, pointers):
    return getattr(gdr.lib(), name)(ctypes.byref(desc), *pointers)


@pytest.fixture(scope="module")
def ops(gdr):
    from chunked_gated_delta_08_gb300 import layer_ops
    return layer_ops


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(dtype=0, res_dtype=1), -3), (dict(weight_dtype=3), -3), (dict(quant=3), -3),
    (dict(flags=1), -3), (dict(M=-1), -2), (dict(M=2 ** 31), -2), (dict(E=0), -2), (dict(E=2 ** 25, ld_x=2 ** 25), -2),
    (dict(ld_x=63), -2), (dict(ld_res=0), -2), (dict(ld_ds=1), -2), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2)])
def test_norm_descriptors(gdr, ops, kw, code):
    for name, n in (("gdr_norm_fwd", 7), ("gdr_norm_bwd", 8)):
        assert call(gdr, name, norm_desc(ops, **kw), [P] * (n - 1) + [None]) == code
        assert gdr.last_error()


def test_norm_pointers(gdr, ops):
    null = gdr.GDR_ERR_NULLPTR
    for missing in (0, 2, 3):  # x, weight, y
        args = [P, None, P, P, None, None, None]
        args[missing] = None
        assert call(gdr, "gdr_norm_fwd", norm_desc(ops), args) == null
    assert call(gdr, "gdr_norm_fwd", norm_desc(ops), [P, P, P, P, None, None, None]) == null  # residual without s
    assert call(gdr, "gdr_norm_fwd", norm_desc(ops, quant=1), [P, None, P, P, None, None, None]) == null  # no scale
    assert call(gdr, "gdr_norm_bwd", norm_desc(ops), [P, None, None, P, P, P, P, None]) == null  # no s
    assert call(gdr, "gdr_norm_bwd", norm_desc(ops, quant=2), [P] * 7 + [None]) == gdr.GDR_ERR_UNSUPPORTED
    assert call(gdr, "gdr_norm_fwd", norm_desc(ops, M=0), [None] * 7) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), -3), (dict(dtype=0, weight_dtype=1), -3), (dict(activation=2), -3), (dict(flags=4), -3),
    (dict(W=1), -2), (dict(W=5), -2), (dict(T=-1), -2), (dict(E=0), -2), (dict(N=2), -2), (dict(ld_x=10), -2),
    (dict(ld_dy=10), -2)])
def test_conv_descriptors(gdr, ops, kw, code):
    for name, n in (("gdr_conv_fwd", 8), ("gdr_conv_bwd", 12)):
        args = [P, P, P, P, None] + [P] * (n - 6) + [None]
        assert call(gdr, name, conv_desc(ops, **kw), args) == code
    if "N" not in kw:
        assert call(gdr, "gdr_conv_step", conv_desc(ops, **dict(dict(T=1), **kw)), [P] * 6 + [None]) == code


def test_conv_layouts_and_pointers(gdr, ops):
    assert call(gdr, "gdr_conv_fwd", conv_desc(ops, B=2, N=1), [P] * 7 + [None]) == gdr.GDR_ERR_SHAPE  # cu with B = 2
    assert call(gdr, "gdr_conv_step", conv_desc(ops, T=2), [P] * 6 + [None]) == gdr.GDR_ERR_SHAPE
    assert call(gdr, "gdr_conv_fwd", conv_desc(ops), [None, P, P, P, None, P, P, None]) == gdr.GDR_ERR_NULLPTR
    assert call(gdr, "gdr_conv_bwd", conv_desc(ops), [P, P, P, P, None, P, P, P, None, P, P, None]) == \
        gdr.GDR_ERR_NULLPTR  # no dweight
    assert call(gdr, "gdr_conv_step", conv_desc(ops, T=1), [P, P, P, P, None, P, None]) == gdr.GDR_ERR_NULLPTR


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), -3), (dict(flags=2), -3), (dict(S=0), -2), (dict(S=65, ld_b=65, ld_c=65), -2), (dict(G=0), -2),
    (dict(G=3, ld_b=48, ld_c=48), -2), (dict(E=0), -2), (dict(N=3), -2), (dict(T=-2), -2), (dict(ld_x=1), -2),
    (dict(ld_dt=1), -2), (dict(ld_z=1), -2), (dict(ld_b=15), -2), (dict(ld_c=15), -2), (dict(ld_dy=1), -2)])
def test_ssm_descriptors(gdr, ops, kw, code):
    for name, n, cu in (("gdr_ssm_fwd", 13, 9), ("gdr_ssm_bwd", 22, 9)):
        args = [P] * n
        args[cu] = None
        assert call(gdr, name, ssm_desc(ops, **kw), args) == code, name
    if "N" not in kw:
        assert call(gdr, "gdr_ssm_step", ssm_desc(ops, **dict(dict(T=1), **kw)), [P] * 12) == code


def test_ssm_layouts_and_pointers(gdr, ops):
    assert call(gdr, "gdr_ssm_fwd", ssm_desc(ops, B=2), [P] * 13) == gdr.GDR_ERR_SHAPE  # cu with B = 2
    args = [P] * 13
    args[9] = args[2] = None  # no a
    assert call(gdr, "gdr_ssm_fwd", ssm_desc(ops), args) == gdr.GDR_ERR_NULLPTR
    args = [P] * 22
    args[9] = args[6] = None  # dz without z
    assert call(gdr, "gdr_ssm_bwd", ssm_desc(ops), args) == gdr.GDR_ERR_NULLPTR
    args = [P] * 12
    args[9] = None  # no state
    assert call(gdr, "gdr_ssm_step", ssm_desc(ops, T=1), args) == gdr.GDR_ERR_NULLPTR
    assert call(gdr, "gdr_ssm_step", ssm_desc(ops, T=3), [P] * 12) == gdr.GDR_ERR_SHAPE


def test_null_descriptor(gdr):
    for name, n in (("gdr_norm_fwd", 7), ("gdr_conv_bwd", 12), ("gdr_ssm_bwd", 22), ("gdr_ssm_step", 12)):
        assert getattr(gdr.lib(), name)(None, *[P] * n) == gdr.GDR_ERR_NULLPTR


def test_cpu_tensors_are_refused(gdr):
    x, w = torch.zeros(2, 3, 8), torch.zeros(8)
    z = torch.zeros(2, 3, 1, 4)
    calls = [lambda: gdr.norm_fwd(x, w), lambda: gdr.norm_bwd(x, x, w), lambda: gdr.conv_fwd(x, torch.zeros(8, 4)),
             lambda: gdr.conv_bwd(x, torch.zeros(8, 4), x),
             lambda: gdr.conv_step(x[0], torch.zeros(3, 3, 8), torch.zeros(8, 4)),
             lambda: gdr.ssm_fwd(x, x, torch.zeros(8, 4), z, z), lambda: gdr.ssm_bwd(x, x, torch.zeros(8, 4), z, z, x),
             lambda: gdr.ssm_step(x[0], x[0], torch.zeros(8, 4), z[0], z[0], torch.zeros(3, 8, 4))]
    for f in calls:
        with pytest.raises(gdr.GdrError, match="CUDA tensor"):
            f()


def test_rank_is_checked_before_the_device(gdr):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match=r"\[B, T, E\]"):
        gdr.conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match=r"\[R, E\]"):
        gdr.conv_step(x[None], torch.zeros(3, 3, 8), torch.zeros(8, 4))
    with pytest.raises(gdr.GdrError, match="unsupported dtype"):
        gdr.norm_fwd(x.half(), torch.zeros(8))
