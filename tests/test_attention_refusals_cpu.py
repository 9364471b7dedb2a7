"""What linear attention and the heads' norm refuse, checked on the host before
anything is launched: the C ABI's codes and the Python entry points' errors."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(16)  # never dereferenced: every call here is refused first
FORMS = (("gdr_la_fwd", 9, 5), ("gdr_la_bwd", 13, 5))  # name, pointers, which is cu_seqlens


@pytest.fixture(scope="module")
def ops(gdr):
    from chunked_gated_delta_08_gb300 import attention_ops
    return attention_ops


def la_desc(m, **kw):
    return m.GdrLaDesc(**dict(dict(B=1, T=8, H=2, HV=4, K=64, V=32, N=1, ld_q=128, ld_k=128, ld_v=128, ld_do=128,
                                   scale=1.0, dtype=1, flags=0), **kw))


def qk_desc(m, **kw):
    return m.GdrQkNormDesc(**dict(dict(M=4, H=2, HK=1, D=64, P=16, R=32, ld_q=128, ld_k=64, ld_dyq=128, ld_dyk=64,
                                       eps=1e-6, dtype=1, weight_dtype=1, interleaved=0, flags=0), **kw))


def call(gdr, name, desc, pointers):
    return getattr(gdr.lib(), name)(ctypes.byref(desc), *pointers)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(flags=1), -3), (dict(B=-1), -2), (dict(T=-1), -2), (dict(N=2), -2), (dict(H=0), -2),
    (dict(HV=5), -2), (dict(HV=0), -2), (dict(H=65536, HV=65536), -2), (dict(K=0), -2), (dict(K=257), -2),
    (dict(V=0), -2), (dict(V=257), -2), (dict(ld_q=127), -2), (dict(ld_k=0), -2), (dict(ld_v=127), -2),
    (dict(ld_do=1), -2), (dict(ld_q=2 ** 31), -2), (dict(scale=float("inf")), -2), (dict(scale=float("nan")), -2),
    (dict(B=2 ** 16, N=2 ** 16, T=2 ** 15), -2), (dict(T=2 ** 31), -2)], ids=str)
def test_attention_descriptors(gdr, ops, kw, code):
    for name, n, cu in FORMS:
        args = [P] * n
        args[cu] = None
        assert call(gdr, name, la_desc(ops, **kw), args) == code, name
        assert gdr.last_error()
    if not {"N", "T", "B"} & set(kw):
        assert call(gdr, "gdr_la_step", la_desc(ops, **dict(dict(T=1), **kw)), [P] * 8) == code


def test_attention_layouts_and_pointers(gdr, ops):
    null, shape = gdr.GDR_ERR_NULLPTR, gdr.GDR_ERR_SHAPE
    for name, n, cu in FORMS:
        assert call(gdr, name, la_desc(ops, B=2, N=1), [P] * n) == shape  # cu_seqlens with B = 2
    for name, n, needed in (("gdr_la_fwd", 9, (0, 1, 2, 3, 6)), ("gdr_la_bwd", 13, (0, 1, 2, 3, 6, 8, 9, 10)),
                            ("gdr_la_step", 8, (0, 1, 2, 3, 5, 6))):
        for missing in needed:
            args = [P] * n
            if name != "gdr_la_step":
                args[5] = None
            args[missing] = None
            assert call(gdr, name, la_desc(ops, T=1), args) == null, (name, missing)
        assert getattr(gdr.lib(), name)(None, *[P] * n) == null
    assert call(gdr, "gdr_la_step", la_desc(ops, T=2), [P] * 8) == shape
    assert call(gdr, "gdr_la_step", la_desc(ops, T=1, B=0), [None] * 8) == 0
    assert call(gdr, "gdr_la_fwd", la_desc(ops, B=0, N=0), [None] * 9) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -3), (dict(dtype=0, weight_dtype=1), -3), (dict(flags=1), -3), (dict(interleaved=2), -3),
    (dict(M=-1), -2), (dict(M=2 ** 31), -2), (dict(H=0), -2), (dict(HK=-1), -2), (dict(H=65536, ld_q=2 ** 30), -2),
    (dict(D=0), -2), (dict(D=257, ld_q=1000, ld_k=1000, ld_dyq=1000, ld_dyk=1000), -2), (dict(R=33), -2),
    (dict(R=-1), -2), (dict(P=-1), -2), (dict(ld_q=127), -2), (dict(ld_k=63), -2), (dict(ld_dyq=1), -2),
    (dict(ld_dyk=1), -2), (dict(ld_q=2 ** 31), -2), (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2)], ids=str)
def test_head_norm_descriptors(gdr, ops, kw, code):
    for name, n in (("gdr_qk_norm_fwd", 10), ("gdr_qk_norm_bwd", 14)):
        assert call(gdr, name, qk_desc(ops, **kw), [P] * n) == code, name
        assert gdr.last_error()


def test_head_norm_pointers(gdr, ops):
    null = gdr.GDR_ERR_NULLPTR
    for name, n in (("gdr_qk_norm_fwd", 10), ("gdr_qk_norm_bwd", 14)):
        for missing in range(n - 1):
            args = [P] * n
            args[missing] = None
            assert call(gdr, name, qk_desc(ops), args) == null, (name, missing)
        assert getattr(gdr.lib(), name)(None, *[P] * n) == null
    assert call(gdr, "gdr_qk_norm_fwd", qk_desc(ops, M=0), [None] * 10) == 0


def test_tensors_that_are_refused(gdr):
    q, v, g = torch.zeros(1, 3, 2, 8), torch.zeros(1, 3, 4, 6), torch.zeros(4)
    w, state = torch.zeros(8), torch.zeros(3, 4, 8, 6)
    calls = [lambda: gdr.la_fwd(q, q, v, g), lambda: gdr.la_bwd(q, q, v, g, v),
             lambda: gdr.la_step(q[0], q[0], v[0], g, state), lambda: gdr.qk_norm_fwd(q, q, w, w),
             lambda: gdr.qk_norm_bwd(q, q, q, q, w, w)]
    for f in calls:
        with pytest.raises(gdr.GdrError, match="CUDA tensor"):
            f()
    with pytest.raises(ValueError, match=r"\[B, T, H, K\]"):
        gdr.la_fwd(q[0], q[0], v[0], g)
    with pytest.raises(ValueError, match=r"\[R, H, K\]"):
        gdr.la_step(q, q, v, g, state)
    with pytest.raises(ValueError, match=r"\[..., H, D\]"):
        gdr.qk_norm_fwd(w, None, w, None)
    for channels in (0, 7, -2):
        with pytest.raises(ValueError, match="even"):
            gdr.rotation_table(4, channels, device="cpu")


def test_rotation_table(gdr):
    cos, sin = gdr.rotation_table(5000, 6, base=100.0, device="cpu")
    assert cos.shape == sin.shape == (5000, 3) and cos.dtype == torch.float32
    angle = torch.tensor(4999.0, dtype=torch.float64) * 100.0 ** (-2 / 3)
    assert abs(float(cos[4999, 2]) - float(torch.cos(angle))) < 1e-6
    assert float(cos[4999, 0]) == pytest.approx(float(torch.cos(torch.tensor(4999.0, dtype=torch.float64))), abs=1e-7)
    assert float(sin[3, 0]) == pytest.approx(float(torch.sin(torch.tensor(3.0, dtype=torch.float64))), abs=1e-7)
