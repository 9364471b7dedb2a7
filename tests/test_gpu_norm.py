"""Root-mean-square norm with the residual's addition, its 8-bit output and its
backward, on the GPU against the 64-bit definition."""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# around the widths at which the kernels change: groups of 128, rows of a warp, of registers, of memory
WIDTHS = [1, 7, 64, 127, 128, 130, 256, 264, 500, 512, 1000, 1024, 2048, 2052, 4096, 4104, 8192, 8200, 16384, 16392,
          20001]
EPS = 1e-6


def rows(M, E, dtype, seed, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * mul).to(dtype)


def weight_of(E, dtype, seed=9):
    return (1 + 0.1 * rows(1, E, F32, seed)[0]).to(dtype)


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("dtype,res", [(F32, None), (BF16, None), (BF16, BF16), (BF16, F32), (F32, F32)],
                         ids=["fp32", "bf16", "bf16_res", "bf16_res32", "fp32_res"])
def test_forward(gdr, E, dtype, res):
    for M in (1, 5):
        x, w = rows(M, E, dtype, E), weight_of(E, F32 if M == 5 else dtype)
        r = None if res is None else rows(M, E, res, E + 1, 3.0)
        y, s = gdr.norm_fwd(x.cuda(), w.cuda(), None if r is None else r.cuda(), eps=EPS)
        stored = x if r is None else ref.stored_sum(x, r)
        if r is None:
            assert s is None
        else:  # the sum of two bf16 or fp32 values, rounded once: the same bits but where fp32 rounds the sum first
            assert s.dtype == res and ref.rel(s, stored) <= 2.0 ** -24 + (0 if res == F32 else 2.0 ** -16)
            stored = s.cpu()
        ref.close(y, ref.norm(stored.double(), w.double(), EPS), E / M, "y")


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("quant", ["row", "group"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_eight_bits(gdr, E, quant, dtype):
    M = 3
    x, w = rows(M, E, dtype, E), weight_of(E, dtype)
    x[1] = 0  # a row of zeros: scale 1
    y8, scale, s = gdr.norm_fwd(x.cuda(), w.cuda(), eps=EPS, quant=quant)
    assert s is None and y8.dtype == torch.float8_e4m3fn and y8.shape == x.shape
    want = ref.norm(x.double(), w.double(), EPS)
    width = E if quant == "row" else 128
    groups = want.split(width, 1)
    top = torch.stack([g.abs().amax(1) for g in groups], 1)
    scales = torch.where(top > 0, top / 448, torch.ones_like(top))
    ref.close(scale, scales[:, 0] if quant == "row" else scales, E, "scale")
    assert scale.cpu().view(M, -1)[1].eq(1).all() and y8.float()[1].eq(0).all()
    # each byte stands for a value within half an e4m3 step of y / scale: 2^-4 of it, or half the smallest
    # subnormal, 2^-10; fp32 roundings move y by a few 2^-24
    back = y8.double().cpu() * scales.repeat_interleave(width, 1)[:, :E]
    step = want.abs() * 2.0 ** -4 + scales.repeat_interleave(width, 1)[:, :E] * 2.0 ** -10
    assert ((back - want).abs() <= step * (1 + 1e-4)).all()
    again = gdr.norm_fwd(x.cuda(), w.cuda(), eps=EPS, quant=quant)[0]
    assert torch.equal(again.view(torch.uint8), y8.view(torch.uint8))


@pytest.mark.parametrize("quant", ["row", "group"])
def test_eight_bits_with_a_residual(gdr, quant):
    x, r, w = rows(4, 300, BF16, 1), rows(4, 300, F32, 2, 3.0), weight_of(300, BF16)
    y8, scale, s = gdr.norm_fwd(x.cuda(), w.cuda(), r.cuda(), eps=EPS, quant=quant)
    y, s2 = gdr.norm_fwd(x.cuda().float(), w.cuda().float(), r.cuda(), eps=EPS)
    assert torch.equal(s, s2)
    spread = scale.view(4, -1).repeat_interleave(300 if quant == "row" else 128, 1)[:, :300]
    assert ((y8.float() * spread - y).abs() <= (y.abs() * 2.0 ** -4 + spread * 2.0 ** -10) * (1 + 1e-4)).all()


def test_nan_and_infinity_stay_in_their_rows(gdr):
    x, w = rows(4, 300, F32, 3), weight_of(300, F32)
    x[1, 7], x[2, 290] = float("nan"), float("inf")
    y, _ = gdr.norm_fwd(x.cuda(), w.cuda(), eps=EPS)
    y = y.cpu()
    assert y[1].isnan().all() and y[2, 290].isnan() and torch.isfinite(y[[0, 3]]).all()
    assert y[2, :290].eq(0).all()  # finite over infinity
    y8, scale, _ = gdr.norm_fwd(x.cuda(), w.cuda(), eps=EPS, quant="group")
    y8, scale = y8.float().cpu(), scale.cpu()
    assert y8[1].isnan().all() and scale[1].isnan().all()
    assert scale[2, 2].isnan() and scale[2, :2].eq(1).all() and torch.isfinite(scale[[0, 3]]).all()


def test_rows_of_a_wider_tensor(gdr):
    wide = rows(6, 3 * 264, BF16, 4).cuda()
    for lo in (0, 264, 3):  # aligned, aligned, not
        x = wide[:, lo:lo + 264]
        res = wide[:, 264:528]
        w = weight_of(264, BF16).cuda()
        y, s = gdr.norm_fwd(x, w, res)
        y2, s2 = gdr.norm_fwd(x.contiguous(), w, res.contiguous())
        assert torch.equal(s, s2)
        assert ref.rel(y, y2) <= 2 * ref.tol(BF16, 264)
        a = gdr.norm_bwd(x, res, w, ds=x)
        b = gdr.norm_bwd(x.contiguous(), res.contiguous(), w, ds=x.contiguous())
        for p, q in zip(a, b):
            assert ref.rel(p, q) <= 2 * ref.tol(p.dtype, 264)


def test_shapes_of_several_dimensions_and_empty(gdr):
    x, w = rows(6, 40, BF16, 5).cuda().view(2, 3, 40), weight_of(40, BF16).cuda()
    y, s = gdr.norm_fwd(x, w, x)
    assert y.shape == s.shape == (2, 3, 40)
    y8, scale, _ = gdr.norm_fwd(x, w, quant="row")
    assert scale.shape == (2, 3) and gdr.norm_fwd(x, w, quant="group")[1].shape == (2, 3, 1)
    e = x[:0]
    assert gdr.norm_fwd(e, w)[0].shape == (0, 3, 40)
    dx, _, dw = gdr.norm_bwd(e, e, w)
    assert dx.shape == (0, 3, 40) and dw.eq(0).all()


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=["fp32", "bf16", "bf16_s32"])
def test_backward(gdr, E, dtype, res):
    for M, with_ds in ((1, True), (70, False)):
        s, dy, w = rows(M, E, res, E, 3.0), rows(M, E, dtype, E + 1), weight_of(E, dtype)
        ds = rows(M, E, res, E + 2) if with_ds else None
        dx, dres, dw = gdr.norm_bwd(dy.cuda(), s.cuda(), w.cuda(), ds=None if ds is None else ds.cuda(), eps=EPS)
        assert dx.dtype == dtype and dres.dtype == res and dw.dtype == F32
        assert (dres is dx) == (dtype == res)
        gs, gw = ref.grads(lambda a, b: (ref.norm(a, b, EPS),), (s, w), (dy.double(),))
        if ds is not None:
            gs = gs + ds.double()
        if E > 1:  # at one column the norm does not depend on s, and its gradient is rounding
            ref.close(dx, gs, E, "dx")
            ref.close(dres, gs, E, "dres")
        ref.close(dw, gw, max(M, E), "dweight")


def test_backward_over_many_rows(gdr):
    """More rows than blocks, so that each block takes several; and the same bits each time."""
    M, E = 3001, 264
    s, dy, w = rows(M, E, F32, 1, 3.0), rows(M, E, F32, 2), weight_of(E, F32)
    got = [gdr.norm_bwd(dy.cuda(), s.cuda(), w.cuda(), eps=EPS) for _ in range(2)]
    assert all(torch.equal(p, q) for p, q in zip(*got))
    gs, gw = ref.grads(lambda a, b: (ref.norm(a, b, EPS),), (s, w), (dy.double(),))
    ref.close(got[0][0], gs, E, "dx")
    ref.close(got[0][2], gw, M, "dweight")


def test_gradient_against_differences(gdr):
    """Central differences of the forward, in fp32: L is off by 2^-24 of its terms' norm, twice, over 2 h."""
    g = torch.Generator().manual_seed(8)
    s, w, dy, v = (torch.randn(4, 96, generator=g).cuda() for _ in range(4))
    w = w[0].contiguous()
    h = 1e-2
    up, down = (gdr.norm_fwd(s + k * v, w)[0].double() for k in (h, -h))
    diff = float(((up - down) * dy.double()).sum()) / (2 * h)
    got = float((gdr.norm_bwd(dy, s, w)[0].double() * v.double()).sum())
    size = float(dy.double().norm() * up.norm())
    assert abs(diff - got) <= size * (2.0 ** -23 * 8 / h + h * h)


@pytest.mark.parametrize("call,error", [
    (lambda g, x, w: g.norm_fwd(x, w[:-1]), ValueError),
    (lambda g, x, w: g.norm_fwd(x, w.double()), RuntimeError),
    (lambda g, x, w: g.norm_fwd(x.half(), w), RuntimeError),
    (lambda g, x, w: g.norm_fwd(x, w, x[:, :8]), ValueError),
    (lambda g, x, w: g.norm_fwd(x, w, x.float().half()), RuntimeError),
    (lambda g, x, w: g.norm_fwd(x, w, quant="tensor"), ValueError),
    (lambda g, x, w: g.norm_fwd(x.t(), w[:4].contiguous()), RuntimeError),
    (lambda g, x, w: g.norm_fwd(x, w, eps=-1.0), ValueError),
    (lambda g, x, w: g.norm_bwd(x, x, w, ds=x.float()), RuntimeError),
    (lambda g, x, w: g.norm_fwd(x, w.cpu()), RuntimeError)])
def test_refusals(gdr, call, error):
    x, w = rows(4, 64, BF16, 1).cuda(), weight_of(64, BF16).cuda()
    with pytest.raises(error):
        call(gdr, x, w)
