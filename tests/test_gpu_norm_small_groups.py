"""The norm's 8-bit output where a scale group holds next to nothing: values so
small that 448 / amax passes the largest fp32 number."""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6
LEAST = 448.0 / torch.finfo(F32).max  # the least amax whose 448 / amax is an fp32 number


@pytest.mark.parametrize("E", [40, 300, 512, 2048, 4100], ids=lambda e: "E%d" % e)  # warp, scalar, vectors, long rows
@pytest.mark.parametrize("quant", ["row", "group"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("size", [1e-35, 1e-36, 1e-37, 2e-38, 1e-40], ids=str)
def test_groups_of_next_to_nothing(gdr, E, quant, dtype, size):
    g = torch.Generator().manual_seed(E)
    x = torch.randn(3, E, generator=g).to(dtype)
    x[:, 1::3] = 0  # zeros beside the small values
    x[2] = 0
    w = torch.full((E,), size).to(dtype)
    if quant == "group" and E > 128:
        w[128:256] = 1  # an ordinary group beside them
    y8, scale, _ = gdr.norm_fwd(x.cuda(), w.cuda(), eps=EPS, quant=quant)
    want = ref.norm(x.double(), w.double(), EPS)
    width = E if quant == "row" else 128
    top = torch.stack([p.abs().amax(1) for p in want.split(width, 1)], 1)
    scales = torch.where(top > 0, top.clamp(min=LEAST) / 448, torch.ones_like(top))
    got = scale.double().cpu().view(3, -1)
    # fp32 values down here are whole multiples of 2^-149: one such step, and the roundings of the sum and the value
    assert ((got - scales).abs() <= scales * ref.tol(F32, E) + 2.0 ** -149).all()
    assert torch.isfinite(y8.float()).all() and (got > 0).all()
    assert y8.float().cpu()[x == 0].eq(0).all()
    # half an e4m3 step of the value, or half the smallest subnormal; two steps of 2^-149 in the value itself
    spread = got.repeat_interleave(width, 1)[:, :E]
    back = y8.double().cpu() * spread
    bound = (want.abs() * 2.0 ** -4 + spread * 2.0 ** -10) * (1 + 1e-4) + 448 * 2.0 ** -149
    assert ((back - want).abs() <= bound).all()


@pytest.mark.parametrize("quant", ["row", "group"])
def test_the_scale_is_of_the_largest_value_down_to_the_least(gdr, quant):
    """One column, of which the norm makes its weight: amax around the border, the byte always +448 above it."""
    for mul in (0.25, 0.5, 1 + 2.0 ** -20, 2.0, 2.0 ** 20):
        amax = LEAST * mul
        x, w = torch.ones(1, 1, device="cuda"), torch.full((1,), amax, device="cuda")
        y8, scale, _ = gdr.norm_fwd(x, w, eps=0.0, quant=quant)
        assert float(y8.float()) == (448.0 if mul >= 1 else 448.0 * mul)
        assert abs(float(scale) * 448 - LEAST * max(mul, 1)) <= 448 * 2.0 ** -149 + amax * 2.0 ** -22
