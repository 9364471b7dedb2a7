"""Single tokens of linear attention over thousands of steps at slow decays."""
import math

import pytest
import torch

from tests.layer_reference import rel
from tests.test_gpu_attention import both_types

pytestmark = pytest.mark.gpu


@both_types
def test_slow_decays_over_many_steps(gdr, dtype):
    """Thousands of tokens that add nothing leave e^(n g) of the state.

    Each step rounds the state to a mantissa m of 24 bits.  Where m g is many units, roundings are independent: sqrt(n)
    2^-24, four for their spread.  Where it changes slowly from step to step (by m g^2), they are a sawtooth of that
    period, whose sums are an eighth of 1 / (m g^2) units at most: 1 / (8 m^2 g^2) of the state, m at least 2^23.
    (A factor e^g rounded once and for all would leave 1e-4 at each of these.)"""
    n, K, V = 8192, 16, 24
    g = torch.tensor([-1e-5, -3e-5, -1e-4, -1e-3, 1e-5])
    first = torch.randn(2, len(g), K, V, generator=torch.Generator().manual_seed(0))
    state = first.cuda()
    z = torch.zeros(2, len(g), K, dtype=dtype, device="cuda")
    v, gd = torch.zeros(2, len(g), V, dtype=dtype, device="cuda"), g.cuda()
    for _ in range(n):
        gdr.la_step(z, z, v, gd, state)
    for h in range(len(g)):
        x = float(g[h].double())
        err = rel(state[:, h], first[:, h].double() * math.exp(n * x))
        bound = 1 / (8 * 2.0 ** 46 * x * x) + 4 * math.sqrt(n) * 2.0 ** -24
        assert err <= bound, f"g = {x}: {err:.3e} over {bound:.3e}"


@both_types
@pytest.mark.parametrize("g", [0.0, -0.3, -0.7, -5.0, -200.0, -math.inf], ids=str)
def test_fast_decays_of_single_tokens(gdr, dtype, g):
    """Three tokens that add nothing: three factors, each off by eight roundings at most and the one of its argument."""
    first = torch.randn(1, 1, 8, 8, generator=torch.Generator().manual_seed(1))
    state, z, gd = first.cuda(), torch.zeros(1, 1, 8, dtype=dtype, device="cuda"), torch.tensor([g], device="cuda")
    for _ in range(3):
        gdr.la_step(z, z, z, gd, state)
    want = first.double() * math.exp(3 * float(gd.double()))
    if g < -25:  # below fp32's range, or nothing
        assert (state == 0).all()
    else:
        assert rel(state, want) <= 3 * (8 + abs(g)) * 2.0 ** -24
