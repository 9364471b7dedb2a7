"""States of linear attention after tens of thousands of tokens that all add to them: what a chunk's sum loses must
not pile up with the number of chunks."""
import math

import pytest
import torch

from tests.layer_reference import rel
from tests.test_gpu_attention import both_types

pytestmark = pytest.mark.gpu


def bound(dtype, T):
    """All terms are positive, so that their relative errors are the sum's: a product's 2^-21, or 2^-17 of bf16 inputs.  A
    chunk of 64 is added to the state in fp32: sqrt(T / 64) roundings of 2^-24, four for their spread.  Within a
    chunk's own sum, tensor cores cut off what they add up, by 2^-23 at most, eight times."""
    product = 2.0 ** -21 if dtype == torch.float32 else 2.0 ** -17
    return product + 4 * math.sqrt(T / 64) * 2.0 ** -24 + 8 * 2.0 ** -23


@both_types
@pytest.mark.parametrize("g", [0.0, -1e-5], ids=str)
@pytest.mark.parametrize("T", [4096, 32768])
@pytest.mark.parametrize("D,HV", [(16, 152), (72, 152), (16, 2)], ids=["many", "wide", "cut"])
def test_states_of_long_sequences(gdr, dtype, g, T, D, HV):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + D)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    q, k, v = rand(1, T, 1, D), rand(1, T, 1, D), rand(1, T, HV, D)
    decay = torch.full((HV,), g, device="cuda")
    before = gdr.launch_count()
    _, ht = gdr.la_fwd(q, k, v, decay, scale=1 / T)
    assert gdr.launch_count() - before == (1 if HV > 100 else 3)
    back = torch.exp(decay[0].double() * (T - 1 - torch.arange(T, device="cuda", dtype=torch.float64)))
    dh0 = gdr.la_bwd(q[:, :, :, :16], k[:, :, :, :16], v[..., :16].contiguous(), decay, v[..., :16].contiguous(),
                     scale=1 / T)[3]
    some = (0, 1, HV - 1)
    for h in some:
        want = (k[0, :, 0].double() * back[:, None]).t() @ v[0, :, h].double()
        err = rel(ht[0, h], want)
        assert err <= bound(dtype, T), f"ht of head {h}: {err:.2e} over {bound(dtype, T):.2e}"
        forth = back.flip(0) * math.exp(float(decay[0].double()))
        want = (q[0, :, 0, :16].double() * forth[:, None]).t() @ v[0, :, h, :16].double() / T
        err = rel(dh0[0, h], want)
        assert err <= bound(dtype, T), f"dh0 of head {h}: {err:.2e} over {bound(dtype, T):.2e}"
