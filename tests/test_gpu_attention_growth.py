"""Heads of linear attention whose states grow, over segments that grow them past fp32's range."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.test_gpu_attention import both_types, put, run, wanted

pytestmark = pytest.mark.gpu


@both_types
@pytest.mark.parametrize("D", [64, 20])
def test_growing_heads_over_segments_without_a_state(gdr, dtype, D):
    """e^(g L) of a segment is past fp32's range, but all states are in it: nothing has entered them yet."""
    T, g = 1500, 1.0
    p = ref.attention_inputs([T], 1, 1, D, D, dtype, seed=6, g=torch.tensor([g]))
    p["h0"].zero_()
    p["dht"].zero_()
    p["k"][:T - 50] = 0
    p["do"][50:] = 0
    want, got = wanted(p, [T], 1.0), run(gdr, put(p), [T], 1.0)
    for k in got:
        assert got[k].isfinite().all(), k
        ref.close(got[k], want[k], dtype, T, k)


@both_types
@pytest.mark.parametrize("D", [64, 20])
@pytest.mark.parametrize("g,at", [(0.36, 1020), (0.72, 1150)])
def test_growing_heads_over_a_segment(gdr, dtype, D, g, at):
    """e^(g L) is past fp32's range for segments of 256 tokens, or of 128; the state that grows by it is not."""
    T = 1300
    p = ref.attention_inputs([T], 1, 1, D, D, dtype, seed=7, g=torch.tensor([g]))
    for k in ("k", "v"):
        p[k][:at] = 0
        p[k][at] *= 1e-15
        p[k][at + 1:] = 0
    q = put(p)
    ht = gdr.la_fwd(q["q"][None], q["k"][None], q["v"][None], q["g"])[1]
    want = p["k"][at, 0].double()[:, None] * p["v"][at, 0].double() * math.exp((T - 1 - at) * p["g"].double()[0])
    assert ht.isfinite().all()
    ref.close(ht[0, 0], want, dtype, T)
