"""Padding tokens of the heads' norm against a rotation table whose rows are not numbers: a table is read for tokens
that have a place in it alone."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.test_gpu_heads import both_types, check, put, run

pytestmark = pytest.mark.gpu


@both_types
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("bad", [math.nan, math.inf], ids=str)
@pytest.mark.parametrize("D,R", [(64, 32), (128, 32), (16, 4), (12, 5)])
def test_padding_does_not_read_the_table(gdr, dtype, interleaved, bad, D, R):
    p = ref.head_inputs(20, 3, 2, D, R, dtype, seed=4)
    p["positions"].clamp_(min=1)
    pad = [0, 7, 8, 19]
    p["positions"][pad] = torch.tensor([-1, -1, -100, -2 ** 40])
    q = put(p)
    for k in ("cos", "sin"):
        q[k] = q[k].clone()
        q[k][0] = bad
    got = run(gdr, q, interleaved)
    check(got, p, interleaved)
    for k in ("yq", "yk", "dq", "dk"):
        assert (got[k][pad] == 0).all(), k
    assert gdr.device_status() == 0


@both_types
@pytest.mark.parametrize("D,R", [(64, 32), (12, 5)])
def test_tokens_past_a_table_do_not_read_it(gdr, dtype, D, R):
    p = put(ref.head_inputs(20, 3, 2, D, R, dtype, seed=4))
    for k in ("cos", "sin"):
        p[k][0] = math.nan
    p["positions"].clamp_(min=1)
    p["positions"][5] = p["cos"].shape[0]
    got = run(gdr, p, False)
    assert gdr.device_status() == gdr.GDR_ERR_POSITION
    for k, v in got.items():
        assert v.isfinite().all(), k
        assert k.startswith("dw") or (v[5] == 0).all(), k
