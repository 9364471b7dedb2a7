"""Sequences that are really cut into segments (longer than any form leaves in one block: 1152 tokens with few heads):
what is not finite, invalid lengths, repeated calls."""
import ctypes
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import cu_of, spans
from tests.test_gpu_attention import both_types, put, run

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
LENS = [40, 1500, 0, 1400, 70]


def cut(gdr, q, lens):
    """Whether the forward makes three launches (of which the lengths on the device decide what they do)."""
    before = gdr.launch_count()
    gdr.la_fwd(q["q"][None], q["k"][None], q["v"][None], q["g"], cu_seqlens=cu_of(lens, "cuda"))
    return gdr.launch_count() - before == 3 and max(lens) > 1152


@both_types
@pytest.mark.parametrize("where", ["q", "k", "v", "do", "h0", "dht"])
@pytest.mark.parametrize("D", [128, 64, 20])
@pytest.mark.parametrize("value", [math.nan, math.inf], ids=str)
def test_cut_sequences_keep_to_themselves(gdr, dtype, where, D, value):
    q = put(ref.attention_inputs(LENS, 1, 2, D, D, dtype, seed=6))
    assert cut(gdr, q, LENS)
    clean = run(gdr, q, LENS, 1.0)
    at = [i for _, i, _ in spans(LENS)]
    for seq in (1, 3, 0, 4):
        r = dict(q)
        r[where] = q[where].clone()
        r[where][seq if where in ("h0", "dht") else slice(at[seq], at[seq] + LENS[seq])] = value
        got = run(gdr, r, LENS, 1.0)
        for n, i, j in spans(LENS):
            for k, v in got.items():
                mine, want = (u[n] if k in ("ht", "dh0") else u[i:j] for u in (v, clean[k]))
                assert n == seq or torch.equal(mine, want), (seq, n, k)


@both_types
@pytest.mark.parametrize("D", [128, 20])
def test_earlier_segments_do_not_see_what_is_not_a_number(gdr, dtype, D):
    q = put(ref.attention_inputs(LENS, 1, 1, D, D, dtype, seed=8))
    args = lambda r: [r[k][None] for k in ("q", "k", "v")] + [r["g"]]  # noqa: E731
    cu = cu_of(LENS, "cuda")
    clean, _ = gdr.la_fwd(*args(q), cu_seqlens=cu)
    at = 40 + 64 * 13 + 5  # in the fourteenth chunk of the sequence of 1500
    for where in ("q", "k", "v"):
        r = dict(q)
        r[where] = q[where].clone()
        r[where][at, 0] = math.nan
        got, ht = gdr.la_fwd(*args(r), cu_seqlens=cu)
        chunk = 40 + 64 * 13
        assert torch.equal(got[0, :chunk], clean[0, :chunk]) and torch.equal(got[0, 1540:], clean[0, 1540:])
        assert got[0, at, 0].isnan().any()
        if where != "q":
            assert got[0, 1539].isnan().any() and ht[1].isnan().any() and ht[[0, 2, 3, 4]].isfinite().all()


@both_types
@pytest.mark.parametrize("D", [128, 20])
def test_cut_results_repeat_bit_for_bit(gdr, dtype, D):
    lens = [1500, 77, 1400]
    q = put(ref.attention_inputs(lens, 2, 4, D, D, dtype, seed=4))
    assert cut(gdr, q, lens)
    a, b = run(gdr, q, lens, 1.0), run(gdr, q, lens, 1.0)
    assert all(torch.equal(a[k], b[k]) for k in a)


@both_types
@pytest.mark.parametrize("bad", [[0, 1400, 1300, 3000], [1, 1500, 3000], [0, 1500, 3001], [0, 1500, 2999]], ids=str)
@pytest.mark.parametrize("D", [64, 20])
def test_bad_lengths_of_cut_batches_touch_nothing(gdr, dtype, bad, D):
    from chunked_gated_delta_08_gb300 import attention_ops as ops
    T, N, H, HV = 3000, len(bad) - 1, 1, 2
    q = put(ref.attention_inputs([T], H, HV, D, D, dtype))
    cu = torch.tensor(bad, device="cuda")
    desc = ops.GdrLaDesc(1, T, H, HV, D, D, N, H * D, H * D, HV * D, HV * D, 1.0, 0 if dtype == F32 else 1, 0)
    full = lambda dt, *s: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
    a, s = (lambda t: t.data_ptr()), torch.cuda.current_stream().cuda_stream  # noqa: E731
    o, ht, dh0 = full(dtype, T, HV, D), full(F32, N, HV, D, D), full(F32, N, HV, D, D)
    dq, dk, dv = full(dtype, T, H, D), full(dtype, T, H, D), full(dtype, T, HV, D)
    head = [a(q["q"]), a(q["k"]), a(q["v"]), a(q["g"]), None, a(cu)]
    before = gdr.launch_count()
    assert gdr.lib().gdr_la_fwd(ctypes.byref(desc), *head, a(o), a(ht), s) == 0
    assert gdr.launch_count() - before == 3
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert gdr.lib().gdr_la_bwd(ctypes.byref(desc), *head, a(q["do"]), None, a(dq), a(dk), a(dv), a(dh0), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert all(t.eq(7.0).all() for t in (o, ht, dq, dk, dv, dh0))


@both_types
@pytest.mark.parametrize("D", [128, 20])
def test_each_head_of_cut_sequences(gdr, dtype, D):
    """Errors head by head and sequence by sequence: slow heads' large states hide nothing."""
    lens = [40, 1300, 0, 70]
    p = ref.attention_inputs(lens, 2, 2, D, D, dtype, seed=9, g=torch.tensor([-1.2, -0.004]))
    q = put(p)
    assert cut(gdr, q, lens)
    got = run(gdr, q, lens, D ** -0.5)
    d = {k: v.double() for k, v in p.items()}
    args = [d[k] for k in ("q", "k", "v", "g", "h0")]
    want = dict(zip(("o", "ht"), ref.attention(*args, lens, D ** -0.5)))
    want.update(zip(("dq", "dk", "dv", "dh0"), ref.attention_grads(*args, lens, D ** -0.5, d["do"], d["dht"])))
    for h in range(2):
        for n, i, j in spans(lens):
            for k, w in want.items():
                mine, there = (u[n, h] if k in ("ht", "dh0") else u[i:j, h] for u in (got[k], w))
                ref.close(mine, there, dtype, max(lens), f"{k} of head {h} in sequence {n}")
