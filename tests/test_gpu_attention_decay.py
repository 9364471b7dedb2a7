"""Decays of linear attention where nothing new covers the old state: fast heads and slow ones, each head by
itself, in one block's chunks and in sequences that are cut into segments.

Tolerances are those of attention_reference, and where a state is only decayed: a factor r^n = e^(g n) has the
rounding of g n, |g n| 2^-24 of it, and a few of exp's own and of the product, eight of 2^-24 at most; over all
factors of T tokens (|g| T + 8 factors) 2^-24."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import cu_of, rel, spans
from tests.test_gpu_attention import both_types, put, run, wanted

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DECAYS = [-0.05, -0.1, -0.25, -0.3]


@both_types
@pytest.mark.parametrize("D", [64, 128, 20])
@pytest.mark.parametrize("T", [64, 200, 256])
@pytest.mark.parametrize("g", DECAYS + [-0.01, -0.011], ids=str)
def test_the_gradient_of_a_state_that_is_only_decayed(gdr, dtype, D, T, g):
    """Without a gradient of o, dh0 = r^T dht; ht of tokens without keys is r^T h0."""
    p = ref.attention_inputs([T], 1, 1, D, D, dtype, seed=T, g=torch.tensor([g]))
    p["do"].zero_()
    p["k"].zero_()
    got = run(gdr, put(p), [T], 1.0)
    factor, g = math.exp(T * float(p["g"][0].double())), abs(g)
    bound = (g * T + 8 * (T // 64 + 1)) * 2.0 ** -24
    for out, of in (("dh0", "dht"), ("ht", "h0")):
        err = rel(got[out], p[of].double() * factor)
        assert err <= bound, f"{out}: {err:.3e} over {bound:.3e}"


@both_types
@pytest.mark.parametrize("D", [64, 72, 20])
@pytest.mark.parametrize("lens", [[130, 64, 5, 400], [1500, 40]], ids=["whole", "cut"])
def test_each_head_behind_tokens_that_add_nothing(gdr, dtype, D, lens):
    """The last tokens have no keys and the first ones no gradient, as many as leave e^-60 of the state."""
    H = len(DECAYS)
    p = ref.attention_inputs(lens, H, H, D, D, dtype, seed=D, g=torch.tensor(DECAYS))
    for n, i, j in spans(lens):
        for h, g in enumerate(DECAYS):
            z = min(j - i - 1, int(-60 / g))
            p["k"][j - z:j, h] = 0
            p["do"][i:i + z, h] = 0
    want, q = wanted(p, lens, D ** -0.5), put(p)
    if max(lens) > 1152:  # longer than what is left in one block by any form
        before = gdr.launch_count()
        gdr.la_fwd(q["q"][None], q["k"][None], q["v"][None], q["g"], cu_seqlens=cu_of(lens, "cuda"))
        assert gdr.launch_count() - before == 3
    got = run(gdr, q, lens, D ** -0.5)
    for h in range(H):
        for k in ("o", "dq", "dk", "dv"):
            ref.close(got[k][:, h], want[k][:, h], dtype, max(lens), f"{k} of head {h}")
        for n, i, j in spans(lens):
            what = f"of head {h} in sequence {n}"
            for k in ("ht", "dh0"):
                ref.close(got[k][n, h], want[k][n, h], dtype, max(lens), f"{k} {what}")
            if max(lens) <= 1152:
                # what the old state alone gives, at the far end (bf16 holds it: e^-60 is in its range)
                ref.close(got["o"][j - 1, h], want["o"][j - 1, h], dtype, max(lens), f"last o {what}")
                ref.close(got["dv"][i, h], want["dv"][i, h], dtype, max(lens), f"first dv {what}")


@both_types
@pytest.mark.parametrize("D", [64, 20])
def test_cut_and_whole_sequences_decay_alike(gdr, dtype, D):
    """The same sequence beside so many heads that it stays whole, and by itself; and token by token."""
    T, many = 1400, 152
    p = ref.attention_inputs([T], many, many, D, D, dtype, seed=5, g=torch.full((many,), -0.1))
    p["k"][T - 400:] = 0
    q = put(p)
    whole = gdr.la_fwd(q["q"][None], q["k"][None], q["v"][None], q["g"], h0=q["h0"])[1]
    one = [q[k][None, :, :1].contiguous() for k in ("q", "k", "v")]
    before = gdr.launch_count()
    cut = gdr.la_fwd(*one, q["g"][:1].clone(), h0=q["h0"][:, :1].contiguous())[1]
    assert gdr.launch_count() - before == 3
    ref.close(cut[0, 0], whole[0, 0].double(), dtype, T, "cut and whole")
    state = whole.new_zeros(1, 1, D, D)
    for t in range(T - 700, T):  # what came before has left e^-30 of what these leave
        gdr.la_step(one[0][:, t], one[1][:, t], one[2][:, t], q["g"][:1].clone(), state)
    ref.close(cut[0, 0], state[0, 0].double(), dtype, T, "cut and token by token")
