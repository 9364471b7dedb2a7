"""Sequences of one packed batch do not reach each other: what is not a number
in one leaves the results of the others as they are, to the bit, where several
chunks of tokens are carried one into the next."""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# the borders lie inside chunks of 16, 32, 48 and 64 tokens
LENS = [100, 30, 90]
PER_TOKEN = ("dx", "ddt", "db", "dc", "dz")


def calls(gdr, p, cu):
    lead = lambda t: t[None]  # noqa: E731
    args = (lead(p["x"]), lead(p["dt"]), p["a"], lead(p["b"]), lead(p["c"]))
    kw = dict(d=p["d"], z=lead(p["z"]), dt_bias=p["dt_bias"], h0=p["h0"], cu_seqlens=cu)
    before = gdr.launch_count()
    y, ht = gdr.ssm_fwd(*args, **kw)
    assert gdr.launch_count() - before == 3  # local, carry, main
    before = gdr.launch_count()
    dx, ddt, _, db, dc, _, dz, _, dh0 = gdr.ssm_bwd(*args, lead(p["dy"]), dht=p["dht"], **kw)
    assert gdr.launch_count() - before == 4  # local, carry, main, sums
    return dict(y=y[0], dx=dx[0], ddt=ddt[0], db=db[0], dc=dc[0], dz=dz[0], ht=ht, dh0=dh0)


@pytest.mark.parametrize("where", ["x", "dt", "b", "c", "z", "dy", "dht", "h0"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("dtype,E,S,G", [(F32, 24, 12, 2), (BF16, 64, 16, 1), (BF16, 40, 33, 1)], ids=str)
def test_other_sequences_keep_their_bits(gdr, dtype, E, S, G, value, where):
    p = ref.scan_inputs(LENS, E, S, G, dtype, seed=S, device="cuda")
    cu = ref.cu_of(LENS, "cuda")
    clean = calls(gdr, p, cu)
    for seq in range(3):
        q = dict(p)
        t = q[where] = p[where].clone()
        if where in ("dht", "h0"):
            t[seq].view(-1)[::5] = value
        else:  # the second token and the last but one
            i, j = sum(LENS[:seq]), sum(LENS[:seq + 1])
            t[[i + 1, j - 2]] = value
        got = calls(gdr, q, cu)
        for n, i, j in ref.spans(LENS):
            if n == seq:
                continue
            for k, v in got.items():
                mine, want = (v[n], clean[k][n]) if k in ("ht", "dh0") else (v[i:j], clean[k][i:j])
                assert torch.isfinite(want).all() and torch.equal(mine, want), (k, seq, n)


@pytest.mark.parametrize("where", ["dt", "c", "z", "dy"])
def test_gradients_before_the_spoilt_sequence(gdr, where):
    """Against the definition of the first sequence alone."""
    p = ref.scan_inputs(LENS, 24, 16, 1, F32, seed=1)
    names = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")
    one = {k: v[:1] if k in ("h0", "dht") else v if k in ("a", "d", "dt_bias") else v[:100] for k, v in p.items()}
    want = ref.grads(lambda *v: ref.scan(*v, [100]), [one[k] for k in names], (one["dy"].double(), one["dht"].double()))
    q = {k: v.cuda() for k, v in p.items()}
    q[where][100:] = float("nan")
    got = calls(gdr, q, ref.cu_of(LENS, "cuda"))
    for k in PER_TOKEN:
        ref.close(got[k][:100], want[names.index(k[1:])], 100, k)
    ref.close(got["dh0"][:1], want[8], 100, "dh0")
