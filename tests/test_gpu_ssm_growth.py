"""States that grow (a > 0, or a negative delta): the decays of a chunk of tokens
multiply to more than fp32 holds, or to less, where no state does.

Bounds, in roundings of 2^-24 beside the operators' own.  The exponent that a run
of 8 or 16 tokens adds up to, 96 here, is off by one rounding of itself for each of: a
times log2(e), its products with delta, delta's sum, its part in a factor; a value
is off by as much as its exponent is.  An exponential is off by up to four, and
the same one each time: once a token in a run, and three in the factor of each run that a
state is carried over.  The terms of a value have one sign, so the bound holds for
each value that is zero or an ordinary fp32 number; one below 2^-126, which fp32
holds to no relative precision, has to stay there.
"""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32 = torch.float32
NAMES = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")
SPAN = 96.0


def inputs(T, E, S, first_up, run):
    """Positive inputs whose states go up and down by e^96 every `run` tokens."""
    p = ref.scan_inputs([T], E, S, 1, F32, seed=T, d=False, z=False, dt_bias=False)
    up = (torch.arange(T) // run % 2 == 0) == first_up
    p["dt"] = torch.where(up, 0.5, -0.5)[:, None].expand(T, E).contiguous()
    p["a"] = torch.full((E, S), SPAN / run / 0.5)
    for k in ("b", "c", "dy", "dht", "h0"):
        p[k] = p[k].abs() + 0.5
    p["x"] = torch.zeros(T, E)
    return p


def call(gdr, p):
    q = {k: None if v is None else v.cuda() for k, v in p.items()}
    lead = lambda t: t[None]  # noqa: E731
    args = (lead(q["x"]), lead(q["dt"]), q["a"], lead(q["b"]), lead(q["c"]))
    before = gdr.launch_count()
    y, ht = gdr.ssm_fwd(*args, h0=q["h0"], dt_softplus=False)
    dx, ddt, da, db, dc, _, _, _, dh0 = gdr.ssm_bwd(*args, lead(q["dy"]), h0=q["h0"], dht=q["dht"], dt_softplus=False)
    assert gdr.launch_count() - before == 3 + 4  # several chunks
    return dict(y=y[0], ht=ht, dx=dx[0], ddt=ddt[0], da=da, db=db[0], dc=dc[0], dh0=dh0)


def definition(p, T):
    fn = lambda *v: ref.scan(*v, [T], False)  # noqa: E731
    y, ht = fn(*[ref.f64(p[k]) for k in NAMES])
    got = ref.grads(fn, [p[k] for k in NAMES], (p["dy"].double(), p["dht"].double()))
    return dict(zip(("y", "ht", "dx", "ddt", "da", "db", "dc", "dh0"), (y, ht, *got[:5], got[8])))


def each_close(got, want, T, run, names):
    bound = ref.tol(F32, T) + (4 * SPAN + 4 * run + 12 * -(-T // run)) * 2.0 ** -24
    for k in names:
        g, w = got[k].double().cpu(), want[k]
        tiny = torch.finfo(F32).tiny
        same = (g == w) | ((w.abs() > 0) & (w.abs() < tiny) & (g.abs() < tiny))
        off = torch.where(same, 0.0, (g - w).abs() / w.abs())  # NaN where g is not finite
        assert bool((off <= bound).all()), f"{k}: {float(off.max()):.2e} over {bound:.2e}"


@pytest.mark.parametrize("first_up", [True, False], ids=["up_first", "down_first"])
@pytest.mark.parametrize("T,E,S", [(600, 8, 16), (161, 5, 3)], ids=str)
@pytest.mark.parametrize("run", [16, 8], ids=["a_chunk", "within_a_chunk"])
def test_up_and_down(gdr, T, E, S, run, first_up):
    """Small states where they go up first, large ones where they go down first: e^96 is 5e41, and no value
    reaches 1e38.  So few channels are cut into chunks of 16 tokens."""
    p = inputs(T, E, S, first_up, run)
    for k in ("h0", "dht", "dy"):
        p[k] = p[k] * 1e-15
    if not first_up:
        p["h0"] = p["h0"] * 1e28
    want = definition(p, T)
    assert all(v.abs().max() < 1e38 for v in want.values())
    each_close(call(gdr, p), want, T, run, ("y", "ht", "dx", "ddt", "dh0"))


def test_nothing_times_a_large_factor(gdr):
    """Growth throughout: states that are zero until the last tokens, gradients that are zero after the first."""
    T = 400
    p = inputs(T, 8, 16, True, 16)
    p["dt"] = torch.full((T, 8), 0.5)
    p["h0"] = torch.zeros_like(p["h0"])
    p["dht"] = torch.zeros_like(p["dht"])
    p["x"][T - 5:] = 1
    p["dy"][8:] = 0
    want = definition(p, T)
    got = call(gdr, p)
    each_close(got, want, T, 16, want)
    assert want["y"][T - 5:].min() > 0 and want["dx"][:8].min() > 0
