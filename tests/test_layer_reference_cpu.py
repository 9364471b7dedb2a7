"""The 64-bit definitions that the layer operators' GPU tests compare with:
closed forms, gradients against differences, and planted mistakes that the
comparisons have to see."""
import math

import pytest
import torch

from tests import layer_reference as ref


def test_norm_closed_form():
    s = torch.tensor([[3.0, 4.0]], dtype=torch.float64)
    w = torch.tensor([1.0, 2.0], dtype=torch.float64)
    got = ref.norm(s, w, 0.0)
    r = math.sqrt(12.5)
    assert torch.allclose(got, torch.tensor([[3 / r, 8 / r]], dtype=torch.float64), rtol=1e-15)


def test_conv_closed_form():
    """An impulse gives the filter backwards, and reaches the state."""
    x = torch.zeros(5, 1, dtype=torch.float64)
    x[1] = 1
    w = torch.tensor([[2.0, 3.0, 5.0]], dtype=torch.float64)
    y, st = ref.conv(x, w, None, torch.zeros(1, 2, 1, dtype=torch.float64), [5], silu=False)
    assert y[:, 0].tolist() == [0, 5, 3, 2, 0] and st[0, :, 0].tolist() == [0, 0]


def test_conv_state_carries_a_cut_sequence():
    p = ref.conv_inputs([9], 3, 4, torch.float32)
    x, w, b, s0 = (p[k].double() for k in ("x", "weight", "bias", "s0"))
    whole, end = ref.conv(x, w, b, s0, [9])
    for cut in (1, 2, 5):
        y1, mid = ref.conv(x[:cut], w, b, s0, [cut])
        y2, st = ref.conv(x[cut:], w, b, mid, [9 - cut])
        assert torch.allclose(torch.cat([y1, y2]), whole, atol=1e-14) and torch.equal(st, end)


def test_scan_closed_form():
    """Constant delta and b = c = 1: a geometric sum."""
    T, a, delta = 6, -0.7, 0.3
    one = torch.ones(T, 1, dtype=torch.float64)
    y, ht = ref.scan(one, one * delta, torch.tensor([[a]], dtype=torch.float64), one[:, :, None], one[:, :, None], None,
                     None, None, torch.zeros(1, 1, 1, dtype=torch.float64), [T], softplus=False)
    k = math.exp(a * delta)
    want = [delta * (1 - k ** (t + 1)) / (1 - k) for t in range(T)]
    assert torch.allclose(y[:, 0], torch.tensor(want, dtype=torch.float64), rtol=1e-13)
    assert abs(float(ht) - want[-1]) < 1e-13


def test_gradients_against_differences():
    """Automatic differentiation of the definitions against central differences."""
    def check(fn, args):
        leaves = tuple(t.detach().double().requires_grad_() for t in args)
        assert torch.autograd.gradcheck(fn, leaves, eps=1e-6, atol=1e-6, rtol=1e-5)
    g = torch.Generator().manual_seed(3)
    check(lambda s, w: ref.norm(s, w, 1e-6), (torch.randn(2, 5, generator=g), torch.randn(5, generator=g)))
    lens = [3, 0, 1, 4]
    p = ref.conv_inputs(lens, 2, 3, torch.float32)
    check(lambda *t: ref.conv(*t, lens), [p[k] for k in ("x", "weight", "bias", "s0")])
    q = ref.scan_inputs([3, 0, 2], 4, 3, 2, torch.float32)
    check(lambda *t: ref.scan(*t, [3, 0, 2]), [q[k] for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")])


MISTAKES = {
    "decay_of_the_token_before": lambda q: dict(q, dt=torch.cat([q["dt"][:1], q["dt"][:-1]])),
    "b_for_c": lambda q: dict(q, c=q["b"]),
    "no_bias": lambda q: dict(q, dt_bias=torch.zeros_like(q["dt_bias"])),
    "groups_interleaved": lambda q: dict(q, b=q["b"].flip(1)),
    "no_initial_state": lambda q: dict(q, h0=torch.zeros_like(q["h0"])),
    "gate_dropped": lambda q: dict(q, z=None),
    "skip_dropped": lambda q: dict(q, d=None),
    "one_sequence_of_two": lambda q: dict(q, lens=[sum(q["lens"]), 0]),
}


@pytest.mark.parametrize("name", MISTAKES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_planted_mistakes_exceed_the_tolerance(name, dtype):
    lens = [20, 12]
    q = dict(ref.scan_inputs(lens, 6, 4, 2, dtype, seed=5), lens=lens)
    names = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")
    run = lambda v: ref.scan(*[ref.f64(v[k]) for k in names], v["lens"])[0]  # noqa: E731
    assert ref.rel(run(MISTAKES[name](q)), run(q)) > 4 * ref.tol(dtype, 32)
