"""The tests' 64-bit definitions against closed forms, and the plain forms of the
measured cases against them."""
import math

import pytest
import torch

from tests import attention_reference as ref

F64 = torch.float64


def test_attention_is_a_decayed_sum():
    """o_t = scale sum_{j <= t} e^{(t - j) g} (q_t . k_j) v_j + scale e^{(t + 1) g} h0^T q_t."""
    p = {k: v.double() for k, v in ref.attention_inputs([7], 2, 4, 3, 5, torch.float32).items()}
    o, ht = ref.attention(p["q"], p["k"], p["v"], p["g"], p["h0"], [7], 0.5)
    for h in range(4):
        g = float(p["g"][h])
        for t in range(7):
            want = math.exp((t + 1) * g) * p["h0"][0, h].t() @ p["q"][t, h // 2]
            for j in range(t + 1):
                want = want + math.exp((t - j) * g) * (p["q"][t, h // 2] @ p["k"][j, h // 2]) * p["v"][j, h]
            assert torch.allclose(o[t, h], 0.5 * want, rtol=1e-12, atol=1e-12)
        want = math.exp(7 * g) * p["h0"][0, h] + sum(
            math.exp((6 - j) * g) * torch.outer(p["k"][j, h // 2], p["v"][j, h]) for j in range(7))
        assert torch.allclose(ht[0, h], want, rtol=1e-12, atol=1e-12)


def test_attention_gradients_against_differences():
    lens = [4, 0, 3]
    p = {k: v.double() for k, v in ref.attention_inputs(lens, 1, 2, 3, 2, torch.float32).items()}
    args = [p[k] for k in ("q", "k", "v", "g", "h0")]
    grads = dict(zip(("q", "k", "v", "h0"), ref.attention_grads(*args, lens, 0.7, p["do"], p["dht"])))

    def loss(q):
        o, ht = ref.attention(*[q[k] for k in ("q", "k", "v", "g", "h0")], lens, 0.7)
        return float((o * p["do"]).sum() + (ht * p["dht"]).sum())
    gen = torch.Generator().manual_seed(1)
    for name, d in grads.items():
        for _ in range(3):
            to = torch.randn(p[name].shape, generator=gen, dtype=F64)
            up, down = (loss(dict(p, **{name: p[name] + e * to})) for e in (1e-5, -1e-5))
            assert abs((up - down) / 2e-5 - float((d * to).sum())) < 1e-6


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    p = ref.head_inputs(5, 2, 1, 8, 3, torch.float32)
    x, w = p["q"].double(), p["wq"].double()
    y = ref.heads(x, w, p["cos"].double(), p["sin"].double(), p["positions"], interleaved)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    at = torch.arange(3)
    a, b = (2 * at, 2 * at + 1) if interleaved else (at, at + 3)
    unit = torch.complex(p["cos"].double(), p["sin"].double())[p["positions"]][:, None]
    turned = torch.complex(n[..., a], n[..., b]) * unit
    assert torch.allclose(y[..., a], turned.real) and torch.allclose(y[..., b], turned.imag)
    assert torch.equal(y[..., 6:], n[..., 6:])
    q = dict(p, positions=torch.tensor([0, -1, 2, -5, 1]))
    z = ref.heads(x, w, p["cos"].double(), p["sin"].double(), q["positions"], interleaved)
    assert (z[1] == 0).all() and (z[3] == 0).all() and (z[0] != 0).all()
