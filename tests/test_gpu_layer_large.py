"""The layer operators past 2^31 elements: the last rows, sequences and slots
give what a small call on them gives."""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
E, M = 2048, 2 ** 31 // 4096 + 5003  # rows of a projection of 2 E: offsets end past 2^31 elements
TAIL = 40


@pytest.fixture(scope="module")
def wide():
    """The halves of one wide projection's output, zero but for the last tokens."""
    t = torch.zeros(1, M, 2 * E, dtype=BF16, device="cuda")
    g = torch.Generator().manual_seed(1)
    t[0, M - TAIL - 8:] = torch.randn(TAIL + 8, 2 * E, generator=g).to(BF16)
    yield t
    del t
    torch.cuda.empty_cache()


def test_norm_rows(gdr, wide):
    x, w = wide[0], torch.ones(2 * E, dtype=BF16, device="cuda")
    y, s = gdr.norm_fwd(x, w, x)
    y2, s2 = gdr.norm_fwd(x[-TAIL:].contiguous(), w, x[-TAIL:].contiguous())
    assert torch.equal(y[-TAIL:], y2) and torch.equal(s[-TAIL:], s2)
    del y, s
    dx, _, _ = gdr.norm_bwd(x, x, w, ds=x)
    dx2, _, _ = gdr.norm_bwd(x[-TAIL:].contiguous(), x[-TAIL:].contiguous(), w, ds=x[-TAIL:].contiguous())
    assert torch.equal(dx[-TAIL:], dx2)


def test_convolution_of_the_last_sequence(gdr, wide):
    p = ref.conv_inputs([TAIL], E, 4, BF16, device="cuda")
    cu = torch.tensor([0, M - TAIL, M], dtype=torch.int64, device="cuda")
    x, dy = wide[..., :E], wide[..., E:]
    s0, dst = torch.cat([p["s0"], p["s0"]]), torch.cat([p["dst"], p["dst"]])
    y, st = gdr.conv_fwd(x, p["weight"], bias=p["bias"], s0=s0, cu_seqlens=cu)
    dx, _, _, ds0 = gdr.conv_bwd(x, p["weight"], dy, bias=p["bias"], s0=s0, dst=dst, cu_seqlens=cu)
    tail = lambda t: t[:, M - TAIL:].contiguous()  # noqa: E731
    y2, st2 = gdr.conv_fwd(tail(x), p["weight"], bias=p["bias"], s0=p["s0"])
    dx2, _, _, ds02 = gdr.conv_bwd(tail(x), p["weight"], tail(dy), bias=p["bias"], s0=p["s0"], dst=p["dst"])
    assert torch.equal(tail(y), y2) and torch.equal(st[1:], st2)
    assert torch.equal(tail(dx), dx2) and torch.equal(ds0[1:], ds02)


def test_scan_of_the_last_sequence(gdr, wide):
    S = 16
    p = ref.scan_inputs([TAIL], E, S, 1, BF16, device="cuda")
    cu = torch.tensor([0, M - TAIL, M], dtype=torch.int64, device="cuda")
    x, dt = wide[..., :E], wide[..., E:]
    bc = wide[..., 64:64 + 2 * S]
    b, c = (bc[..., i:i + S].unflatten(-1, (1, S)) for i in (0, S))
    h0, dht = torch.cat([p["h0"], p["h0"]]), torch.cat([p["dht"], p["dht"]])
    kw = dict(d=p["d"], dt_bias=p["dt_bias"])
    tail = lambda t: t[:, M - TAIL:].contiguous()  # noqa: E731
    y, ht = gdr.ssm_fwd(x, dt, p["a"], b, c, z=x, h0=h0, cu_seqlens=cu, **kw)
    small = [tail(t) for t in (x, dt, b, c)]
    y2, ht2 = gdr.ssm_fwd(small[0], small[1], p["a"], small[2], small[3], z=small[0], h0=p["h0"], **kw)
    # the chunks fall elsewhere: two results, each within the bound of the exact one
    assert ref.rel(tail(y), y2) <= 2 * ref.tol(BF16, TAIL) and ref.rel(ht[1:], ht2) <= 2 * ref.tol(torch.float32, TAIL)
    del y
    got = gdr.ssm_bwd(x, dt, p["a"], b, c, dt, z=x, h0=h0, dht=dht, cu_seqlens=cu, **kw)
    want = gdr.ssm_bwd(small[0], small[1], p["a"], small[2], small[3], small[1], z=small[0], h0=p["h0"], dht=p["dht"], **kw)
    for i in (0, 1, 3, 4, 6):
        assert ref.rel(tail(got[i]), want[i]) <= 2 * ref.tol(BF16, TAIL)
    assert ref.rel(got[8][1:], want[8]) <= 2 * ref.tol(torch.float32, TAIL)
    assert gdr.device_status() == 0


def test_slots_of_a_large_pool(gdr):
    """States of a pool of more than 2^31 elements."""
    S, P = 16, 2 ** 31 // (2048 * 16) + 100
    p = ref.scan_inputs([1, 1, 1], 2048, S, 1, BF16, device="cuda")
    pool = torch.empty(P, 2048, S, device="cuda")
    slots = torch.tensor([P - 1, 3, P - 50], dtype=torch.int32, device="cuda")
    pool[slots.long()] = p["h0"]
    state = p["h0"].clone()
    args = (p["x"], p["dt"], p["a"], p["b"], p["c"])
    y = gdr.ssm_step(*args, pool, z=p["z"], slots=slots)
    y2 = gdr.ssm_step(*args, state, z=p["z"])
    assert torch.equal(y, y2) and torch.equal(pool[slots.long()], state)
    q = ref.conv_inputs([1, 1, 1], 2048, 4, BF16, device="cuda")
    n = 2 ** 31 // (3 * 2048) + 100
    pool = torch.empty(n, 3, 2048, dtype=BF16, device="cuda")
    slots = torch.tensor([n - 1, 3, n - 50], dtype=torch.int32, device="cuda")
    pool[slots.long()] = q["s0"]
    state = q["s0"].clone()
    assert torch.equal(gdr.conv_step(q["x"], pool, q["weight"], slots=slots), gdr.conv_step(q["x"], state, q["weight"]))
    assert torch.equal(pool[slots.long()], state)
