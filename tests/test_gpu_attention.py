"""Linear attention with a decay for each head on the GPU: forward, backward and
single tokens against the 64-bit definition."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import cu_of, spans

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
both_types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])


def put(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def run(gdr, q, lens, scale, dense=False, **kw):
    """All outputs of the forward and the backward, tokens flat."""
    lead = (lambda t: t.view(len(lens), -1, *t.shape[1:])) if dense else (lambda t: t[None])
    cu = None if dense else cu_of(lens, "cuda")
    args = (lead(q["q"]), lead(q["k"]), lead(q["v"]), q["g"])
    o, ht = gdr.la_fwd(*args, h0=q["h0"], cu_seqlens=cu, scale=scale, **kw)
    dq, dk, dv, dh0 = gdr.la_bwd(*args, lead(q["do"]), h0=q["h0"], dht=q["dht"], cu_seqlens=cu, scale=scale, **kw)
    assert gdr.device_status() == 0, gdr.last_error()
    return dict(o=o.flatten(0, 1), ht=ht, dq=dq.flatten(0, 1), dk=dk.flatten(0, 1), dv=dv.flatten(0, 1), dh0=dh0)


def wanted(p, lens, scale):
    d = {k: v.double() for k, v in p.items()}
    args = [d[k] for k in ("q", "k", "v", "g", "h0")]
    want = dict(zip(("o", "ht"), ref.attention(*args, lens, scale)))
    want.update(zip(("dq", "dk", "dv", "dh0"), ref.attention_grads(*args, lens, scale, d["do"], d["dht"])))
    return want


def check(got, want, dtype, lens, what=""):
    for k, w in want.items():
        ref.close(got[k], w, dtype, max(lens), f"{what} {k}")


LENS = [[1], [2, 63], [64], [65], [128, 1, 0, 127], [30, 0, 0, 200, 3]]


@both_types
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,HV,K,V", [(1, 1, 128, 128), (2, 4, 64, 128), (1, 3, 128, 64), (2, 2, 60, 100), (1, 1, 7, 5),
                                      (1, 2, 256, 40), (2, 2, 96, 200)], ids=str)
def test_packed(gdr, dtype, lens, H, HV, K, V):
    p = ref.attention_inputs(lens, H, HV, K, V, dtype, seed=K + V)
    check(run(gdr, put(p), lens, K ** -0.5), wanted(p, lens, K ** -0.5), dtype, lens)


@both_types
@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (2, 64), (3, 100), (1, 700)])
@pytest.mark.parametrize("H,HV,K,V", [(2, 2, 128, 128), (1, 2, 32, 48)], ids=str)
def test_dense(gdr, dtype, B, T, H, HV, K, V):
    lens = [T] * B
    p = ref.attention_inputs(lens, H, HV, K, V, dtype, seed=T)
    check(run(gdr, put(p), lens, 1.0, dense=True), wanted(p, lens, 1.0), dtype, lens)


@both_types
@pytest.mark.parametrize("K,V", [(128, 128), (36, 20)], ids=str)
@pytest.mark.parametrize("lens", [[2500], [700, 1, 0, 1300, 256, 90], [200] * 8], ids=["one", "cut", "not_worth_it"])
def test_sequences_cut_into_segments(gdr, dtype, K, V, lens):
    """Few heads: states of segments first, then carried, then the passes from there."""
    p = ref.attention_inputs(lens, 1, 1, K, V, dtype, seed=3)
    q = put(p)
    before = gdr.launch_count()
    gdr.la_fwd(q["q"][None], q["k"][None], q["v"][None], q["g"], h0=q["h0"], cu_seqlens=cu_of(lens, "cuda"))
    assert gdr.launch_count() - before == 3
    check(run(gdr, q, lens, K ** -0.5), wanted(p, lens, K ** -0.5), dtype, lens)


@both_types
def test_many_short_sequences_and_a_long_one(gdr, dtype):
    """5000 sequences of a token or none beside one that is worth cutting; few heads, no initial states."""
    lens = [1, 0] * 1250 + [3000] + [1, 0] * 1250
    p = put(ref.attention_inputs(lens, 1, 2, 16, 16, dtype, seed=11))
    cu = cu_of(lens, "cuda")
    args = (p["q"][None], p["k"][None], p["v"][None], p["g"])
    o, ht = gdr.la_fwd(*args, h0=p["h0"], cu_seqlens=cu, scale=0.25)
    d = {k: v.double() for k, v in p.items()}
    want, s = ref.attention(*[d[k] for k in ("q", "k", "v", "g", "h0")], lens, 0.25)
    ref.close(o[0], want, dtype, 3000, "o")
    ref.close(ht, s, dtype, 3000, "ht")
    got = gdr.la_bwd(*args, p["do"][None], h0=p["h0"], dht=p["dht"], cu_seqlens=cu, scale=0.25)
    # the long sequence by itself, and the first of the short ones
    for n, i, j in ((2500, 1250, 4250), (0, 0, 1)):
        part = [p[k][None, i:j] for k in ("q", "k", "v")] + [p["g"], p["do"][None, i:j]]
        alone = gdr.la_bwd(*part, h0=p["h0"][n:n + 1], dht=p["dht"][n:n + 1], scale=0.25)
        for k, a, b in zip(("dq", "dk", "dv", "dh0"), got, alone):
            ref.close(a[n:n + 1] if k == "dh0" else a[:, i:j], b.double(), dtype, 3000, k)
    assert gdr.device_status() == 0


@pytest.mark.parametrize("B,T,HV", [(1, 8192, 100), (1, 6400, 160), (2, 4096, 40), (1, 5000, 3)], ids=str)
def test_how_sequences_are_cut_does_not_matter(gdr, B, T, HV):
    """Heads and lengths on both sides of where sequences are cut: the same values as head by head."""
    p = put(ref.attention_inputs([T] * B, HV, HV, 16, 16, BF16, seed=12))
    lead = lambda t: t.view(B, T, *t.shape[1:])  # noqa: E731
    o, ht = gdr.la_fwd(lead(p["q"]), lead(p["k"]), lead(p["v"]), p["g"], h0=p["h0"])
    packed = gdr.la_fwd(p["q"][None], p["k"][None], p["v"][None], p["g"], h0=p["h0"], cu_seqlens=cu_of([T] * B, "cuda"))
    for a, b in zip((o.flatten(0, 1)[None], ht), packed):
        ref.close(a, b.double(), BF16, T)
    for h in (0, HV - 1):
        one = slice(h, h + 1)
        a, s = gdr.la_fwd(lead(p["q"])[:, :, one], lead(p["k"])[:, :, one], lead(p["v"])[:, :, one],
                          p["g"][one].clone(), h0=p["h0"][:, one].contiguous())
        ref.close(o[:, :, one], a.double(), BF16, T, "o")
        ref.close(ht[:, one], s.double(), BF16, T, "ht")
    assert gdr.device_status() == 0


@both_types
@pytest.mark.parametrize("g", [0.0, -1e-5, -0.3, -5.0, -200.0, -math.inf, 0.01], ids=str)
@pytest.mark.parametrize("K", [128, 24])
def test_decays(gdr, dtype, g, K):
    lens = [150, 5]
    p = ref.attention_inputs(lens, 2, 2, K, K, dtype, seed=1, g=torch.tensor([g, -0.1]))
    check(run(gdr, put(p), lens, 0.3), wanted(p, lens, 0.3), dtype, lens)


def test_slow_decays_over_many_chunks(gdr):
    """exp(64 g) near 1, 256 times over: decays are not rounded away."""
    lens, g = [16384], torch.tensor([-1e-5, -1e-4])
    p = ref.attention_inputs(lens, 2, 2, 16, 16, F32, seed=1, g=g)
    o, ht = gdr.la_fwd(*[p[k].cuda()[None] for k in ("q", "k", "v")], g.cuda(), h0=p["h0"].cuda())
    t = torch.arange(16384, dtype=torch.float64)
    for h in range(2):
        w = torch.exp((16383 - t) * p["g"][h].double())
        want = (p["k"][:, h].double() * w[:, None]).t() @ p["v"][:, h].double()
        want = want + torch.exp(16384 * p["g"][h].double()) * p["h0"][0, h].double()
        ref.close(ht[0, h], want, F32, 16384, f"ht {h}")


@both_types
def test_without_states(gdr, dtype):
    lens = [100]
    p = ref.attention_inputs(lens, 1, 2, 64, 64, dtype, seed=8)
    p["h0"].zero_()
    p["dht"].zero_()
    want, q = wanted(p, lens, 1.0), put(p)
    args = (q["q"][None], q["k"][None], q["v"][None], q["g"])
    o, ht = gdr.la_fwd(*args, output_final_state=False)
    assert ht is None
    dq, dk, dv, dh0 = gdr.la_bwd(*args, q["do"][None])
    del want["ht"]
    check(dict(o=o[0], dq=dq[0], dk=dk[0], dv=dv[0], dh0=dh0), want, dtype, lens)


@both_types
def test_nothing_to_do(gdr, dtype):
    z = lambda *s: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    g, h0 = torch.zeros(2, device="cuda"), torch.randn(3, 2, 8, 4, device="cuda")
    cu = torch.zeros(4, dtype=torch.int64, device="cuda")
    o, ht = gdr.la_fwd(z(1, 0, 2, 8), z(1, 0, 2, 8), z(1, 0, 2, 4), g, h0=h0, cu_seqlens=cu)
    assert o.shape == (1, 0, 2, 4) and torch.equal(ht, h0)
    got = gdr.la_bwd(z(1, 0, 2, 8), z(1, 0, 2, 8), z(1, 0, 2, 4), g, z(1, 0, 2, 4), h0=h0, dht=h0, cu_seqlens=cu)
    assert torch.equal(got[3], h0)
    o, ht = gdr.la_fwd(z(3, 0, 2, 8), z(3, 0, 2, 8), z(3, 0, 2, 4), g)
    assert (ht == 0).all()
    o, ht = gdr.la_fwd(z(0, 5, 2, 8), z(0, 5, 2, 8), z(0, 5, 2, 4), g)
    assert o.numel() == 0 and ht.shape[0] == 0
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    gdr.la_fwd(z(1, 0, 2, 8), z(1, 0, 2, 8), z(1, 0, 2, 4), g, cu_seqlens=none)
    assert gdr.device_status() == 0
    gdr.la_fwd(z(1, 5, 2, 8), z(1, 5, 2, 8), z(1, 5, 2, 4), g, cu_seqlens=none)
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS


@both_types
@pytest.mark.parametrize("bad", [[0, 30, 20, 90], [1, 40, 90], [0, 40, 91], [0, 40, 89], [0, 300, 200, 1000]], ids=str)
@pytest.mark.parametrize("D", [64, 20])
def test_bad_cu_seqlens_touch_nothing(gdr, dtype, bad, D):
    import ctypes
    from chunked_gated_delta_08_gb300 import attention_ops as ops
    T = 1000 if bad[-1] == 1000 else 90
    N, H, HV = len(bad) - 1, 1, 2
    q = put(ref.attention_inputs([T], H, HV, D, D, dtype))
    cu = torch.tensor(bad, device="cuda")
    desc = ops.GdrLaDesc(1, T, H, HV, D, D, N, H * D, H * D, HV * D, HV * D, 1.0, 0 if dtype == F32 else 1, 0)
    full = lambda dt, *s: torch.full(s, 7.0, dtype=dt, device="cuda")  # noqa: E731
    a, s = (lambda t: t.data_ptr()), torch.cuda.current_stream().cuda_stream  # noqa: E731
    o, ht, dh0 = full(dtype, T, HV, D), full(F32, N, HV, D, D), full(F32, N, HV, D, D)
    dq, dk, dv = full(dtype, T, H, D), full(dtype, T, H, D), full(dtype, T, HV, D)
    head = [a(q["q"]), a(q["k"]), a(q["v"]), a(q["g"]), None, a(cu)]
    assert gdr.lib().gdr_la_fwd(ctypes.byref(desc), *head, a(o), a(ht), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert gdr.lib().gdr_la_bwd(ctypes.byref(desc), *head, a(q["do"]), None, a(dq), a(dk), a(dv), a(dh0), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert all(t.eq(7.0).all() for t in (o, ht, dq, dk, dv, dh0))


@both_types
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("D", [64, 24])
def test_slices_and_unaligned_bases(gdr, dtype, offset, D):
    """q, k, v and do as parts of wider rows."""
    lens, H, HV = [150, 40], 1, 2
    p = ref.attention_inputs(lens, H, HV, D, D, dtype, seed=2)
    q = put(p)
    wide = torch.zeros(190, (2 * H + 2 * HV) * D + 8 + offset, dtype=dtype, device="cuda")
    at = offset
    for k in ("q", "k", "v", "do"):
        n = p[k][0].numel()
        wide[:, at:at + n] = q[k].flatten(1)
        q[k] = wide[:, at:at + n].unflatten(1, p[k].shape[1:])
        at += n
    assert not q["q"].is_contiguous()
    check(run(gdr, q, lens, 0.1), wanted(p, lens, 0.1), dtype, lens)


@both_types
@pytest.mark.parametrize("where", ["q", "k", "v", "do", "h0", "dht"])
@pytest.mark.parametrize("D", [128, 20])
@pytest.mark.parametrize("value", [math.nan, math.inf], ids=str)
def test_sequences_keep_to_themselves(gdr, dtype, where, D, value):
    """What is not a number in one sequence leaves the others' results as they are, to the bit."""
    lens = [100, 30, 300, 90]
    q = put(ref.attention_inputs(lens, 1, 1, D, D, dtype, seed=6))
    clean = run(gdr, q, lens, 1.0)
    for seq in (1, 2):
        r = dict(q)
        r[where] = q[where].clone()
        i = sum(lens[:seq])
        r[where][seq if where in ("h0", "dht") else slice(i, i + lens[seq])] = value
        got = run(gdr, r, lens, 1.0)
        for n, i, j in spans(lens):
            for k, v in got.items():
                mine, want = (u[n] if k in ("ht", "dh0") else u[i:j] for u in (v, clean[k]))
                assert n == seq or torch.equal(mine, want), (k, n)


@both_types
@pytest.mark.parametrize("D", [128, 20])
def test_earlier_chunks_and_heads_do_not_see_what_is_not_a_number(gdr, dtype, D):
    lens = [200]
    q = put(ref.attention_inputs(lens, 2, 2, D, D, dtype, seed=6))
    args = lambda r: [r[k][None] for k in ("q", "k", "v")] + [r["g"]]  # noqa: E731
    clean, _ = gdr.la_fwd(*args(q))
    for where in ("q", "k", "v"):
        r = dict(q)
        r[where] = q[where].clone()
        r[where][130, 0] = math.nan
        got, _ = gdr.la_fwd(*args(r))
        assert torch.equal(got[0, :128], clean[0, :128]) and torch.equal(got[0, :, 1], clean[0, :, 1])
        assert got[0, 130, 0].isnan().all()
        if where == "q":
            assert torch.equal(got[0, 131:], clean[0, 131:])


@both_types
@pytest.mark.parametrize("D", [64, 20])
def test_a_decay_that_is_not_a_number_spoils_its_head_alone(gdr, dtype, D):
    lens = [1500, 70]
    q = put(ref.attention_inputs(lens, 3, 3, D, D, dtype, seed=6))
    clean = run(gdr, q, lens, 1.0)
    got = run(gdr, dict(q, g=torch.stack([q["g"][0], q["g"][1] * math.nan, q["g"][2]])), lens, 1.0)
    for k, v in got.items():
        assert torch.equal(v[:, [0, 2]], clean[k][:, [0, 2]]) and v[:, 1].isnan().any(), k


@both_types
def test_cut_sequences_without_states(gdr, dtype):
    lens = [2600]
    p = ref.attention_inputs(lens, 1, 2, 32, 32, dtype, seed=13)
    p["h0"].zero_()
    p["dht"].zero_()
    want, q = wanted(p, lens, 0.2), put(p)
    args = (q["q"][None], q["k"][None], q["v"][None], q["g"])
    before = gdr.launch_count()
    o, _ = gdr.la_fwd(*args, scale=0.2, output_final_state=False)
    assert gdr.launch_count() - before == 3
    dq, dk, dv, dh0 = gdr.la_bwd(*args, q["do"][None], scale=0.2)
    del want["ht"]
    check(dict(o=o[0], dq=dq[0], dk=dk[0], dv=dv[0], dh0=dh0), want, dtype, lens)


@both_types
def test_results_repeat_bit_for_bit(gdr, dtype):
    lens = [1000, 77, 400]
    q = put(ref.attention_inputs(lens, 2, 4, 128, 128, dtype, seed=4))
    a, b = run(gdr, q, lens, 1.0), run(gdr, q, lens, 1.0)
    assert all(torch.equal(a[k], b[k]) for k in a)


@both_types
def test_other_streams_and_graphs(gdr, dtype):
    """A call on its own stream, and one captured and replayed on other inputs."""
    lens = [500, 20]
    p = ref.attention_inputs(lens, 1, 2, 64, 64, dtype, seed=5)
    q, want = put(p), wanted(p, lens, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(gdr, q, lens, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(got, want, dtype, lens)
    cu = cu_of(lens, "cuda")
    fixed = {k: torch.zeros_like(v) for k, v in q.items()}
    args = (fixed["q"][None], fixed["k"][None], fixed["v"][None], fixed["g"])
    kw = dict(h0=fixed["h0"], cu_seqlens=cu)
    gdr.la_bwd(*args, fixed["do"][None], dht=fixed["dht"], **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, ht = gdr.la_fwd(*args, **kw)
        dq, dk, dv, dh0 = gdr.la_bwd(*args, fixed["do"][None], dht=fixed["dht"], **kw)
    for k, v in q.items():
        fixed[k].copy_(v)
    graph.replay()
    check(dict(o=o[0], ht=ht, dq=dq[0], dk=dk[0], dv=dv[0], dh0=dh0), want, dtype, lens)


# ------------------------------------------------------------------------------------ single tokens
@both_types
@pytest.mark.parametrize("R,H,HV,K,V", [(1, 1, 1, 128, 128), (5, 2, 4, 60, 100), (3, 1, 1, 256, 256), (4, 1, 2, 7, 5),
                                        (2, 1, 1, 1, 1), (7, 3, 3, 130, 33), (300, 1, 1, 8, 8)], ids=str)
def test_steps(gdr, dtype, R, H, HV, K, V):
    """Three tokens for rows whose states lie scattered over a pool; a padding row; slots of no row stay."""
    gen = torch.Generator().manual_seed(R)
    P = R + 3
    slots = torch.randperm(P, generator=gen)[:R].int()
    if R > 1:
        slots[R // 2] = -1
    p = ref.attention_inputs([R] * 3, H, HV, K, V, dtype, seed=K)
    state = torch.randn(P, HV, K, V, generator=gen)
    s64, pool = state.double(), state.cuda()
    real = slots >= 0
    at = slots[real].long()
    for t in range(3):
        q, k, v = (p[n][t * R:(t + 1) * R] for n in ("q", "k", "v"))
        o = gdr.la_step(q.cuda(), k.cuda(), v.cuda(), p["g"].cuda(), pool, slots=slots.cuda(), scale=0.5)
        want, s = ref.attention(*(x.double()[real] for x in (q, k, v)), p["g"].double(), s64[at], [1] * int(real.sum()),
                                0.5)
        s64[at] = s
        ref.close(o.cpu()[real], want, dtype, 3, "o")
        assert (o.cpu()[~real] == 0).all()
    ref.close(pool, s64, F32, 3, "state")
    others = torch.ones(P, dtype=torch.bool)
    others[at] = False
    assert torch.equal(pool.cpu()[others], state[others])
    assert gdr.device_status() == 0


def test_steps_go_on_from_a_prompt(gdr):
    lens = [130, 64, 1]
    p = put(ref.attention_inputs(lens, 2, 2, 64, 64, BF16, seed=9))
    more = put(ref.attention_inputs([1] * 3, 2, 2, 64, 64, BF16, seed=10))
    _, state = gdr.la_fwd(*[p[k][None] for k in ("q", "k", "v")], p["g"], cu_seqlens=cu_of(lens, "cuda"), scale=0.125)
    o = gdr.la_step(more["q"], more["k"], more["v"], p["g"], state, scale=0.125)
    for n, i, j in spans(lens):
        whole = [torch.cat([p[k][i:j], more[k][n:n + 1]]).double().cpu() for k in ("q", "k", "v")]
        want, s = ref.attention(*whole, p["g"].double().cpu(), torch.zeros(1, 2, 64, 64, dtype=torch.float64),
                                [j - i + 1], 0.125)
        ref.close(o[n], want[-1], BF16, 130)
        ref.close(state[n], s[0], BF16, 130)


def test_steps_with_bad_slots(gdr):
    p = put(ref.attention_inputs([4], 1, 2, 16, 16, F32))
    state = torch.randn(3, 2, 16, 16, device="cuda")
    kept = state.clone()
    slots = torch.tensor([0, 3, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda")
    o = gdr.la_step(p["q"], p["k"], p["v"], p["g"], state, slots=slots)
    assert gdr.device_status() == gdr.GDR_ERR_SLOTS
    assert (o[1:] == 0).all() and (o[0] != 0).any() and torch.equal(state[1:], kept[1:])


def test_shapes_and_types_are_checked(gdr):
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, v, g = z(1, 4, 2, 16), z(1, 4, 4, 8), z(4, dt=F32)
    bad = [(ValueError, lambda: gdr.la_fwd(q, q[:, :3], v, g)), (ValueError, lambda: gdr.la_fwd(q, q, v[:, :3], g)),
           (gdr.GdrError, lambda: gdr.la_fwd(q, q.float(), v, g)), (gdr.GdrError, lambda: gdr.la_fwd(q, q, v.float(), g)),
           (ValueError, lambda: gdr.la_fwd(q, q, v, g[:3])), (gdr.GdrError, lambda: gdr.la_fwd(q, q, v, g.bfloat16())),
           (ValueError, lambda: gdr.la_fwd(q, q, z(1, 4, 3, 8), z(3, dt=F32))),
           (ValueError, lambda: gdr.la_fwd(q, q, v, g, h0=z(1, 4, 8, 16, dt=F32))),
           (gdr.GdrError, lambda: gdr.la_fwd(q.half(), q.half(), v.half(), g)),
           (ValueError, lambda: gdr.la_bwd(q, q, v, g, v[..., :7])),
           (gdr.GdrError, lambda: gdr.la_fwd(q, q, v, g, cu_seqlens=z(2, dt=torch.int32))),
           (ValueError, lambda: gdr.la_step(q[0], q[0], v[0], g, z(3, 4, 16, 8, dt=F32))),
           (ValueError, lambda: gdr.la_step(q[0], q[0], v[0], g, z(4, 4, 8, 16, dt=F32))),
           (gdr.GdrError, lambda: gdr.la_step(q[0], q[0], v[0], g, z(4, 4, 16, 8))),
           (ValueError, lambda: gdr.la_fwd(z(1, 4, 2, 300), z(1, 4, 2, 300), v, g)),
           (gdr.GdrError, lambda: gdr.la_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, v, g))]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
    assert gdr.device_status() == 0
