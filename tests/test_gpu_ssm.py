"""The selective state space scan, forward, backward and one token at a time,
on the GPU against the 64-bit recurrence."""
import ctypes

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")
OUT = ("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh0")
# around tiles of 16 and runs of 8 tokens; sequences that start and end inside them, empty ones anywhere
LENGTHS = [[1], [7], [8], [16], [17], [65], [0, 5, 0, 0, 1, 20, 0], [1] * 19, [15, 1, 16, 33], [0, 0], [40, 40]]
# (E, S, G): states of one, two and four lanes' worth, odd widths, groups that end inside a block
SIZES = [(64, 16, 1), (1, 1, 1), (6, 3, 2), (136, 4, 1), (130, 16, 2), (200, 12, 1), (48, 17, 3), (96, 32, 1), (40, 33, 2),
         (72, 64, 1)]


def put(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def forward(gdr, q, cu, **kw):
    lead = lambda t: None if t is None else t[None]  # noqa: E731
    return gdr.ssm_fwd(lead(q["x"]), lead(q["dt"]), q["a"], lead(q["b"]), lead(q["c"]), d=q["d"], z=lead(q["z"]),
                       dt_bias=q["dt_bias"], h0=q["h0"], cu_seqlens=cu, **kw)


def backward(gdr, q, cu, **kw):
    lead = lambda t: None if t is None else t[None]  # noqa: E731
    return gdr.ssm_bwd(lead(q["x"]), lead(q["dt"]), q["a"], lead(q["b"]), lead(q["c"]), lead(q["dy"]), d=q["d"],
                       z=lead(q["z"]), dt_bias=q["dt_bias"], h0=q["h0"], dht=q["dht"], cu_seqlens=cu, **kw)


def check(gdr, p, q, lens, softplus=True, cu="packed", exact_on="cpu"):
    cu = ref.cu_of(lens, "cuda") if cu == "packed" else None
    T, M = max([1] + list(lens)), max(1, sum(lens))
    fn = lambda *v: ref.scan(*v, lens, softplus)  # noqa: E731
    src = p if exact_on == "cpu" else q
    y, ht = forward(gdr, q, cu, dt_softplus=softplus)
    want_y, want_ht = fn(*[ref.f64(src[k]) for k in NAMES])
    ref.close(y[0], want_y, T, "y")
    ref.close(ht, want_ht, T, "ht")
    got = dict(zip(OUT, backward(gdr, q, cu, dt_softplus=softplus)))
    want = dict(zip(("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh0"),
                    ref.grads(fn, [src[k] for k in NAMES], (src["dy"].double(), src["dht"].double()))))
    for k in OUT:
        assert (got[k] is None) == (src[{"dx": "x", "ddt": "dt", "dd": "d", "dz": "z", "ddt_bias": "dt_bias"}.get(
            k, "x")] is None), k
        if got[k] is not None and want[k] is not None:
            packed = k in ("dx", "ddt", "db", "dc", "dz")
            ref.close(got[k][0] if packed else got[k], want[k], T if packed or k == "dh0" else M, k)
    assert gdr.device_status() == 0


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "_".join(map(str, v))[:24])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_packed(gdr, lens, dtype):
    for E, S, G in SIZES[:3] if sum(lens) > 40 else SIZES:
        p = ref.scan_inputs(lens, E, S, G, dtype, seed=E + S)
        check(gdr, p, put(p), lens)


@pytest.mark.parametrize("missing", ["d", "z", "dt_bias", "all"])
@pytest.mark.parametrize("softplus", [True, False])
def test_optional_terms(gdr, missing, softplus):
    have = {k: missing not in (k, "all") for k in ("d", "z", "dt_bias")}
    p = ref.scan_inputs([30, 3], 24, 16, 1, F32, seed=3, **have)
    if not softplus:  # delta is dt (and bias) itself: small and positive
        p["dt"] = p["dt"].abs() * 0.1
        if p["dt_bias"] is not None:
            p["dt_bias"] = p["dt_bias"].abs() * 0.01
    check(gdr, p, put(p), [30, 3], softplus=softplus)


@pytest.mark.parametrize("size", SIZES, ids=lambda v: "E%d_S%d_G%d" % v)
def test_every_width_over_several_chunks(gdr, size):
    E, S, G = size
    p = ref.scan_inputs([50, 90], E, S, G, BF16, seed=S)
    check(gdr, p, put(p), [50, 90])


def test_dense_batch_without_initial_states(gdr):
    for B, T in ((3, 40), (2, 1), (1, 100), (4, 0), (0, 8)):
        lens, E, S = [T] * B, 32, 16
        p = ref.scan_inputs(lens, E, S, 1, BF16, seed=T)
        q = put(p)
        lead = lambda t, *s: t.view(B, T, *s)  # noqa: E731
        args = (lead(q["x"], E), lead(q["dt"], E), q["a"], lead(q["b"], 1, S), lead(q["c"], 1, S))
        kw = dict(d=q["d"], z=lead(q["z"], E), dt_bias=q["dt_bias"])
        y, ht = gdr.ssm_fwd(*args, **kw)
        assert y.shape == (B, T, E) and ht.shape == (B, E, S)
        got = dict(zip(OUT, gdr.ssm_bwd(*args, lead(q["dy"], E), **kw)))
        if B * T == 0:
            assert ht.eq(0).all() and got["da"].eq(0).all() and got["dh0"].eq(0).all() and got["ddt_bias"].eq(0).all()
            continue
        none = torch.zeros(B, E, S, dtype=torch.float64)
        fn = lambda *v: ref.scan(*v, none, lens)  # noqa: E731
        want_y, want_ht = fn(*[ref.f64(p[k]) for k in NAMES[:-1]])
        ref.close(y.flatten(0, 1), want_y, T, "y")
        ref.close(ht, want_ht, T, "ht")
        want = ref.grads(lambda *v: fn(*v)[:1], [p[k] for k in NAMES[:-1]], (p["dy"].double(),))
        for k, w in zip(OUT, want):
            ref.close(got[k].flatten(0, 1) if k in ("dx", "ddt", "db", "dc", "dz") else got[k], w, B * T, k)
        y2, none_t = gdr.ssm_fwd(*args, **kw, output_final_state=False)
        assert none_t is None and torch.equal(y, y2)


def test_one_long_sequence(gdr):
    """Chunks of many tiles, carried over a long axis."""
    lens = [20000]
    p = put(ref.scan_inputs(lens, 128, 16, 1, BF16, seed=6))
    y, ht = forward(gdr, p, None)
    want_y, want_ht = ref.scan(*[ref.f64(p[k]) for k in NAMES], lens)
    ref.close(y[0], want_y, 1000, "y")  # a state remembers at most some thousand tokens (delta a >= 5e-4)
    ref.close(ht, want_ht, 1000, "ht")
    again = forward(gdr, p, None)
    assert torch.equal(y, again[0]) and torch.equal(ht, again[1])


def test_wide_backward_over_whole_chunks(gdr):
    """Enough blocks that chunks have their full 64 tokens; the same bits each time."""
    lens = [1500, 1, 0, 700, 300]
    p = put(ref.scan_inputs(lens, 1024, 16, 2, BF16, seed=7))
    check(gdr, p, p, lens, exact_on="gpu")
    cu = ref.cu_of(lens, "cuda")
    a, b = backward(gdr, p, cu), backward(gdr, p, cu)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_slices_and_unaligned_bases(gdr, offset, dtype):
    """x, dt, z, b and c as parts of wider rows: the contiguous call's results."""
    lens, E, S = [30, 21], 64, 16
    p = put(ref.scan_inputs(lens, E, S, 1, dtype, seed=3))
    cu = ref.cu_of(lens, "cuda")
    wide = torch.zeros(51, 3 * E + 2 * S + 8 + offset, dtype=dtype, device="cuda")
    at, q = offset, dict(p)
    for k, n in (("x", E), ("dt", E), ("z", E), ("b", S), ("c", S)):
        wide[:, at:at + n] = p[k].flatten(1)
        q[k] = wide[:, at:at + n].unflatten(1, p[k].shape[1:])
        at += n
    for u, v in zip(forward(gdr, q, cu), forward(gdr, p, cu)):
        assert torch.equal(u, v)
    for u, v in zip(backward(gdr, q, cu), backward(gdr, p, cu)):
        assert torch.equal(u, v)


def test_unaligned_states(gdr):
    """States, a and final states one element past a 16-byte border."""
    lens = [20, 13]
    p = put(ref.scan_inputs(lens, 24, 16, 1, F32, seed=4))
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    q = dict(p, a=off(p["a"]), h0=off(p["h0"]), dht=off(p["dht"]))
    cu = ref.cu_of(lens, "cuda")
    assert q["h0"].data_ptr() % 16
    for u, v in zip(forward(gdr, q, cu) + backward(gdr, q, cu), forward(gdr, p, cu) + backward(gdr, p, cu)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("size", SIZES, ids=lambda v: "E%d_S%d_G%d" % v)
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_steps_follow_the_recurrence(gdr, size, dtype):
    """Five rows, five tokens each, one by one through a pool of slots with a padding row."""
    E, S, G = size
    R, T = 5, 5
    p = ref.scan_inputs([T] * R, E, S, G, dtype, seed=9)
    q = put(p)
    want_y, want_ht = ref.scan(*[ref.f64(p[k]) for k in NAMES], [T] * R)
    pool = torch.full((9, E, S), 9.0, device="cuda")
    slots = torch.tensor([8, 0, -1, 3, 5, 1], dtype=torch.int32, device="cuda")
    real = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    pool[slots[real].long()] = q["h0"]
    row = lambda k, t: torch.cat([v := q[k].view(R, T, *q[k].shape[1:])[:, t], v[:1]])[[0, 1, 5, 2, 3, 4]]  # noqa: E731
    ys = []
    for t in range(T):
        y = gdr.ssm_step(row("x", t), row("dt", t), q["a"], row("b", t), row("c", t), pool, d=q["d"], z=row("z", t),
                         dt_bias=q["dt_bias"], slots=slots)
        assert y[2].eq(0).all()
        ys.append(y[real])
    ref.close(torch.stack(ys, 1).flatten(0, 1), want_y, T, "y")
    ref.close(pool[slots[real].long()], want_ht, T, "states")
    assert pool[[2, 4, 6, 7]].eq(9.0).all() and gdr.device_status() == 0


def test_step_without_slots_or_options(gdr):
    p = ref.scan_inputs([1, 1, 1], 20, 16, 1, F32, d=False, z=False, dt_bias=False)
    q = put(p)
    state = q["h0"].clone()
    y = gdr.ssm_step(q["x"], q["dt"], q["a"], q["b"], q["c"], state)
    want_y, want_ht = ref.scan(*[ref.f64(p[k]) for k in NAMES], [1, 1, 1])
    ref.close(y, want_y, 1, "y")
    ref.close(state, want_ht, 1, "state")
    assert gdr.ssm_step(q["x"][:0], q["dt"][:0], q["a"], q["b"][:0], q["c"][:0], state).shape == (0, 20)


def test_slots_past_the_pool_are_reported(gdr):
    p = put(ref.scan_inputs([1] * 3, 32, 16, 1, F32))
    pool = torch.ones(2, 32, 16, device="cuda")
    y = gdr.ssm_step(p["x"], p["dt"], p["a"], p["b"], p["c"], pool,
                     slots=torch.tensor([2, 0, 2 ** 30], dtype=torch.int32, device="cuda"))
    assert gdr.device_status() == gdr.GDR_ERR_SLOTS and gdr.device_status() == 0
    assert y[[0, 2]].eq(0).all() and not y[1].eq(0).all() and pool[1].eq(1).all()


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [1, 4, 8], [0, 4, 9], [0, 4, 7]])
def test_bad_cu_seqlens_touch_nothing(gdr, cu):
    from chunked_gated_delta_08_gb300 import layer_ops as ops
    N, E, S = len(cu) - 1, 16, 8
    p = put(ref.scan_inputs([8], E, S, 1, F32))
    cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
    shapes = dict(y=(8, E), dx=(8, E), ddt=(8, E), dz=(8, E), db=(8, S), dc=(8, S), da=(E, S), dd=(E,), dbias=(E,),
                  ht=(N, E, S), dh0=(N, E, S))
    o = {k: torch.full(s, 7.0, device="cuda") for k, s in shapes.items()}
    desc = ops.GdrSsmDesc(1, 8, E, S, 1, N, E, E, E, S, S, E, 0, 1)
    a = lambda t: t.data_ptr()  # noqa: E731
    head = [a(p[k]) for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias")] + [None, a(cu)]
    s = torch.cuda.current_stream().cuda_stream
    assert gdr.lib().gdr_ssm_fwd(ctypes.byref(desc), *head, a(o["y"]), a(o["ht"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert gdr.lib().gdr_ssm_bwd(ctypes.byref(desc), *head, a(p["dy"]), None, a(o["dx"]), a(o["ddt"]), a(o["da"]),
                                 a(o["db"]), a(o["dc"]), a(o["dd"]), a(o["dz"]), a(o["dbias"]), a(o["dh0"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert all(t.eq(7.0).all() for t in o.values())


def test_extreme_deltas(gdr):
    """Large, tiny and negative dt: the state forgotten at once, kept for ever, and softplus's ends."""
    lens, E = [24], 8
    p = ref.scan_inputs(lens, E, 16, 1, F32, dt_bias=False)
    p["dt"] = torch.linspace(-60, 60, 24)[:, None].expand(24, E).contiguous()
    check(gdr, p, put(p), lens)


def test_nan_stays_in_its_channel_and_sequence(gdr):
    lens, E = [20, 20], 8
    p = put(ref.scan_inputs(lens, E, 16, 1, F32))
    p["x"][6, 3] = float("nan")
    y, ht = forward(gdr, p, ref.cu_of(lens, "cuda"))
    bad = y[0].isnan()
    assert bad[6:20, 3].all() and bad.sum() == 14
    assert ht[0, 3].isnan().all() and ht.isnan().sum() == 16


def test_gradient_against_differences(gdr):
    g = torch.Generator().manual_seed(8)
    lens = [12, 9]
    p = put(ref.scan_inputs(lens, 20, 8, 1, F32, seed=2))
    cu, h = ref.cu_of(lens, "cuda"), 1e-3
    names = ("x", "dt", "b", "c", "z", "h0")
    v = {k: torch.randn(p[k].shape, generator=g).cuda() for k in names}
    loss = lambda q: sum(float((o.double() * w.double()).sum()) for o, w in zip(forward(gdr, q, cu), (p["dy"], p["dht"])))  # noqa: E731
    up, down = (loss({**p, **{k: p[k] + s * v[k] for k in names}}) for s in (h, -h))
    got = dict(zip(OUT, backward(gdr, p, cu)))
    total = sum(float((got["d" + k].double().view(v[k].shape) * v[k].double()).sum()) for k in names)
    y, ht = forward(gdr, p, cu)
    size = float(y.double().norm() * p["dy"].double().norm() + ht.double().norm() * p["dht"].double().norm())
    # each value of y and ht is off by tol() of the norms; the third-order term
    assert abs((up - down) / (2 * h) - total) <= size * (ref.tol(F32, 12) / h / 4 + 200 * h * h)


@pytest.mark.parametrize("change,error", [
    (dict(a=lambda t: t.double()), RuntimeError), (dict(a=lambda t: t[:, :3].contiguous()), ValueError),
    (dict(a=lambda t: t.t().contiguous().t()), RuntimeError), (dict(b=lambda t: t[:, :, 0]), ValueError),
    (dict(c=lambda t: t[:, :, :, :3]), ValueError), (dict(dt=lambda t: t.float()), RuntimeError),
    (dict(b=lambda t: t.transpose(2, 3).contiguous().transpose(2, 3)), RuntimeError),
    (dict(x=lambda t: t[:, :, ::2].repeat(1, 1, 2)[:, :, ::1].transpose(1, 2).contiguous().transpose(1, 2)),
     RuntimeError)])
def test_refusals(gdr, change, error):
    q = dict(x=torch.zeros(1, 6, 16, dtype=BF16, device="cuda"), dt=torch.zeros(1, 6, 16, dtype=BF16, device="cuda"),
             a=torch.zeros(16, 4, device="cuda"), b=torch.zeros(1, 6, 2, 4, dtype=BF16, device="cuda"),
             c=torch.zeros(1, 6, 2, 4, dtype=BF16, device="cuda"))
    gdr.ssm_fwd(**q)
    with pytest.raises(error):
        gdr.ssm_fwd(**{k: change.get(k, lambda t: t)(v) for k, v in q.items()})


def test_thousands_of_short_sequences(gdr):
    g = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 4, (2500,), generator=g).tolist()
    p = ref.scan_inputs(lens, 10, 4, 1, F32, seed=12)
    check(gdr, p, put(p), lens)
