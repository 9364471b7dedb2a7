"""The short causal convolution, forward, backward and one token at a time, on
the GPU against the 64-bit definition."""
import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# borders at the first and last tokens of runs and batches, sequences shorter than the filter, empty ones anywhere
LENGTHS = [[1], [2], [3], [33], [16, 16], [0, 5, 0, 0, 1, 2, 3, 40, 0], [1] * 20, [7, 9, 8, 24, 1, 63], [0, 0], [100, 28]]
SIZES = [(1, 4), (3, 2), (8, 4), (64, 3), (130, 4), (520, 2), (1031, 4), (2048, 4)]


def put(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def batch(p, *names):
    return [p[k][None] for k in names]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "_".join(map(str, v))[:24])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_forward_and_backward(gdr, lens, dtype):
    for (E, W), bias, silu in zip(SIZES, [True, False] * 4, [True, True, False] * 3):
        p = ref.conv_inputs(lens, E, W, dtype, seed=E, bias=bias, wdtype=F32 if E == 64 else None)
        q, cu, act = put(p), ref.cu_of(lens, "cuda"), "silu" if silu else None
        M = max(1, sum(lens))
        y, st = gdr.conv_fwd(q["x"][None], q["weight"], bias=q["bias"], s0=q["s0"], cu_seqlens=cu, activation=act)
        fn = lambda x, w, b, s0: ref.conv(x, w, b, s0, lens, silu)  # noqa: E731
        want_y, want_st = fn(*[ref.f64(p[k]) for k in ("x", "weight", "bias", "s0")])
        ref.close(y[0], want_y, W, "y")
        assert torch.equal(st.cpu().double(), want_st)
        dx, dw, db, ds0 = gdr.conv_bwd(q["x"][None], q["weight"], q["dy"][None], bias=q["bias"], s0=q["s0"],
                                       dst=q["dst"], cu_seqlens=cu, activation=act)
        want = ref.grads(fn, [p[k] for k in ("x", "weight", "bias", "s0")], (p["dy"].double(), p["dst"].double()))
        ref.close(dx[0], want[0], W, "dx")
        ref.close(dw, want[1], M, "dweight")
        assert (db is None) == (not bias)
        if bias:
            ref.close(db, want[2], M, "dbias")
        ref.close(ds0, want[3], W, "ds0")
        assert gdr.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
def test_dense_batch_without_states(gdr, dtype):
    for B, T in ((3, 50), (2, 1), (1, 129), (0, 4), (2, 0)):
        lens = [T] * B
        p = ref.conv_inputs(lens, 96, 4, dtype, seed=T)
        x = p["x"].view(B, T, 96)
        y, st = gdr.conv_fwd(x.cuda(), p["weight"].cuda(), bias=p["bias"].cuda())
        none = torch.zeros(B, 3, 96, dtype=torch.float64)
        assert y.shape == x.shape and st.shape == none.shape
        if B:
            want_y, want_st = ref.conv(*[ref.f64(p[k]) for k in ("x", "weight", "bias")], none, lens)
            ref.close(y.flatten(0, 1), want_y, 4, "y")
            assert torch.equal(st.cpu().double(), want_st)
        y2, st2 = gdr.conv_fwd(x.cuda(), p["weight"].cuda(), bias=p["bias"].cuda(), output_final_state=False)
        assert st2 is None and torch.equal(y2, y)
        got = gdr.conv_bwd(x.cuda(), p["weight"].cuda(), p["dy"].view(B, T, 96).cuda(), bias=p["bias"].cuda())
        if B:
            fn = lambda x, w, b: ref.conv(x, w, b, none, lens)[:1]  # noqa: E731
            want = ref.grads(fn, [p[k] for k in ("x", "weight", "bias")], (p["dy"].double(),))
            ref.close(got[0].flatten(0, 1), want[0], 4, "dx")
            ref.close(got[1], want[1], max(1, B * T), "dweight")
            ref.close(got[2], want[2], max(1, B * T), "dbias")
        else:
            assert got[1].eq(0).all() and got[2].eq(0).all()


def test_long_runs(gdr):
    """Enough tokens that a run is many batches long; borders inside runs; the same bits each time."""
    lens, E = [30000, 1, 0, 20011, 2, 15000], 512
    p = put(ref.conv_inputs(lens, E, 4, BF16, seed=2))
    cu = ref.cu_of(lens, "cuda")
    args = dict(bias=p["bias"], s0=p["s0"], cu_seqlens=cu)
    y, st = gdr.conv_fwd(p["x"][None], p["weight"], **args)
    fn = lambda x, w, b, s0: ref.conv(x, w, b, s0, lens)  # noqa: E731
    want_y, want_st = fn(*[ref.f64(p[k]) for k in ("x", "weight", "bias", "s0")])
    ref.close(y[0], want_y, 4, "y")
    assert torch.equal(st.double(), want_st)
    got = [gdr.conv_bwd(p["x"][None], p["weight"], p["dy"][None], dst=p["dst"], **args) for _ in range(2)]
    assert all(torch.equal(u, v) for u, v in zip(*got))
    want = ref.grads(fn, [p[k] for k in ("x", "weight", "bias", "s0")], (p["dy"].double(), p["dst"].double()))
    for u, v, n, what in zip(got[0], want, (4, sum(lens), sum(lens), 4), ("dx", "dweight", "dbias", "ds0")):
        ref.close(u[0] if what == "dx" else u, v, n, what)


@pytest.mark.parametrize("offset", [0, 1, 4])
def test_slices_and_unaligned_bases(gdr, offset):
    lens, E = [19, 21], 64
    p = put(ref.conv_inputs(lens, E, 4, BF16, seed=3))
    cu = ref.cu_of(lens, "cuda")
    wide = torch.zeros(40, 2 * E + 5, dtype=BF16, device="cuda")  # rows 133 apart
    wide[:, offset:offset + E] = p["x"]
    x = wide[None, :, offset:offset + E]
    assert not x.is_contiguous()
    a = gdr.conv_fwd(x, p["weight"], bias=p["bias"], s0=p["s0"], cu_seqlens=cu)
    b = gdr.conv_fwd(p["x"][None], p["weight"], bias=p["bias"], s0=p["s0"], cu_seqlens=cu)
    assert all(torch.equal(u, v) for u, v in zip(a, b))  # one order of operations for every alignment
    c = gdr.conv_bwd(x, p["weight"], x, bias=p["bias"], s0=p["s0"], cu_seqlens=cu)
    d = gdr.conv_bwd(p["x"][None], p["weight"], p["x"][None], bias=p["bias"], s0=p["s0"], cu_seqlens=cu)
    assert all(torch.equal(u, v) for u, v in zip(c, d))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,W", [(1, 2), (7, 4), (64, 3), (1000, 4), (1031, 4)])
def test_steps_equal_a_prompt(gdr, E, W, dtype):
    """Tokens one by one through a pool of slots give what the prompt gives, and its final state."""
    lens = [6, 6, 6]
    p = put(ref.conv_inputs(lens, E, W, dtype, seed=4))
    x = p["x"].view(3, 6, E)
    y, st = gdr.conv_fwd(x, p["weight"], bias=p["bias"], s0=p["s0"])
    pool = torch.full((7, W - 1, E), 9.0, dtype=dtype, device="cuda")
    slots = torch.tensor([5, 0, 3, -1], dtype=torch.int32, device="cuda")
    pool[slots[:3].long()] = p["s0"]
    for t in range(6):
        row = torch.cat([x[:, t], x[:1, t]])
        out = gdr.conv_step(row, pool, p["weight"], bias=p["bias"], slots=slots)
        assert torch.equal(out[:3], y[:, t]) and out[3].eq(0).all()
    assert torch.equal(pool[slots[:3].long()], st)
    assert pool[[1, 2, 4, 6]].eq(9.0).all() and gdr.device_status() == 0


def test_slots_past_the_pool_are_reported(gdr):
    p = put(ref.conv_inputs([3], 32, 4, BF16))
    pool = torch.ones(2, 3, 32, dtype=BF16, device="cuda")
    y = gdr.conv_step(p["x"], pool, p["weight"], slots=torch.tensor([2, 0, 2 ** 30], dtype=torch.int32, device="cuda"))
    assert gdr.device_status() == gdr.GDR_ERR_SLOTS and gdr.device_status() == 0
    assert y[[0, 2]].eq(0).all() and not y[1].eq(0).all() and pool[1].eq(1).all()


@pytest.mark.parametrize("cu", [[0, 3, 2, 8], [1, 4, 8], [0, 4, 9], [0, 4, 7]])
def test_bad_cu_seqlens_touch_nothing(gdr, cu):
    from chunked_gated_delta_08_gb300 import layer_ops as ops
    import ctypes
    N, E = len(cu) - 1, 16
    p = put(ref.conv_inputs([8], E, 4, F32))
    cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
    out = {n: torch.full(s, 7.0, device="cuda") for n, s in
           (("y", (8, E)), ("st", (N, 3, E)), ("dw", (E, 4)), ("db", (E,)))}
    desc = ops.GdrConvDesc(1, 8, E, N, 4, E, E, 0, 0, 1, 0)
    a = lambda t: t.data_ptr()  # noqa: E731
    s = torch.cuda.current_stream().cuda_stream
    assert gdr.lib().gdr_conv_fwd(ctypes.byref(desc), a(p["x"]), a(p["weight"]), None, None, a(cu), a(out["y"]),
                                  a(out["st"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert gdr.lib().gdr_conv_bwd(ctypes.byref(desc), a(p["x"]), a(p["weight"]), a(p["bias"]), None, a(cu), a(p["dy"]),
                                  None, a(out["y"]), a(out["dw"]), a(out["db"]), a(out["st"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert all(t.eq(7.0).all() for t in out.values())


def test_nan_stays_in_its_channel_and_reach(gdr):
    p = put(ref.conv_inputs([10, 10], 8, 4, F32))
    p["x"][3, 2] = float("nan")
    y, _ = gdr.conv_fwd(p["x"][None], p["weight"], cu_seqlens=ref.cu_of([10, 10], "cuda"))
    bad = y[0].isnan()
    assert bad[3:7, 2].all() and bad.sum() == 4


def test_gradient_against_differences(gdr):
    g = torch.Generator().manual_seed(8)
    x, v, dy = (torch.randn(2, 9, 40, generator=g).cuda() for _ in range(3))
    w, u = (torch.randn(40, 4, generator=g).cuda() for _ in range(2))
    h = 1e-2
    up, down = (gdr.conv_fwd(x + k * v, w + k * u)[0].double() for k in (h, -h))
    diff = float(((up - down) * dy.double()).sum()) / (2 * h)
    dx, dw, _, _ = gdr.conv_bwd(x, w, dy)
    got = float((dx.double() * v.double()).sum() + (dw.double() * u.double()).sum())
    size = float(dy.double().norm() * up.norm())
    # rounding of the two values over 2 h; the third-order term, whose directions are a unit per element and tap
    assert abs(diff - got) <= size * (2.0 ** -23 * 8 / h + 8 * h * h)


@pytest.mark.parametrize("call,error", [
    (lambda g, x, w: g.conv_fwd(x, w[:, :1].contiguous()), ValueError),
    (lambda g, x, w: g.conv_fwd(x, torch.cat([w, w], 1)), ValueError),
    (lambda g, x, w: g.conv_fwd(x, w[:8]), ValueError),
    (lambda g, x, w: g.conv_fwd(x, w, activation="relu"), ValueError),
    (lambda g, x, w: g.conv_fwd(x, w, s0=x), ValueError),
    (lambda g, x, w: g.conv_fwd(x, w, bias=w[:, 0]), RuntimeError),
    (lambda g, x, w: g.conv_fwd(x, w, cu_seqlens=torch.tensor([0, 6], device="cuda")), ValueError),
    (lambda g, x, w: g.conv_fwd(x, w, cu_seqlens=torch.tensor([0, 6], dtype=torch.int32, device="cuda")), RuntimeError),
    (lambda g, x, w: g.conv_fwd(x.transpose(1, 2), w[:6]), RuntimeError),
    (lambda g, x, w: g.conv_fwd(x.expand(2, 6, 16)[:, :1].expand(2, 6, 16), w), RuntimeError),
    (lambda g, x, w: g.conv_step(x[0], torch.zeros(5, 3, 16, device="cuda", dtype=BF16), w), ValueError),
    (lambda g, x, w: g.conv_step(x[0], torch.zeros(6, 3, 16, device="cuda"), w), RuntimeError),
    (lambda g, x, w: g.conv_step(x[0], torch.zeros(6, 3, 16, device="cuda", dtype=BF16), w,
                                 slots=torch.zeros(6, dtype=torch.int64, device="cuda")), RuntimeError)])
def test_refusals(gdr, call, error):
    x = torch.zeros(2, 6, 16, dtype=BF16, device="cuda")
    with pytest.raises(error):
        call(gdr, x, torch.zeros(16, 4, dtype=BF16, device="cuda"))


def test_thousands_of_short_sequences(gdr):
    g = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 7, (2500,), generator=g).tolist()
    p = ref.conv_inputs(lens, 20, 4, F32, seed=12)
    q, cu = put(p), ref.cu_of(lens, "cuda")
    fn = lambda x, w, b, s0: ref.conv(x, w, b, s0, lens)  # noqa: E731
    y, st = gdr.conv_fwd(q["x"][None], q["weight"], bias=q["bias"], s0=q["s0"], cu_seqlens=cu)
    want_y, want_st = fn(*[ref.f64(p[k]) for k in ("x", "weight", "bias", "s0")])
    ref.close(y[0], want_y, 4, "y")
    assert torch.equal(st.cpu().double(), want_st)
    got = gdr.conv_bwd(q["x"][None], q["weight"], q["dy"][None], bias=q["bias"], s0=q["s0"], dst=q["dst"], cu_seqlens=cu)
    want = ref.grads(fn, [p[k] for k in ("x", "weight", "bias", "s0")], (p["dy"].double(), p["dst"].double()))
    for u, v, n, what in zip(got, want, (4, sum(lens), sum(lens), 4), ("dx", "dweight", "dbias", "ds0")):
        ref.close(u[0] if what == "dx" else u, v, n, what)
