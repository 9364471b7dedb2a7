"""The layer operators' edge cases in calls of several launches, and in those of
one: lengths of up to 64 tokens are one chunk (scan) or one run (convolution
backward), longer ones are cut and carried.  The count of launches says which
path a call took."""
import ctypes

import pytest
import torch

from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("x", "dt", "a", "b", "c", "d", "z", "dt_bias", "h0")
OUT = ("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh0")
SHORT, LONG = [30, 21], [90, 5, 0, 130]
both_lengths = pytest.mark.parametrize("lens", [SHORT, LONG], ids=["one_chunk", "chunks"])
both_types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])


def put(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


class Launches:
    def __init__(self, gdr, expected):
        self.gdr, self.expected = gdr, expected

    def __enter__(self):
        self.before = self.gdr.launch_count()

    def __exit__(self, kind, *_):
        if kind is None:
            assert self.gdr.launch_count() - self.before == self.expected


def scan(gdr, q, lens, **kw):
    lead = lambda t: None if t is None else t[None]  # noqa: E731
    cu, many = ref.cu_of(lens, "cuda"), sum(lens) > 64
    args = (lead(q["x"]), lead(q["dt"]), q["a"], lead(q["b"]), lead(q["c"]))
    kw = dict(d=q["d"], z=lead(q["z"]), dt_bias=q["dt_bias"], h0=q["h0"], cu_seqlens=cu, **kw)
    with Launches(gdr, 3 if many else 1):
        y, ht = gdr.ssm_fwd(*args, **kw)
    with Launches(gdr, 4 if many else 2):
        back = gdr.ssm_bwd(*args, lead(q["dy"]), dht=q["dht"], **kw)
    assert gdr.device_status() == 0
    return dict(zip(("y", "ht") + OUT, (y, ht) + back))


def check_scan(gdr, p, lens, softplus=True):
    fn = lambda *v: ref.scan(*v, lens, softplus)  # noqa: E731
    got = scan(gdr, put(p), lens, dt_softplus=softplus)
    want = dict(zip(("y", "ht"), fn(*[ref.f64(p[k]) for k in NAMES])))
    want.update(zip(OUT, ref.grads(fn, [p[k] for k in NAMES], (p["dy"].double(), p["dht"].double()))))
    T, M = max(lens), sum(lens)
    for k, w in want.items():
        assert (got[k] is None) == (w is None), k
        if w is not None:
            packed = k in ("y", "dx", "ddt", "db", "dc", "dz")
            ref.close(got[k][0] if packed else got[k], w, T if packed or k in ("ht", "dh0") else M, k)


@both_lengths
@both_types
@pytest.mark.parametrize("softplus", [True, False], ids=["softplus", "raw"])
@pytest.mark.parametrize("missing", ["d", "z", "dt_bias", "all", "none"])
def test_scan_optional_terms(gdr, lens, dtype, softplus, missing):
    have = {k: missing not in (k, "all") for k in ("d", "z", "dt_bias")}
    p = ref.scan_inputs(lens, 24, 16, 1, dtype, seed=3, **have)
    if not softplus:  # delta is dt (and bias) itself: small and positive
        p["dt"] = p["dt"].abs() * 0.1
        if p["dt_bias"] is not None:
            p["dt_bias"] = p["dt_bias"].abs() * 0.01
    check_scan(gdr, p, lens, softplus)


@both_lengths
@pytest.mark.parametrize("S,G", [(3, 2), (12, 1), (32, 1), (33, 2), (64, 1)], ids=str)
def test_scan_numbers_of_states(gdr, lens, S, G):
    check_scan(gdr, ref.scan_inputs(lens, 40, S, G, BF16, seed=S), lens)


@both_lengths
@both_types
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_scan_slices_and_unaligned_bases(gdr, lens, dtype, offset):
    """x, dt, z, b, c and dy as parts of wider rows: the contiguous call's results."""
    E, S = 64, 16
    p = put(ref.scan_inputs(lens, E, S, 1, dtype, seed=3))
    wide = torch.zeros(sum(lens), 4 * E + 2 * S + 8 + offset, dtype=dtype, device="cuda")
    at, q = offset, dict(p)
    for k, n in (("x", E), ("dt", E), ("z", E), ("dy", E), ("b", S), ("c", S)):
        wide[:, at:at + n] = p[k].flatten(1)
        q[k] = wide[:, at:at + n].unflatten(1, p[k].shape[1:])
        at += n
    a, b = scan(gdr, q, lens), scan(gdr, p, lens)
    assert all(torch.equal(a[k], b[k]) for k in a)


@both_lengths
@both_types
def test_scan_unaligned_states(gdr, lens, dtype):
    """States, a and the states' gradients one element past a 16-byte border."""
    p = put(ref.scan_inputs(lens, 24, 16, 1, dtype, seed=4))
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    q = dict(p, a=off(p["a"]), h0=off(p["h0"]), dht=off(p["dht"]))
    assert q["h0"].data_ptr() % 16 and q["dht"].data_ptr() % 16 and q["a"].data_ptr() % 16
    a, b = scan(gdr, q, lens), scan(gdr, p, lens)
    assert all(torch.equal(a[k], b[k]) for k in a)


@both_lengths
def test_scan_extreme_deltas(gdr, lens):
    """Large, tiny and negative dt within each sequence: the state forgotten at once, kept for ever."""
    p = ref.scan_inputs(lens, 8, 16, 1, F32, dt_bias=False)
    p["dt"] = torch.cat([torch.linspace(-60, 60, n) for n in lens])[:, None].expand(-1, 8).contiguous()
    check_scan(gdr, p, lens)


BAD = [lambda T: [0, 30, 20, T], lambda T: [1, 40, T], lambda T: [0, 40, T + 1], lambda T: [0, 40, T - 1]]


@pytest.mark.parametrize("T", [50, 220], ids=["one_chunk", "chunks"])
@pytest.mark.parametrize("bad", range(len(BAD)))
@both_types
def test_bad_cu_seqlens_touch_nothing(gdr, T, bad, dtype):
    from chunked_gated_delta_08_gb300 import layer_ops as ops
    cu = torch.tensor(BAD[bad](T), dtype=torch.int64, device="cuda")
    N, E, S, code = cu.numel() - 1, 16, 8, 0 if dtype == F32 else 1
    s, many = torch.cuda.current_stream().cuda_stream, T > 64
    a = lambda t: t.data_ptr()  # noqa: E731
    full = lambda dt, **shapes: {k: torch.full(v, 7.0, dtype=dt, device="cuda") for k, v in shapes.items()}  # noqa: E731
    p = put(ref.scan_inputs([T], E, S, 1, dtype))
    o = {**full(dtype, y=(T, E), dx=(T, E), ddt=(T, E), dz=(T, E), db=(T, S), dc=(T, S)),
         **full(F32, da=(E, S), dd=(E,), dbias=(E,), ht=(N, E, S), dh0=(N, E, S))}
    desc = ops.GdrSsmDesc(1, T, E, S, 1, N, E, E, E, S, S, E, code, 1)
    head = [a(p[k]) for k in ("x", "dt", "a", "b", "c", "d", "z", "dt_bias")] + [None, a(cu)]
    with Launches(gdr, 3 if many else 1):
        assert gdr.lib().gdr_ssm_fwd(ctypes.byref(desc), *head, a(o["y"]), a(o["ht"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    with Launches(gdr, 4 if many else 2):
        assert gdr.lib().gdr_ssm_bwd(ctypes.byref(desc), *head, a(p["dy"]), None, a(o["dx"]), a(o["ddt"]), a(o["da"]),
                                     a(o["db"]), a(o["dc"]), a(o["dd"]), a(o["dz"]), a(o["dbias"]), a(o["dh0"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    q = put(ref.conv_inputs([T], E, 4, dtype))
    c = {**full(dtype, y=(T, E), dx=(T, E), st=(N, 3, E), ds0=(N, 3, E)), **full(F32, dw=(E, 4), db=(E,))}
    cdesc = ops.GdrConvDesc(1, T, E, N, 4, E, E, code, code, 1, 0)
    assert gdr.lib().gdr_conv_fwd(ctypes.byref(cdesc), a(q["x"]), a(q["weight"]), a(q["bias"]), None, a(cu), a(c["y"]),
                                  a(c["st"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    with Launches(gdr, 2 if many else 1):
        assert gdr.lib().gdr_conv_bwd(ctypes.byref(cdesc), a(q["x"]), a(q["weight"]), a(q["bias"]), None, a(cu),
                                      a(q["dy"]), None, a(c["dx"]), a(c["dw"]), a(c["db"]), a(c["ds0"]), s) == 0
    assert gdr.device_status() == gdr.GDR_ERR_SEQLENS
    assert all(t.eq(7.0).all() for t in [*o.values(), *c.values()])


def test_dense_sequences_of_several_tiles_in_one_launch(gdr):
    """Enough sequences to fill the GPU: each is one chunk, whatever its length."""
    B, T, E, S = 304, 40, 256, 16
    p = ref.scan_inputs([T] * B, E, S, 1, BF16, seed=5, device="cuda")
    lead = lambda t: t.view(B, T, *t.shape[1:])  # noqa: E731
    with Launches(gdr, 1):
        y, ht = gdr.ssm_fwd(lead(p["x"]), lead(p["dt"]), p["a"], lead(p["b"]), lead(p["c"]), d=p["d"], z=lead(p["z"]),
                            dt_bias=p["dt_bias"], h0=p["h0"])
    for n in (0, 1, 151, 302, 303):
        part = lambda k: p[k].double() if k in ("a", "d", "dt_bias") else p[k][n:n + 1].double() if k == "h0" \
            else p[k][n * T:(n + 1) * T].double()  # noqa: E731
        want_y, want_ht = ref.scan(*[part(k) for k in NAMES], [T])
        ref.close(y[n], want_y, T, "y")
        ref.close(ht[n:n + 1], want_ht, T, "ht")


@both_lengths
@both_types
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_conv_slices_and_unaligned_bases(gdr, lens, dtype, offset):
    E, M = 64, sum(lens)
    p = ref.conv_inputs(lens, E, 4, dtype, seed=3)
    q, cu = put(p), ref.cu_of(lens, "cuda")
    wide = torch.zeros(M, 2 * E + 5, dtype=dtype, device="cuda")  # rows 133 apart
    wide[:, offset:offset + E], wide[:, E + offset:2 * E + offset] = q["x"], q["dy"]
    x, dy = wide[None, :, offset:offset + E], wide[None, :, E + offset:2 * E + offset]
    assert not x.is_contiguous()
    y, st = gdr.conv_fwd(x, q["weight"], bias=q["bias"], s0=q["s0"], cu_seqlens=cu)
    with Launches(gdr, 2 if M > 64 else 1):
        got = gdr.conv_bwd(x, q["weight"], dy, bias=q["bias"], s0=q["s0"], dst=q["dst"], cu_seqlens=cu)
    fn = lambda x, w, b, s0: ref.conv(x, w, b, s0, lens)  # noqa: E731
    want_y, want_st = fn(*[ref.f64(p[k]) for k in ("x", "weight", "bias", "s0")])
    ref.close(y[0], want_y, 4, "y")
    assert torch.equal(st.cpu().double(), want_st)
    want = ref.grads(fn, [p[k] for k in ("x", "weight", "bias", "s0")], (p["dy"].double(), p["dst"].double()))
    for u, v, n, what in zip(got, want, (4, M, M, 4), ("dx", "dweight", "dbias", "ds0")):
        ref.close(u[0] if what == "dx" else u, v, n, what)


@both_types
@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("where", ["x", "dt", "b", "c", "z", "dy", "dht", "h0"])
def test_scan_sequences_keep_to_themselves_in_one_chunk(gdr, dtype, where, value):
    lens = [20, 12, 30]
    p = put(ref.scan_inputs(lens, 24, 12, 2, dtype, seed=6))
    clean = scan(gdr, p, lens)
    q = dict(p)
    q[where] = p[where].clone()
    q[where][1 if where in ("dht", "h0") else slice(20, 32)] = value
    got = scan(gdr, q, lens)
    for n, i, j in ref.spans(lens):
        for k in ("y", "dx", "ddt", "db", "dc", "dz", "ht", "dh0"):
            mine, want = (v[n] if k in ("ht", "dh0") else v[0, i:j] for v in (got[k], clean[k]))
            assert n == 1 or torch.equal(mine, want), (k, n)


@both_types
@pytest.mark.parametrize("lens", [[20, 12, 30], [100, 30, 90]], ids=["one_run", "runs"])
@pytest.mark.parametrize("where", ["x", "dy", "s0", "dst"])
def test_conv_sequences_keep_to_themselves(gdr, lens, dtype, where):
    E = 24
    p, cu = put(ref.conv_inputs(lens, E, 4, dtype, seed=6)), ref.cu_of(lens, "cuda")

    def call(q):
        y, st = gdr.conv_fwd(q["x"][None], q["weight"], bias=q["bias"], s0=q["s0"], cu_seqlens=cu)
        with Launches(gdr, 2 if sum(lens) > 64 else 1):
            dx, _, _, ds0 = gdr.conv_bwd(q["x"][None], q["weight"], q["dy"][None], bias=q["bias"], s0=q["s0"],
                                         dst=q["dst"], cu_seqlens=cu)
        return dict(y=y[0], dx=dx[0], st=st, ds0=ds0)
    clean, q = call(p), dict(p)
    for value in (float("nan"), float("inf")):
        q[where] = p[where].clone()
        q[where][1 if where in ("s0", "dst") else slice(lens[0], lens[0] + lens[1])] = value
        got = call(q)
        for n, i, j in ref.spans(lens):
            for k, v in got.items():
                mine, want = (u[n] if k in ("st", "ds0") else u[i:j] for u in (v, clean[k]))
                assert n == 1 or torch.equal(mine, want), (k, n)
