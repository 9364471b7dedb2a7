"""Norm of queries and keys for each head with the position rotation, on the GPU,
against the 64-bit definition."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.layer_reference import HALF_STEP, grads, rel

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
both_types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])


def close(got, want, rows=1, what="", terms=None):
    """One rounding of the output's type, and fp32 operations before it: the reciprocal root (2^-22), sums of up to 256
    products (16 roundings of 2^-24), a dozen more; sums over rows grow like sqrt(rows); four for cancellation.

    dx = rho (p - x rho^2 mean(p x)), p = w dn, is a difference of two `terms`: rho p, and its projection on x, whose
    norm is at most that of rho p.  Each is off by those 32 roundings of itself, so dx by at most 64 2^-24 |rho p|, a
    bound on the difference however much of it cancels (of one channel, all but eps does)."""
    err = rel(got, want)
    grows = 1.0 if terms is None or not float(want.norm()) else max(1.0, float(terms.norm() / want.norm()))
    bound = HALF_STEP[got.dtype] + 4 * (4 + 16 + 12) * math.sqrt(rows) * 2.0 ** -24 * grows
    assert err <= bound, f"{what}: relative error {err:.3e} over {bound:.3e}"


def put(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def run(gdr, q, interleaved, **kw):
    kw = dict(cos=q["cos"], sin=q["sin"], positions=q["positions"], interleaved=interleaved, **kw)
    yq, yk = gdr.qk_norm_fwd(q["q"], q["k"], q["wq"], q["wk"], **kw)
    dq, dk, dwq, dwk = gdr.qk_norm_bwd(q["dyq"], q["dyk"], q["q"], q["k"], q["wq"], q["wk"], **kw)
    return dict(yq=yq, yk=yk, dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def wanted(p, interleaved):
    d = {k: None if v is None else v if k == "positions" else v.double().cpu() for k, v in p.items()}
    pos = None if p["positions"] is None else p["positions"].cpu()
    want = {}
    for n in ("q", "k"):
        if p[n] is None:
            want.update({"y" + n: None, "d" + n: None, "dw" + n: None})
            continue
        fn = lambda x, w: (ref.heads(x, w, d["cos"], d["sin"], pos, interleaved),)  # noqa: E731
        want["y" + n] = fn(d[n], d["w" + n])[0]
        want["d" + n], want["dw" + n] = grads(fn, [d[n], d["w" + n]], (d["dy" + n],))
        # rho p: a turn keeps norms, so w dn is bounded by the largest weight times dy
        rho = 1 / torch.sqrt((d[n] * d[n]).mean(-1, keepdim=True) + 1e-6)
        want["terms d" + n] = rho * d["dy" + n] * float(d["w" + n].abs().max())
    return want


def check(got, p, interleaved):
    want = wanted(p, interleaved)
    for k, v in got.items():
        assert (want[k] is None) == (v is None), k
        if v is not None:
            rows = p["q"].shape[0] * max(p["q"].shape[1], 4) if k.startswith("dw") else 1
            close(v, want[k], rows, k, want.get("terms " + k))


@both_types
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("M,H,HK,D,R", [(1, 1, 1, 128, 64), (5, 4, 2, 128, 32), (33, 5, 3, 64, 32), (3, 2, 1, 256, 128),
                                        (4, 9, 0, 32, 16), (2, 1, 1, 8, 4), (3, 2, 2, 96, 48), (2, 3, 1, 200, 20),
                                        (40, 32, 8, 128, 64), (3, 2, 2, 24, 0), (2, 1, 1, 1, 0), (9, 2, 1, 7, 3),
                                        (5, 3, 2, 34, 17), (4, 2, 2, 250, 125), (3, 1, 2, 12, 6), (3, 2, 1, 255, 2),
                                        (700, 3, 1, 16, 8), (600, 3, 2, 10, 5)], ids=str)
def test_forward_and_backward(gdr, dtype, interleaved, M, H, HK, D, R):
    p = ref.head_inputs(M, H, HK, D, R, dtype, seed=D)
    got = run(gdr, put(p), interleaved)
    check(got, p, interleaved)
    assert gdr.device_status() == 0


@pytest.mark.parametrize("D,R", [(128, 64), (20, 5)])
def test_fp32_weights_of_bf16_heads(gdr, D, R):
    p = ref.head_inputs(6, 3, 2, D, R, BF16, seed=1, wdtype=F32)
    check(run(gdr, put(p), False), p, False)


@both_types
@pytest.mark.parametrize("D,R", [(64, 32), (12, 5)])
def test_padding_tokens(gdr, dtype, D, R):
    """Negative positions: rows of zeros, whatever lies in the padding, and no part in the weights' gradients."""
    p = ref.head_inputs(20, 3, 2, D, R, dtype, seed=2)
    p["positions"][[0, 7, 8, 19]] = torch.tensor([-1, -1, -100, -2 ** 40])
    want = p
    q = put({k: v.clone() for k, v in p.items()})
    for k in ("q", "k", "dyq", "dyk"):
        q[k][[0, 7, 8, 19]] = math.nan
    got = run(gdr, q, True)
    check(got, want, True)
    for k in ("yq", "yk", "dq", "dk"):
        assert (got[k][[0, 7, 8, 19]] == 0).all()
    assert gdr.device_status() == 0


@both_types
@pytest.mark.parametrize("D,R", [(64, 32), (12, 5)])
def test_positions_past_the_table(gdr, dtype, D, R):
    p = put(ref.head_inputs(20, 3, 2, D, R, dtype, seed=2))
    clean = run(gdr, p, False)
    p["positions"] = p["positions"].clone()
    p["positions"][3], p["positions"][11] = 64, 2 ** 62
    got = run(gdr, p, False)
    assert gdr.device_status() == gdr.GDR_ERR_POSITION
    rest = [i for i in range(20) if i not in (3, 11)]
    for k in ("yq", "yk", "dq", "dk"):
        assert (got[k][[3, 11]] == 0).all() and torch.equal(got[k][rest], clean[k][rest])


@both_types
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
@pytest.mark.parametrize("D,R", [(64, 32), (24, 5)])
def test_slices_and_unaligned_bases(gdr, dtype, offset, D, R):
    """q, k and their outputs' gradients as parts of wider rows; a batch of sequences."""
    p = ref.head_inputs(30, 4, 2, D, R, dtype, seed=3)
    q = put(p)
    wide = torch.zeros(30, 12 * D + 8 + offset, dtype=dtype, device="cuda")
    at = offset
    for k in ("q", "k", "dyq", "dyk"):
        n = p[k][0].numel()
        wide[:, at:at + n] = q[k].flatten(1)
        q[k] = wide[:, at:at + n].unflatten(1, p[k].shape[1:])
        at += n
    check(run(gdr, q, False), p, False)
    b = {k: v.view(3, 10, *v.shape[1:]) if k in ("q", "k", "dyq", "dyk", "positions") else v for k, v in q.items()}
    got = run(gdr, b, False)
    check({k: v.flatten(0, 1) if k in ("yq", "yk", "dq", "dk") else v for k, v in got.items()}, p, False)


@both_types
@pytest.mark.parametrize("D,R", [(64, 16), (12, 5)])
def test_rows_keep_to_themselves(gdr, dtype, D, R):
    p = put(ref.head_inputs(9, 4, 2, D, R, dtype, seed=4))
    clean = run(gdr, p, False)
    q = dict(p, q=p["q"].clone(), dyk=p["dyk"].clone())
    q["q"][4, 1, 3], q["dyk"][5, 0, 2] = math.nan, math.inf
    got = run(gdr, q, False)
    for k in ("yq", "yk", "dq", "dk"):
        hit = {"yq": (4, 1), "dq": (4, 1), "dk": (5, 0), "yk": None}[k]
        same = (got[k] == clean[k]).all(-1)
        if hit:
            assert not torch.isfinite(got[k][hit]).all()
            same[hit] = True
        assert same.all(), k


@both_types
def test_bits_repeat_and_graphs_replay(gdr, dtype):
    p = put(ref.head_inputs(1000, 8, 2, 64, 32, dtype, seed=5))
    a, b = run(gdr, p, False), run(gdr, p, False, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
    fixed = {k: torch.zeros_like(v) for k, v in p.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = run(gdr, fixed, False)
    for k, v in p.items():
        fixed[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], c[k]) for k in a)


def test_no_tokens(gdr):
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    yq, yk = gdr.qk_norm_fwd(z(0, 2, 8), z(0, 1, 8), z(8), z(8))
    assert yq.shape == (0, 2, 8) and yk.shape == (0, 1, 8)
    _, _, dwq, dwk = gdr.qk_norm_bwd(z(0, 2, 8), z(0, 1, 8), z(0, 2, 8), z(0, 1, 8), z(8), z(8))
    assert (dwq == 0).all() and (dwk == 0).all()


def test_shapes_and_types_are_checked(gdr):
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, k, w = z(4, 2, 16), z(4, 1, 16), z(16)
    cos, pos = z(8, 4, dt=F32), z(4, dt=torch.int64)
    f = gdr.qk_norm_fwd
    bad = [(ValueError, lambda: f(q, k[:3], w, w)), (ValueError, lambda: f(q, z(4, 1, 8), w, w)),
           (ValueError, lambda: f(q, k, w[:8], w)), (gdr.GdrError, lambda: f(q, k.float(), w, w)),
           (gdr.GdrError, lambda: f(q, k, w, w.float())), (gdr.GdrError, lambda: f(q, k, w, None)),
           (ValueError, lambda: f(q, k, w, w, None, cos, pos)), (ValueError, lambda: f(q, k, w, w, positions=pos)),
           (gdr.GdrError, lambda: f(q, k, w, w, cos)), (gdr.GdrError, lambda: f(q, k, w, w, cos, cos)),
           (ValueError, lambda: f(q, k, w, w, cos, cos[:7], pos)), (ValueError, lambda: f(q, k, w, w, cos, cos, pos[:3])),
           (gdr.GdrError, lambda: f(q, k, w, w, cos, cos, pos.int())),
           (ValueError, lambda: f(q, k, w, w, z(8, 9, dt=F32), z(8, 9, dt=F32), pos)),
           (ValueError, lambda: gdr.qk_norm_bwd(q[:, :1], k, q, k, w, w)), (gdr.GdrError, lambda: f(q.half(), None, w, None))]
    for kind, g in bad:
        with pytest.raises(kind):
            g()
    assert gdr.device_status() == 0
