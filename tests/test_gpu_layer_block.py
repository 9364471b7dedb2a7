"""The layer operators together, as examples/ssm_layer.py runs them: prefill,
decode and training step; on another stream; captured into a graph."""
import torch

import pytest

from examples.ssm_layer import SsmLayer, main
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu


def batch(layer, T, seed=0, B=1):
    g = torch.Generator().manual_seed(seed)
    width = layer.p["norm"].numel()
    return [torch.randn(B, T, width, generator=g).to(device="cuda", dtype=layer.dtype) for _ in range(2)]


def reference_layer(p, x, residual, lens, rank, states):
    """The layer in 64 bits with automatic differentiation."""
    s = x + residual
    n = ref.norm(s, p["norm"], 1e-6)
    xz = n @ p["w_in"].t()
    inner = p["w_out"].shape[1]
    N, W = len(lens), p["conv_w"].shape[1]
    u, _ = ref.conv(xz[:, :inner], p["conv_w"], p["conv_b"], xz.new_zeros(N, W - 1, inner), lens)
    dbc = u @ p["w_bc"].t()
    b, c = (dbc[:, i:i + states][:, None] for i in (rank, rank + states))
    y, _ = ref.scan(u, dbc[:, :rank] @ p["w_dt"].t(), p["a"], b, c, p["d"], xz[:, inner:], p["dt_bias"],
                    xz.new_zeros(N, inner, states), lens)
    return y @ p["w_out"].t(), s


def test_layer_against_the_definition(gdr):
    """fp32, so that matrix products in 64 bits and in 32 differ by a few roundings of their terms."""
    lens = [40, 1, 0, 23]
    layer = SsmLayer(width=48, inner=72, states=12, rank=5, dtype=torch.float32)
    x, residual = batch(layer, 64)
    cu = ref.cu_of(lens, "cuda")
    out, res, _, saved = layer.prefill(x, residual, cu_seqlens=cu)
    g = torch.Generator().manual_seed(4)
    dout, ds = (torch.randn(1, 64, 48, generator=g).cuda() for _ in range(2))
    dx, grads = layer.backward(saved, dout, ds)
    leaves = {k: v.double().requires_grad_() for k, v in layer.p.items()}
    lx = x[0].double().requires_grad_()
    want_out, want_res = reference_layer(leaves, lx, residual[0].double(), lens, 5, 12)
    loss = (want_out * dout[0].double()).sum() + (want_res * ds[0].double()).sum()
    want = torch.autograd.grad(loss, [lx, *leaves.values()])
    # each of the layer's six stages hands on its own roundings: six times one operator's bound
    n = 6 * 6 * 64
    ref.close(out[0], want_out, n, "out")
    ref.close(dx[0], want[0], n, "dx")
    for k, w in zip(leaves, want[1:]):
        ref.close(grads[k], w, n, k)


def test_decode_continues_a_prefill(gdr):
    """The states that a prefill leaves, moved to slots, carry on as the longer prompt does: within fp32
    roundings, through six stages."""
    layer = SsmLayer(width=64, inner=136, states=16, rank=8, dtype=torch.float32)
    x, residual = batch(layer, 40, seed=1, B=3)
    want, _, (want_st, want_ht), _ = layer.prefill(x, residual)
    _, _, (st, ht), _ = layer.prefill(x[:, :33].contiguous(), residual[:, :33].contiguous())
    pool = layer.empty_states(5)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool[0][slots.long()], pool[1][slots.long()] = st, ht
    for t in range(33, 40):
        y, _ = layer.step(x[:, t].contiguous(), residual[:, t].contiguous(), pool, slots)
        assert ref.rel(y, want[:, t]) <= ref.tol(torch.float32, 36 * 40)
    assert ref.rel(pool[1][slots.long()], want_ht) <= ref.tol(torch.float32, 36 * 40)


def test_another_stream_gives_the_same(gdr):
    p = ref.scan_inputs([700, 300], 256, 16, 1, torch.bfloat16, device="cuda")
    q = ref.conv_inputs([700, 300], 256, 4, torch.bfloat16, device="cuda")
    cu = ref.cu_of([700, 300], "cuda")
    r = torch.randn(1000, 256, device="cuda")
    w = torch.ones(256, device="cuda")

    def run(stream):
        lead = [p[k][None] for k in ("x", "dt")]
        bc = [p[k][None] for k in ("b", "c")]
        kw = dict(h0=p["h0"], cu_seqlens=cu, stream=stream)
        return [*gdr.ssm_fwd(*lead, p["a"], *bc, **kw),
                *gdr.ssm_bwd(*lead, p["a"], *bc, p["dy"][None], dht=p["dht"], **kw)[:5],
                *gdr.conv_fwd(q["x"][None], q["weight"], s0=q["s0"], cu_seqlens=cu, stream=stream),
                *gdr.conv_bwd(q["x"][None], q["weight"], q["dy"][None], cu_seqlens=cu, stream=stream)[:2],
                *gdr.norm_bwd(r, r, w, stream=stream), *gdr.norm_fwd(r, w, r, quant="group", stream=stream)]
    here = run(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = run(side)
    torch.cuda.current_stream().wait_stream(side)
    for u, v in zip(here, there):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_captured_into_graphs(gdr):
    """A decode step and a training step replay from graphs, on new inputs in the same memory, with the eager results."""
    layer = SsmLayer(width=64, inner=128, states=16, rank=8)
    x, residual = batch(layer, 50, seed=2)
    pool = layer.empty_states(3)
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    row, row_res = x[0, :2].clone(), residual[0, :2].clone()

    def train():
        out, res, _, saved = layer.prefill(x, residual)
        dx, g = layer.backward(saved, out, res)
        return [out, dx, *g.values()]

    def decode():
        return list(layer.step(row, row_res, pool, slots))
    for fn in (train, decode):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # warm-up: the status word and the scratch pool are made
            fn()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = fn()
        for seed in (5, 6):
            new_x, new_res = batch(layer, 50, seed=seed)
            x.copy_(new_x), residual.copy_(new_res)
            row.copy_(new_x[0, 3:5]), row_res.copy_(new_res[0, 3:5])
            before = [t.clone() for t in pool]
            graph.replay()
            got = [t.clone() for t in held] + [t.clone() for t in pool]
            for t, v in zip(pool, before):
                t.copy_(v)
            want = fn() + list(pool)
            assert all(torch.equal(u, v) for u, v in zip(got, want))
    assert gdr.device_status() == 0


def test_example_runs(gdr, capsys):
    main()
    text = capsys.readouterr().out
    losses = [float(line.split()[-1]) for line in text.splitlines() if line.startswith("step")]
    assert len(losses) == 5 and losses[-1] < losses[0]
    assert float(text.split("relative difference ")[1].split()[0]) <= 6 * 2.0 ** -8  # six stages' bf16 roundings
