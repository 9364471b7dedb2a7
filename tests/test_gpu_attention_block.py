"""Linear attention and its norms together, as examples/linear_attention_layer.py
runs them: prefill, decode and training step; captured into graphs; on another
stream; unaligned states; offsets past 32 bits."""
import pytest
import torch

from examples.linear_attention_layer import LinearAttentionLayer, main
from tests import attention_reference as ref
from tests import layer_reference

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def batch(layer, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    width = layer.p["norm"].numel()
    return [torch.randn(1, T, width, generator=g).to(device="cuda", dtype=layer.dtype) for _ in range(2)]


def places(lens):
    return torch.cat([torch.arange(n) for n in lens]).cuda()


def reference_layer(layer, p, x, residual, lens):
    """The layer in 64 bits with automatic differentiation, on the CPU."""
    H, HV, K, V = layer.H, layer.HV, layer.K, layer.V
    s = x + residual
    qkv = layer_reference.norm(s, p["norm"], 1e-6) @ p["w_in"].t()
    cos, sin, at = layer.cos.double().cpu(), layer.sin.double().cpu(), places(lens).cpu()
    q, k = (ref.heads(qkv[:, i * H * K:(i + 1) * H * K].unflatten(-1, (H, K)), p[w], cos, sin, at, False)
            for i, w in ((0, "norm_q"), (1, "norm_k")))
    v = qkv[:, 2 * H * K:].unflatten(-1, (HV, V))
    o, _ = ref.attention(q, k, v, layer.decay.double().cpu(), v.new_zeros(len(lens), HV, K, V), lens, layer.scale)
    return layer_reference.norm(o, p["norm_o"], 1e-6).flatten(-2) @ p["w_out"].t(), s


def test_layer_against_the_definition(gdr):
    """fp32, so that matrix products in 64 bits and in 32 differ by a few roundings of their terms."""
    lens = [40, 1, 0, 23]
    layer = LinearAttentionLayer(width=48, heads=2, value_heads=4, K=12, V=20, rotated=8, dtype=F32)
    x, residual = batch(layer, 64)
    cu, at = layer_reference.cu_of(lens, "cuda"), places(lens)[None]
    out, res, _, saved = layer.prefill(x, residual, at, cu_seqlens=cu)
    g = torch.Generator().manual_seed(4)
    dout, ds = (torch.randn(1, 64, 48, generator=g).cuda() for _ in range(2))
    dx, grads = layer.backward(saved, dout, ds)
    leaves = {k: v.double().cpu().requires_grad_() for k, v in layer.p.items()}
    lx = x[0].double().cpu().requires_grad_()
    want_out, want_res = reference_layer(layer, leaves, lx, residual[0].double().cpu(), lens)
    loss = (want_out * dout[0].double().cpu()).sum() + (want_res * ds[0].double().cpu()).sum()
    want = torch.autograd.grad(loss, [lx, *leaves.values()])
    # each of the layer's six stages hands on its own roundings: six times one operator's bound
    n = 6 * 6 * 64
    ref.close(out[0], want_out, F32, n, "out")
    ref.close(dx[0], want[0], F32, n, "dx")
    for k, w in zip(leaves, want[1:]):
        ref.close(grads[k], w, F32, n, k)


def test_decode_continues_a_prefill(gdr):
    """The states that a prefill leaves, moved to slots, carry on as the longer prompt does; a padding row between."""
    lens, more = [70, 5, 130], 3
    layer = LinearAttentionLayer(width=64, heads=2, value_heads=2, K=32, V=48, rotated=32, dtype=F32)
    x, residual = batch(layer, sum(lens) + more * len(lens), seed=1)
    cut = [n + more for n in lens]
    whole, _, _, _ = layer.prefill(x, residual, places(cut)[None], cu_seqlens=layer_reference.cu_of(cut, "cuda"))
    first = torch.cat([torch.arange(i, j - more) for _, i, j in layer_reference.spans(cut)]).cuda()
    _, _, st, _ = layer.prefill(x[:, first], residual[:, first], places(lens)[None],
                                cu_seqlens=layer_reference.cu_of(lens, "cuda"))
    pool = layer.empty_states(7)
    slots = torch.tensor([5, 0, -1, 3], dtype=torch.int32, device="cuda")
    real = torch.tensor([0, 1, 3], device="cuda")
    pool[slots[real].long()] = st
    for t in range(more):
        at = torch.tensor([j - more + t for _, i, j in layer_reference.spans(cut)], device="cuda")
        rows = [torch.full((4, 64), float("nan"), device="cuda") for _ in range(2)]
        rows[0][real], rows[1][real] = x[0, at], residual[0, at]
        pos = torch.tensor([lens[0] + t, lens[1] + t, -1, lens[2] + t], device="cuda")
        y, _ = layer.step(*rows, pos, pool, slots)
        ref.close(y[real], whole[0, at], F32, 6 * 6 * 140, "y")
    assert gdr.device_status() == 0


def test_prefill_and_training_step_in_a_graph(gdr):
    """bf16: captured calls, of which two captures share the library's workspaces, give the eager calls' bits."""
    layer = LinearAttentionLayer()
    lens = [200, 3, 900]
    cu, at = layer_reference.cu_of(lens, "cuda"), places(lens)[None]
    x, residual = batch(layer, sum(lens), seed=2)
    dout, ds = batch(layer, sum(lens), seed=3)

    def all_of(x, residual):
        out, res, st, saved = layer.prefill(x, residual, at, cu_seqlens=cu)
        dx, grads = layer.backward(saved, dout, ds)
        return [out, res, st, dx, *grads.values()]
    want = all_of(x, residual)
    torch.cuda.synchronize()
    fixed = [[torch.zeros_like(x), torch.zeros_like(residual)] for _ in range(2)]
    graphs, got = [], []
    for f in fixed:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(all_of(*f))
    fixed[0][0].copy_(x), fixed[0][1].copy_(residual)
    fixed[1][0].copy_(residual), fixed[1][1].copy_(x)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got[0], all_of(residual, x)):
        assert torch.equal(a, b)
    for a, b in zip(all_of(residual, x), got[1]):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = all_of(x, residual)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_two_calls_at_once(gdr):
    """On two streams: each call has its own workspace."""
    lens = [2500]
    p, q = (ref.attention_inputs(lens, 1, 2, 128, 128, BF16, seed=s, ) for s in (1, 2))
    p, q = ({k: v.cuda() for k, v in d.items()} for d in (p, q))

    def call(d):
        return gdr.la_fwd(d["q"][None], d["k"][None], d["v"][None], d["g"], h0=d["h0"])
    want = [call(p), call(q)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, d in zip(streams, (p, q)):
            with torch.cuda.stream(s):
                got.append(call(d))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[70], [2500, 40]], ids=str)
def test_unaligned_states(gdr, dtype, lens):
    """h0, dht and a pool of states one element past a 16-byte border: the aligned call's results."""
    p = {k: v.cuda() for k, v in ref.attention_inputs(lens, 1, 1, 64, 64, dtype, seed=4).items()}
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    cu = layer_reference.cu_of(lens, "cuda")
    args = (p["q"][None], p["k"][None], p["v"][None], p["g"])
    assert off(p["h0"]).data_ptr() % 16
    a = gdr.la_fwd(*args, h0=p["h0"], cu_seqlens=cu) + gdr.la_bwd(*args, p["do"][None], h0=p["h0"], dht=p["dht"],
                                                                  cu_seqlens=cu)
    b = gdr.la_fwd(*args, h0=off(p["h0"]), cu_seqlens=cu) + gdr.la_bwd(*args, p["do"][None], h0=off(p["h0"]),
                                                                       dht=off(p["dht"]), cu_seqlens=cu)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    rows = len(lens)
    s, t = p["h0"].clone(), off(p["h0"])
    u = gdr.la_step(p["q"][:rows], p["k"][:rows], p["v"][:rows], p["g"], s)
    v = gdr.la_step(p["q"][:rows], p["k"][:rows], p["v"][:rows], p["g"], t)
    ref.close(v, u.double(), dtype, 1)
    ref.close(t, s.double(), F32, 1)


def test_offsets_past_32_bits(gdr):
    """Rows 2^20 elements apart, 4200 tokens: byte offsets past 2^32 and element offsets past 2^31."""
    T, ld, K = 4200, 2 ** 20, 64
    wide = torch.zeros(T * ld, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    small = {k: torch.randn(1, T, 1, K, generator=g, device="cuda").to(BF16) for k in ("q", "k", "v", "do")}
    far = {}
    for i, (k, t) in enumerate(small.items()):
        far[k] = wide.as_strided((1, T, 1, K), (T * ld, ld, K, 1), 64 * i)
        far[k].copy_(t)
    decay = torch.tensor([-0.01], device="cuda")
    for a, b in zip(gdr.la_fwd(small["q"], small["k"], small["v"], decay), gdr.la_fwd(far["q"], far["k"], far["v"], decay)):
        assert torch.equal(a, b)
    for a, b in zip(gdr.la_bwd(*[small[k] for k in ("q", "k", "v")], decay, small["do"]),
                    gdr.la_bwd(*[far[k] for k in ("q", "k", "v")], decay, far["do"])):
        assert torch.equal(a, b)
    w = torch.ones(K, dtype=BF16, device="cuda")
    cos, sin = gdr.rotation_table(T, K)
    kw = dict(cos=cos, sin=sin, positions=torch.arange(T, device="cuda")[None])
    for a, b in zip(gdr.qk_norm_fwd(small["q"], small["k"], w, w, **kw), gdr.qk_norm_fwd(far["q"], far["k"], w, w, **kw)):
        assert torch.equal(a, b)
    for a, b in zip(gdr.qk_norm_bwd(small["do"], small["v"], small["q"], small["k"], w, w, **kw),
                    gdr.qk_norm_bwd(far["do"], far["v"], far["q"], far["k"], w, w, **kw)):
        assert torch.equal(a, b)


def test_state_pool_past_32_bits(gdr):
    """A pool of 2^31 + elements: the last slot's state lies past 32-bit offsets."""
    P, HV, K = 4100, 32, 128
    pool = torch.zeros(P, HV, K, K, device="cuda")  # 8.6 GB
    p = {k: v.cuda() for k, v in ref.attention_inputs([2], HV, HV, K, K, BF16, seed=7).items()}
    state = torch.randn(2, HV, K, K, device="cuda")
    slots = torch.tensor([P - 1, 4097], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    want = gdr.la_step(p["q"], p["k"], p["v"], p["g"], state)
    got = gdr.la_step(p["q"], p["k"], p["v"], p["g"], pool, slots=slots)
    assert torch.equal(got, want) and torch.equal(pool[slots.long()], state)
    assert not pool[:4097].any()


def test_example_runs(gdr, capsys):
    main()
    assert "step 4 loss" in capsys.readouterr().out
