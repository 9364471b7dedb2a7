"""Cases and plain forms of the operators around a recurrent layer: the
root-mean-square norm with the residual's addition (and an 8-bit output with
scales), the short causal convolution, and the selective state space scan;
each in the directions that serving and training use.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the calls
a user makes of chunked_gated_delta_08_gb300.  ``exact`` evaluates the same
definitions token by token in 64 bits.

Definitions (per sequence; t counts its tokens)
  norm   s = round(x + r);  y = s / sqrt(mean(s^2) + eps) * w;
         8 bits: scale = amax(y) / 448 over the row or over 128 columns, y8 = e4m3(y * (448 / amax(y)))
  conv   y_t = act(bias + sum_j w[:, j] x_{t - W + 1 + j}), x_{-1}, x_{-2}, .. from the state
  scan   D_t = softplus(dt_t + dt_bias);  h_t = exp(D_t A) h_{t-1} + D_t x_t B_t;
         y_t = (C_t . h_t + d x_t) * silu(z_t)
"""
import math

import torch

own = False

EPS = 1e-6
FP8_MAX = 448.0
GROUP = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases
def _norm(name, op, M, E, dtype, residual, quant):
    return {"name": name, "op": op, "M": M, "E": E, "dtype": dtype, "residual": residual, "quant": quant}


def _conv(name, op, lens, E, W, dtype, bias):
    return {"name": name, "op": op, "lens": lens, "E": E, "W": W, "dtype": dtype, "bias": bias}


def _scan(name, op, lens, E, S, G, dtype, gate):
    return {"name": name, "op": op, "lens": lens, "E": E, "S": S, "G": G, "dtype": dtype, "gate": gate}


def listed():
    return [
        # one decode step of 16 requests: the layer's first operation, a few hundred KB
        _norm("norm decode 16x4096", "norm_fwd", 16, 4096, "bf16", "bf16", "none"),
        # a packed prompt on its way into an 8-bit projection
        _norm("norm fp8 16384x4096", "norm_fwd", 16384, 4096, "bf16", "bf16", "group"),
        # a training step that keeps its residual stream in fp32
        _norm("norm bwd 16384x4096", "norm_bwd", 16384, 4096, "bf16", "fp32", "none"),
        # one token for each of 256 running requests, states in a pool of slots
        _conv("conv step 256x4096", "conv_step", "256", 4096, 4, "bf16", True),
        # a packed prefill of requests of different lengths, some of a single token
        _conv("conv packed 16384x4096", "conv_fwd", "5000,1,3,4096,777,6011,496", 4096, 4, "bf16", True),
        # a training step on four sequences
        _conv("conv bwd 4x4096x4096", "conv_bwd", "4096x4", 4096, 4, "bf16", True),
        # the smallest call: one request, one token
        _scan("scan step 1x4096", "scan_step", "1", 4096, 16, 1, "bf16", True),
        # one token for each of 256 running requests: the states are read and written once
        _scan("scan step 256x4096", "scan_step", "256", 4096, 16, 1, "bf16", True),
        # a packed prefill of requests of different lengths
        _scan("scan packed 16384x4096", "scan_fwd", "5000,1,3,4096,777,6011,496", 4096, 16, 1, "bf16", True),
        # one long prompt: few rows, a long axis
        _scan("scan long 32768x1024", "scan_fwd", "32768", 1024, 16, 1, "bf16", True),
        # a training step on four sequences
        _scan("scan bwd 4x4096x2048", "scan_bwd", "4096x4", 2048, 16, 1, "bf16", True),
        # a ragged fp32 training batch with odd widths and two groups of B and C
        _scan("scan bwd odd 1501x1000", "scan_bwd", "700,1,0,800", 1000, 12, 2, "fp32", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lens(rng, total):
    """A dense batch "LxB" or packed lengths (zero and one among them) of about `total` tokens."""
    if rng.random() < 0.4:
        b = rng.choice([1, 2, 3, 4])
        return "%dx%d" % (max(1, total // b), b)
    lens, left = [], total
    for _ in range(rng.randint(2, 9)):
        n = min(left, rng.choice([0, 1, rng.randint(0, left)]))
        lens.append(n)
        left -= n
    lens.append(left)
    rng.shuffle(lens)
    return ",".join(str(n) for n in lens)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd",
                     "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    E = rng.choice([64 * rng.randint(1, 64), _log_int(rng, 48, 4096)])
    if op.startswith("norm"):
        residual = rng.choice(["none", dtype, "fp32"]) if op == "norm_fwd" else rng.choice([dtype, "fp32"])
        quant = rng.choice(["none", "row", "group"]) if op == "norm_fwd" else "none"
        c = _norm("", op, _log_int(rng, 1, 16384), E, dtype, residual, quant)
        del c["name"]
        return c
    step = op.endswith("step")
    if op.startswith("conv"):
        lens = str(_log_int(rng, 1, 256)) if step else _draw_lens(rng, _log_int(rng, 1, 16384))
        c = _conv("", op, lens, E, rng.choice([2, 3, 4, 4, 4]), dtype, rng.random() < 0.7)
    else:
        S = rng.choice([16, 16, 16, 1, 4, 12, 32, 64])
        G = rng.choice([1, 1, 2])
        E += E % G
        most = 16384 * 2048 * 16 if op == "scan_bwd" else 16384 * 4096 * 16
        lens = str(_log_int(rng, 1, 256)) if step else _draw_lens(rng, _log_int(rng, 1, min(16384, most // (E * S))))
        c = _scan("", op, lens, E, S, G, dtype, rng.random() < 0.8)
    del c["name"]
    return c


def _lengths(lens):
    if "x" in lens:
        n, b = lens.split("x")
        return [int(n)] * int(b), True
    v = [int(n) for n in lens.split(",")]
    return v, len(v) == 1


# --------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, mul=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * mul).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    op, E = case["op"], case["E"]
    p = {"case": case, "op": op}
    if op.startswith("norm"):
        M = case["M"]
        p["weight"] = randn(E, mul=0.1).add_(1.0).to(dt)
        rdt = DTYPES.get(case["residual"])
        if op == "norm_fwd":
            p["x"] = randn(M, E, dtype=dt)
            p["residual"] = None if rdt is None else randn(M, E, dtype=rdt, mul=3.0)
        else:
            p["s"] = randn(M, E, dtype=rdt, mul=3.0)
            p["dy"], p["ds"] = randn(M, E, dtype=dt), randn(M, E, dtype=rdt)
        return p
    lens, dense = _lengths(case["lens"])
    if op.endswith("step"):
        R = lens[0]
        pool = R + R // 4 + 1
        p["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:R].to(torch.int32)
        lead = (R,)
    else:
        N = len(lens)
        B, T = (N, lens[0]) if dense else (1, sum(lens))
        lead = (B, T)
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        p["cu"] = None if dense else torch.tensor(ends, dtype=torch.int64, device="cuda")
    # x and z (the gate) are the halves of one projection's output, as a layer has them
    xz = randn(*lead, 2 * E, dtype=dt)
    p["x"] = xz[..., :E]
    if op.startswith("conv"):
        W = case["W"]
        p["weight"] = randn(E, W, mul=W ** -0.5).to(dt)
        p["bias"] = randn(E, mul=0.1).to(dt) if case["bias"] else None
        if op == "conv_step":
            p["state"] = randn(pool, W - 1, E, dtype=dt)
        else:
            p["s0"] = randn(N, W - 1, E, dtype=dt)
        if op == "conv_bwd":
            p["dy"], p["dst"] = randn(*lead, E, dtype=dt), randn(N, W - 1, E, dtype=dt)
        return p
    S, G = case["S"], case["G"]
    # dt starts log-uniform in [1e-3, 1e-1] after the softplus, A at -1 .. -S: the usual initial values, perturbed
    d0 = torch.exp(rand(E) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    p["dt_bias"] = d0 + torch.log(-torch.expm1(-d0))
    p["a"] = -torch.arange(1, S + 1, device="cuda", dtype=torch.float32) * (0.5 + rand(E, S))
    p["d"] = randn(E, mul=0.1).add_(1.0)
    p["dt"] = randn(*lead, E, dtype=dt, mul=0.5)
    # B and C are parts of one small projection's output
    bc = randn(*lead, 2 * G * S, dtype=dt)
    p["b"], p["c"] = bc[..., :G * S].unflatten(-1, (G, S)), bc[..., G * S:].unflatten(-1, (G, S))
    p["z"] = xz[..., E:] if case["gate"] else None
    if op == "scan_step":
        p["state"] = randn(pool, E, S, mul=0.3)
    else:
        p["h0"] = randn(N, E, S, mul=0.3)
    if op == "scan_bwd":
        p["dy"], p["dht"] = randn(*lead, E, dtype=dt), randn(N, E, S)
    return p


# ----------------------------------------------------------------------------------------- plain forms
def _f(t):
    return None if t is None else t.float()


def _plain_norm_fwd(p):
    x, w, quant = p["x"], p["weight"].float(), p["case"]["quant"]
    s = None
    v = x.float()
    if p["residual"] is not None:
        s = (v + p["residual"].float()).to(p["residual"].dtype)
        v = s.float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w
    if quant == "none":
        return {"y": y.to(x.dtype), "s": s}
    M, E = y.shape
    width = E if quant == "row" else GROUP
    groups = -(-E // width)
    yg = torch.nn.functional.pad(y, (0, groups * width - E)).view(M, groups, width)
    amax = yg.abs().amax(-1, keepdim=True)
    amax = torch.where(amax == 0, FP8_MAX, amax)
    y8 = (yg * (FP8_MAX / amax)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    scale = (amax / FP8_MAX).view(M, groups)
    return {"y8": y8.view(M, -1)[:, :E].contiguous(), "scale": scale[:, 0] if quant == "row" else scale, "s": s}


def _plain_norm_bwd(p):
    v, w, dy = p["s"].float(), p["weight"].float(), p["dy"].float()
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    wd = w * dy
    g = p["ds"].float() + r * (wd - v * (r * r * (wd * v).mean(-1, keepdim=True)))
    return {"dx": g.to(p["dy"].dtype), "dres": g.to(p["s"].dtype), "dw": (dy * v * r).sum(0)}


def _rows(p):
    """Of each token: its sequence and its place there; of each sequence: its first token and length."""
    lead = p["x"].shape[:2]
    dev = p["x"].device
    if p["cu"] is None:
        cu = torch.arange(lead[0] + 1, device=dev) * lead[1]
    else:
        cu = p["cu"]
    M = lead[0] * lead[1]
    t = torch.arange(M, device=dev)
    seq = torch.bucketize(t, cu[1:], right=True)
    return seq, t - cu[seq], cu[:-1], cu[1:] - cu[:-1]


def _taps(p):
    """[M, W, E]: the W inputs under the filter at each token, earliest first; and the rows after the last tokens."""
    W = p["case"]["W"]
    x, s0 = p["x"].flatten(0, 1), p["s0"]
    seq, pos, first, lens = _rows(p)
    back = torch.arange(W - 1, -1, -1, device=x.device)
    at = pos[:, None] - back  # place in the sequence; negative: in the state
    rows = (first[seq][:, None] + at).clamp(min=0)
    old = s0[seq[:, None], (at + W - 1).clamp(max=W - 2)]
    taps = torch.where((at >= 0)[..., None], x[rows], old)
    at = lens[:, None] - torch.arange(W - 1, 0, -1, device=x.device)
    n = torch.arange(lens.numel(), device=x.device)[:, None]
    st = torch.where((at >= 0)[..., None], x[(first[:, None] + at).clamp(0, max(0, x.shape[0] - 1))],
                     s0[n, (at + W - 1).clamp(max=W - 2)])
    return taps, st


def _plain_conv_fwd(p):
    taps, st = _taps(p)
    pre = (taps.float() * p["weight"].float().t()).sum(1)
    if p["bias"] is not None:
        pre = pre + p["bias"].float()
    return {"y": (pre * torch.sigmoid(pre)).to(p["x"].dtype).view(p["x"].shape), "st": st}


def _plain_conv_bwd(p):
    W, w = p["case"]["W"], p["weight"].float()
    taps, _ = _taps(p)
    taps = taps.float()
    pre = (taps * w.t()).sum(1)
    if p["bias"] is not None:
        pre = pre + p["bias"].float()
    sg = torch.sigmoid(pre)
    g = p["dy"].flatten(0, 1).float() * sg * (1 + pre * (1 - sg))
    dw = (g[:, None] * taps).sum(0).t()
    # one long row of states and inputs of all sequences: W - 1 state rows before each sequence's tokens
    seq, pos, first, lens = _rows(p)
    N, E = lens.numel(), g.shape[1]
    start = first + torch.arange(N, device=g.device) * (W - 1)
    acc = torch.zeros(g.shape[0] + N * (W - 1), E, device=g.device)
    here = start[seq] + pos  # the earliest tap of a token
    put = here[:, None] + torch.arange(W, device=g.device)
    acc.index_add_(0, put.flatten(), (g[:, None] * w.t()).flatten(0, 1))
    tail = (start + lens)[:, None] + torch.arange(W - 1, device=g.device)
    acc.index_add_(0, tail.flatten(), p["dst"].float().flatten(0, 1))
    dt = p["x"].dtype
    return {"dx": acc[here + W - 1].to(dt).view(p["x"].shape), "dw": dw,
            "dbias": None if p["bias"] is None else g.sum(0),
            "ds0": acc[start[:, None] + torch.arange(W - 1, device=g.device)].to(dt)}


def _plain_conv_step(p):
    slots = p["slots"].long()
    taps = torch.cat([p["state"][slots], p["x"][:, None]], 1)
    pre = (taps.float() * p["weight"].float().t()).sum(1)
    if p["bias"] is not None:
        pre = pre + p["bias"].float()
    p["state"][slots] = taps[:, 1:]
    return {"y": (pre * torch.sigmoid(pre)).to(p["x"].dtype), "state": p["state"]}


def _affine_scan(a, u):
    """h_t = a_t h_{t-1} + u_t for all t at once, by doubling; both arguments are consumed."""
    k = 1
    while k < a.shape[0]:
        u[k:] += a[k:] * u[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return u


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _scan_terms(p):
    """delta [M, E], decay [M, E, S], B and C per channel [M, E, S], x [M, E] (fp32)."""
    E, G, S = p["case"]["E"], p["case"]["G"], p["case"]["S"]
    n = p["x"].dim() - 1
    x = p["x"].flatten(0, n - 1).float()
    v = p["dt"].flatten(0, n - 1).float() + p["dt_bias"]
    delta = _softplus(v)
    per = lambda t: t.flatten(0, n - 1).float()[:, :, None, :].expand(-1, G, E // G, S).reshape(-1, E, S)  # noqa: E731
    return x, v, delta, torch.exp(delta[..., None] * p["a"]), per(p["b"]), per(p["c"])


def _silu_gate(p, n):
    if p["z"] is None:
        return None, None
    z = p["z"].flatten(0, n).float()
    return z, torch.sigmoid(z)


def _scan_states(p, decay, u, first, lens):
    """h_t [M, E, S] and the state before each token, of all sequences."""
    start = first[lens > 0]
    h0 = p["h0"][lens > 0]
    a = decay.clone()
    a[start] = 0
    u = u.clone()
    u[start] += decay[start] * h0
    h = _affine_scan(a, u)
    prev = torch.cat([h[:1], h[:-1]])
    prev[start] = h0
    return h, prev


def _last(h, h0, first, lens):
    if h.shape[0] == 0:
        return h0.clone()
    end = h[(first + lens - 1).clamp(0, h.shape[0] - 1)]
    return torch.where((lens > 0)[:, None, None], end, h0)


def _plain_scan_fwd(p):
    x, _, delta, decay, b, c = _scan_terms(p)
    _, _, first, lens = _rows(p)
    h, _ = _scan_states(p, decay, (delta * x)[..., None] * b, first, lens)
    y = (h * c).sum(-1) + p["d"] * x
    z, sg = _silu_gate(p, 1)
    if z is not None:
        y = y * (z * sg)
    return {"y": y.to(p["x"].dtype).view(p["x"].shape), "ht": _last(h, p["h0"], first, lens)}


def _plain_scan_bwd(p):
    E, G, S = p["case"]["E"], p["case"]["G"], p["case"]["S"]
    x, v, delta, decay, b, c = _scan_terms(p)
    _, _, first, lens = _rows(p)
    h, prev = _scan_states(p, decay, (delta * x)[..., None] * b, first, lens)
    dy = p["dy"].flatten(0, 1).float()
    z, sg = _silu_gate(p, 1)
    dz = None
    if z is not None:
        dz = dy * ((h * c).sum(-1) + p["d"] * x) * (sg * (1 + z * (1 - sg)))
        dy = dy * (z * sg)
    # g_t = dL/dh_t = C_t dy_t + decay_{t+1} g_{t+1}, from the last token of each sequence back
    some = lens > 0
    end, start = (first + lens - 1)[some], first[some]
    back = torch.cat([decay[1:], torch.zeros_like(decay[:1])])
    back[end] = 0
    u = dy[..., None] * c
    u[end] += p["dht"][some]
    g = _affine_scan(back.flip(0), u.flip(0)).flip(0)
    dc = (dy[..., None] * h).view(-1, G, E // G, S).sum(2)
    da_t = g * prev * decay
    da = (da_t * delta[..., None]).sum(0)
    ddelta = (da_t * p["a"]).sum(-1)
    gb = (g * b).sum(-1)
    dx = p["d"] * dy + delta * gb
    ddelta = ddelta + x * gb
    db = (g * (delta * x)[..., None]).view(-1, G, E // G, S).sum(2)
    ddt = ddelta * torch.sigmoid(v)
    dh0 = p["dht"].clone()
    dh0[some] = decay[start] * g[start]
    dt, sh, gsh = p["x"].dtype, p["x"].shape, p["b"].shape
    return {"dx": dx.to(dt).view(sh), "ddt": ddt.to(dt).view(sh), "da": da, "db": db.to(dt).view(gsh),
            "dc": dc.to(dt).view(gsh), "dd": (dy * x).sum(0), "dz": None if z is None else dz.to(dt).view(sh),
            "ddt_bias": ddt.sum(0), "dh0": dh0}


def _plain_scan_step(p):
    slots = p["slots"].long()
    x, _, delta, decay, b, c = _scan_terms(p)
    h = decay * p["state"][slots] + (delta * x)[..., None] * b
    p["state"][slots] = h
    y = (h * c).sum(-1) + p["d"] * x
    z, sg = _silu_gate(p, 0)
    if z is not None:
        y = y * (z * sg)
    return {"y": y.to(p["x"].dtype), "state": p["state"]}


# ------------------------------------------------------------------------------------------- own calls
def _own(p):
    import chunked_gated_delta_08_gb300 as gdr
    op = p["op"]
    if op == "norm_fwd":
        quant = p["case"]["quant"]
        if quant == "none":
            y, s = gdr.norm_fwd(p["x"], p["weight"], p["residual"], eps=EPS)
            return {"y": y, "s": s}
        y8, scale, s = gdr.norm_fwd(p["x"], p["weight"], p["residual"], eps=EPS, quant=quant)
        return {"y8": y8, "scale": scale, "s": s}
    if op == "norm_bwd":
        dx, dres, dw = gdr.norm_bwd(p["dy"], p["s"], p["weight"], ds=p["ds"], eps=EPS)
        return {"dx": dx, "dres": dres, "dw": dw}
    if op == "conv_fwd":
        y, st = gdr.conv_fwd(p["x"], p["weight"], bias=p["bias"], s0=p["s0"], cu_seqlens=p["cu"])
        return {"y": y, "st": st}
    if op == "conv_bwd":
        dx, dw, dbias, ds0 = gdr.conv_bwd(p["x"], p["weight"], p["dy"], bias=p["bias"], s0=p["s0"], dst=p["dst"],
                                          cu_seqlens=p["cu"])
        return {"dx": dx, "dw": dw, "dbias": dbias, "ds0": ds0}
    if op == "conv_step":
        y = gdr.conv_step(p["x"], p["state"], p["weight"], bias=p["bias"], slots=p["slots"])
        return {"y": y, "state": p["state"]}
    if op == "scan_fwd":
        y, ht = gdr.ssm_fwd(p["x"], p["dt"], p["a"], p["b"], p["c"], d=p["d"], z=p["z"], dt_bias=p["dt_bias"],
                            h0=p["h0"], cu_seqlens=p["cu"])
        return {"y": y, "ht": ht}
    if op == "scan_bwd":
        got = gdr.ssm_bwd(p["x"], p["dt"], p["a"], p["b"], p["c"], p["dy"], d=p["d"], z=p["z"],
                          dt_bias=p["dt_bias"], h0=p["h0"], dht=p["dht"], cu_seqlens=p["cu"])
        return dict(zip(("dx", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh0"), got))
    y = gdr.ssm_step(p["x"], p["dt"], p["a"], p["b"], p["c"], p["state"], d=p["d"], z=p["z"], dt_bias=p["dt_bias"],
                     slots=p["slots"])
    return {"y": y, "state": p["state"]}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "conv_fwd": _plain_conv_fwd,
          "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step, "scan_fwd": _plain_scan_fwd,
          "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step}


def run(state):
    got = _own(state) if own else _PLAIN[state["op"]](state)
    return {k: v for k, v in got.items() if v is not None}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, E = case["op"], case["E"]
    el = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        M, rel = case["M"], {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
        if op == "norm_fwd":
            out = el if case["quant"] == "none" else 1
            scales = 0 if case["quant"] == "none" else 4 * M * (1 if case["quant"] == "row" else -(-E // GROUP))
            return {"bytes": M * E * (el + 2 * rel + out) + E * el + scales, "flops": M * E * 5}
        # where the two gradients have one type they are one tensor
        outs = el if rel == el else el + rel
        return {"bytes": M * E * (el + 2 * rel + outs) + E * (el + 4), "flops": M * E * 12}
    lens, _ = _lengths(case["lens"])
    step = op.endswith("step")
    M, N = (lens[0], lens[0]) if step else (sum(lens), len(lens))
    if op.startswith("conv"):
        W = case["W"]
        state, par = N * (W - 1) * E * el, E * (W + 1) * el
        if op == "conv_bwd":
            return {"bytes": 3 * M * E * el + 3 * state + par + 4 * E * (W + 1), "flops": M * E * (6 * W + 12)}
        return {"bytes": 2 * M * E * el + 2 * state + par, "flops": M * E * (2 * W + 5)}
    S, G = case["S"], case["G"]
    state, par, gate = 4 * N * E * S, 4 * E * (S + 2), 1 if case["gate"] else 0
    if op == "scan_bwd":
        return {"bytes": M * E * el * (5 + 2 * gate) + 4 * M * G * S * el + 3 * state + 2 * par,
                "flops": M * E * (24 * S + 30)}
    return {"bytes": M * E * el * (3 + gate) + 2 * M * G * S * el + 2 * state + par, "flops": M * E * (7 * S + 15)}


# ----------------------------------------------------------------------------------------------- exact
def _exact_norm(p):
    f64, w = torch.float64, p["weight"].double()
    if p["op"] == "norm_bwd":
        v, dy = p["s"].double(), p["dy"].double()
        n = v.shape[1]
        root = torch.sqrt((v * v).sum(1, keepdim=True) / n + EPS)
        unit = v / root
        t = dy * w
        g = p["ds"].double() + (t - unit * ((t * unit).sum(1, keepdim=True) / n)) / root
        return {"dx": g, "dres": g, "dw": (dy * unit).sum(0)}
    v, s = p["x"].double(), None
    if p["residual"] is not None:
        s = (v + p["residual"].double()).to(p["residual"].dtype)
        v = s.to(f64)
    y = v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS) * w
    s = None if s is None else s.to(f64)
    if p["case"]["quant"] == "none":
        return {"y": y, "s": s}
    width = y.shape[1] if p["case"]["quant"] == "row" else GROUP
    y8, scales = [], []
    for part in y.split(width, 1):
        top = part.abs().max(1, keepdim=True).values
        scale = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
        y8.append((part / scale).float().clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).to(f64))
        scales.append(scale)
    scale = torch.cat(scales, 1)
    return {"y8": torch.cat(y8, 1), "scale": scale[:, 0] if p["case"]["quant"] == "row" else scale, "s": s}


def _spans(p):
    lens, _ = _lengths(p["case"]["lens"])
    at = 0
    for n, length in enumerate(lens):
        yield n, at, at + length
        at += length


def _exact_conv(p):
    W, w = p["case"]["W"], p["weight"].double()
    bias = 0.0 if p["bias"] is None else p["bias"].double()
    if p["op"] == "conv_step":
        slots = p["slots"].long()
        old, x = p["state"].double(), p["x"].double()
        pre = x * w[:, W - 1] + bias
        for j in range(W - 1):
            pre = pre + old[slots, j] * w[:, j]
        new = old.clone()
        for j in range(W - 2):
            new[slots, j] = old[slots, j + 1]
        new[slots, W - 2] = x
        return {"y": pre / (1 + torch.exp(-pre)), "state": new}
    x = p["x"].flatten(0, 1).double()
    bwd = p["op"] == "conv_bwd"
    y, st, dx, ds0 = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros(w.shape[0], dtype=torch.float64, device=w.device)
    dy = p["dy"].flatten(0, 1).double() if bwd else None
    for n, i, j in _spans(p):
        full = torch.cat([p["s0"][n].double(), x[i:j]])
        pre = torch.zeros(j - i, x.shape[1], dtype=torch.float64, device=x.device) + bias
        for k in range(W):
            pre = pre + full[k:k + j - i] * w[:, k]
        if not bwd:
            y.append(pre / (1 + torch.exp(-pre)))
            st.append(full[full.shape[0] - (W - 1):])
            continue
        q = 1 / (1 + torch.exp(-pre))
        g = dy[i:j] * (q + pre * q * (1 - q))
        dfull = torch.zeros_like(full)
        dfull[full.shape[0] - (W - 1):] += p["dst"][n].double()
        for k in range(W):
            dfull[k:k + j - i] += g * w[:, k]
            dw[:, k] += (g * full[k:k + j - i]).sum(0)
        db += g.sum(0)
        dx.append(dfull[W - 1:])
        ds0.append(dfull[:W - 1])
    if not bwd:
        return {"y": torch.cat(y).view(p["x"].shape), "st": torch.stack(st)}
    return {"dx": torch.cat(dx).view(p["x"].shape), "dw": dw, "dbias": None if p["bias"] is None else db,
            "ds0": torch.stack(ds0)}


def _exact_scan(p):
    """Token by token, forwards and for the gradients backwards."""
    E, S, G = p["case"]["E"], p["case"]["S"], p["case"]["G"]
    op = p["op"]
    flat = (lambda t: t.double()) if op == "scan_step" else (lambda t: t.flatten(0, 1).double())
    A, d = p["a"].double(), p["d"].double()
    x, B, C = flat(p["x"]), flat(p["b"]), flat(p["c"])
    raw = flat(p["dt"]) + p["dt_bias"].double()
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    z = None if p["z"] is None else flat(p["z"])
    gate = 1.0 if z is None else z / (1 + torch.exp(-z))
    wide = lambda r: r.repeat_interleave(E // G, 0)  # noqa: E731  [G, S] -> [E, S]
    if op == "scan_step":
        new = p["state"].double()
        y = torch.empty_like(x)
        for r, slot in enumerate(p["slots"].tolist()):
            new[slot] = torch.exp(step[r][:, None] * A) * new[slot] + (step[r] * x[r])[:, None] * wide(B[r])
            y[r] = (new[slot] * wide(C[r])).sum(1) + d * x[r]
        return {"y": y * gate, "state": new}
    M = x.shape[0]
    pre = torch.empty_like(x)
    ht = p["h0"].double()
    if op == "scan_fwd":
        for n, i, j in _spans(p):
            h = ht[n]
            for t in range(i, j):
                h = torch.exp(step[t][:, None] * A) * h + (step[t] * x[t])[:, None] * wide(B[t])
                pre[t] = (h * wide(C[t])).sum(1)
            ht[n] = h
        return {"y": ((pre + d * x) * gate).view(p["x"].shape), "ht": ht}
    dy = flat(p["dy"])
    up = dy * gate
    dstep, dxs, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
    dB, dC, dh0 = torch.zeros_like(B), torch.zeros_like(C), p["dht"].double()
    for n, i, j in _spans(p):
        hs = [ht[n]]
        for t in range(i, j):
            hs.append(torch.exp(step[t][:, None] * A) * hs[-1] + (step[t] * x[t])[:, None] * wide(B[t]))
        g = dh0[n]
        for t in range(j - 1, i - 1, -1):
            h, before = hs[t - i + 1], hs[t - i]
            pre[t] = (h * wide(C[t])).sum(1)
            dC[t] = (up[t][:, None] * h).view(G, E // G, S).sum(1)
            g = g + up[t][:, None] * wide(C[t])
            gb = (g * wide(B[t])).sum(1)
            dB[t] = (g * (step[t] * x[t])[:, None]).view(G, E // G, S).sum(1)
            g = g * torch.exp(step[t][:, None] * A)
            q = g * before
            dA += q * step[t][:, None]
            dstep[t] = (q * A).sum(1) + x[t] * gb
            dxs[t] = step[t] * gb
        dh0[n] = g
        del hs
    ddt = dstep / (1 + torch.exp(-raw))
    dz = None
    if z is not None:
        q = 1 / (1 + torch.exp(-z))
        dz = (dy * (pre + d * x) * (q + z * q * (1 - q))).view(p["x"].shape)
    sh, gsh = p["x"].shape, p["b"].shape
    return {"dx": (dxs + d * up).view(sh), "ddt": ddt.view(sh), "da": dA, "db": dB.view(gsh), "dc": dC.view(gsh),
            "dd": (up * x).sum(0), "dz": dz, "ddt_bias": ddt.sum(0), "dh0": dh0}


def exact(case, seed):
    p = prepare(case, seed)
    got = (_exact_norm if p["op"].startswith("norm") else _exact_conv if p["op"].startswith("conv") else _exact_scan)(p)
    return {k: v for k, v in got.items() if v is not None}
