"""Cases and plain forms of linear attention with a decay for each head, and of
the norm of queries and keys for each head with the position rotation in the
same pass: prompts, single tokens with states in a pool of slots, and the
gradients of both.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the calls
a user makes of chunked_gated_delta_08_gb300.  ``exact`` evaluates the same
definitions in 64 bits, the attention token by token.

Definitions (per sequence; t counts its tokens; value head h reads the q and k
head h // (HV / H))
  attention  S_t = exp(g_h) S_{t-1} + k_t v_t^T;  o_t = scale * S_t^T q_t
  head norm  n = x / sqrt(mean(x^2) + eps) * w over the channels of one head, then the first 2 R channels are
             rotated by the angles of the token's position p: for the pair (a, b) = (n_i, n_{i+R}), or
             (n_{2i}, n_{2i+1}) where pairs are interleaved,  a' = a cos[p, i] - b sin[p, i],  b' = b cos + a sin
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64  # tokens in a chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases
def _head(name, op, M, H, HK, K, rot, style, dtype):
    return {"name": name, "op": op, "M": M, "H": H, "HK": HK, "K": K, "rot": rot, "style": style, "dtype": dtype}


def _attn(name, op, lens, H, HV, K, V, dtype):
    return {"name": name, "op": op, "lens": lens, "H": H, "HV": HV, "K": K, "V": V, "dtype": dtype}


def listed():
    return [
        # one decode step of 16 requests: 32 query and 8 key heads of one projection
        _head("heads decode 16x40x128", "head_fwd", 16, 32, 8, 128, 128, "half", "bf16"),
        # a packed prompt, whole heads rotated
        _head("heads prompt 16384x40x128", "head_fwd", 16384, 32, 8, 128, 128, "half", "bf16"),
        # a training step on heads of which a part is rotated, in neighbouring pairs
        _head("heads bwd 16384x40x128", "head_bwd", 16384, 32, 8, 128, 64, "interleaved", "bf16"),
        # the smallest call: one request, one token
        _attn("attn step 1x32x128", "attn_step", "1", 32, 32, 128, 128, "bf16"),
        # one token for each of 256 running requests: the states are read and written once
        _attn("attn step 256x32x128", "attn_step", "256", 32, 32, 128, 128, "bf16"),
        # the forward of a training step on four sequences
        _attn("attn 4x4096x32x128", "attn_fwd", "4096x4", 32, 32, 128, 128, "bf16"),
        # a packed prefill of requests of different lengths, value heads in groups
        _attn("attn packed 16384x32x128", "attn_fwd", "5000,1,3,4096,777,6011,496", 8, 32, 128, 128, "bf16"),
        # one long prompt and few heads: a long axis and little beside it
        _attn("attn long 32768x4x128", "attn_fwd", "32768", 4, 4, 128, 128, "bf16"),
        # small heads in fp32
        _attn("attn fp32 2x2048x8x64", "attn_fwd", "2048x2", 8, 8, 64, 64, "fp32"),
        # a training step on four sequences
        _attn("attn bwd 4x4096x32x128", "attn_bwd", "4096x4", 32, 32, 128, 128, "bf16"),
        # a ragged fp32 training batch with odd widths and two value heads to a q and k head
        _attn("attn bwd odd 1501x4x60x100", "attn_bwd", "700,1,0,800", 2, 4, 60, 100, "fp32"),
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
    op = rng.choice(["head_fwd", "head_bwd", "attn_fwd", "attn_fwd", "attn_bwd", "attn_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("head"):
        K = rng.choice([128, 128, 64, 256, 2 * _log_int(rng, 8, 128)])
        rot = rng.choice([K, K, K // 2 // 2 * 2, 0])
        HK = rng.choice([1, 2, 4, 8])
        c = _head("", op, _log_int(rng, 1, 16384), HK * rng.choice([1, 2, 4]), HK, K, rot,
                  rng.choice(["half", "interleaved"]), dtype)
        while c["M"] * (c["H"] + HK) * K > 16384 * 40 * 128:
            c["M"] //= 2
    else:
        K = rng.choice([128, 128, 64, 8 * rng.randint(2, 16), _log_int(rng, 16, 128)])
        V = rng.choice([K, K, 128, 64, _log_int(rng, 16, 128)])
        H = rng.choice([1, 2, 3, 4, 8, 16, 32])
        HV = H * rng.choice([1, 1, 1, 2, 4]) if H <= 8 else H
        if op == "attn_step":
            lens = str(_log_int(rng, 1, 256))
        else:
            most = min(16384, 16384 * 32 * 128 * 128 // (HV * K * V * (4 if dtype == "fp32" else 1)))
            lens = _draw_lens(rng, _log_int(rng, 1, most))
        c = _attn("", op, lens, H, HV, K, V, dtype)
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

    dt = DTYPES[case["dtype"]]
    op, K = case["op"], case["K"]
    p = {"case": case, "op": op}
    if op.startswith("head"):
        M, H, HK, R = case["M"], case["H"], case["HK"], case["rot"] // 2
        # queries and keys are parts of one projection's output, values beside them
        qkv = randn(M, (H + 2 * HK) * K, dtype=dt, mul=1.7)
        p["q"], p["k"] = qkv[:, :H * K].unflatten(-1, (H, K)), qkv[:, H * K:(H + HK) * K].unflatten(-1, (HK, K))
        p["wq"], p["wk"] = randn(K, mul=0.1).add_(1.0).to(dt), randn(K, mul=0.1).add_(1.0).to(dt)
        p["cos"] = p["sin"] = p["positions"] = None
        if R:
            # the table a program makes once, its angles in 64 bits
            freq = 10000.0 ** (-torch.arange(R, dtype=torch.float64, device="cuda") / R)
            angle = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * freq
            p["cos"], p["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
            p["positions"] = torch.randint(0, 32768, (M,), generator=gen, device="cuda")
        if op == "head_bwd":
            p["dyq"], p["dyk"] = randn(M, H, K, dtype=dt), randn(M, HK, K, dtype=dt)
        return p
    lens, dense = _lengths(case["lens"])
    H, HV, V = case["H"], case["HV"], case["V"]
    if op == "attn_step":
        R = lens[0]
        pool = R + R // 4 + 1
        p["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:R].to(torch.int32)
        p["state"] = randn(pool, HV, K, V)
        lead = (R,)
    else:
        N = len(lens)
        lead = (N, lens[0]) if dense else (1, sum(lens))
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        p["cu"] = None if dense else torch.tensor(ends, dtype=torch.int64, device="cuda")
        p["h0"] = randn(N, HV, K, V)
    p["q"], p["k"] = randn(*lead, H, K, dtype=dt), randn(*lead, H, K, dtype=dt)
    p["v"] = randn(*lead, HV, V, dtype=dt)
    # decays as layers have them, geometric over the heads from 2^-8 up, perturbed
    slope = torch.exp2(-8.0 * torch.arange(1, HV + 1, device="cuda") / HV)
    p["g"] = -slope * (0.5 + torch.rand(HV, generator=gen, device="cuda"))
    p["scale"] = K ** -0.5
    if op == "attn_bwd":
        p["do"], p["dht"] = randn(*lead, HV, V, dtype=dt), randn(N, HV, K, V)
    return p


# ----------------------------------------------------------------------------------------- plain forms
def _rotate(n, p, back=False):
    """n [M, heads, K] rotated by its token's angles; `back` by their negatives."""
    R = p["case"]["rot"] // 2
    if not R:
        return n
    cos, sin = p["cos"][p["positions"]][:, None], p["sin"][p["positions"]][:, None]
    sin = -sin if back else sin
    if p["case"]["style"] == "half":
        a, b, rest = n[..., :R], n[..., R:2 * R], n[..., 2 * R:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b, rest = n[..., :2 * R:2], n[..., 1:2 * R:2], n[..., 2 * R:]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_heads(p, x, w):
    v = x.float()
    return _rotate(v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float(), p).to(x.dtype)


def _plain_heads_back(p, x, w, dy):
    v, dn = x.float(), _rotate(dy.float(), p, back=True)
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    wd = w.float() * dn
    dx = r * (wd - v * (r * r * (wd * v).mean(-1, keepdim=True)))
    return dx.to(x.dtype), (dn * v * r).sum((0, 1))


def _plain_head_fwd(p):
    return {"yq": _plain_heads(p, p["q"], p["wq"]), "yk": _plain_heads(p, p["k"], p["wk"])}


def _plain_head_bwd(p):
    dq, dwq = _plain_heads_back(p, p["q"], p["wq"], p["dyq"])
    dk, dwk = _plain_heads_back(p, p["k"], p["wk"], p["dyk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _grid(p):
    """The chunk grid: the flat token at each place [NC, CHUNK] (the count of tokens: nothing there), each chunk's
    sequence, whether it is its sequence's first and last, and its count of tokens."""
    B, T = p["v"].shape[:2]
    dev = p["v"].device
    cu = torch.arange(B + 1, device=dev) * T if p["cu"] is None else p["cu"]
    lens = cu[1:] - cu[:-1]
    chunks = (lens + CHUNK - 1) // CHUNK
    first = torch.cumsum(chunks, 0) - chunks
    NC = int(sum(-(-n // CHUNK) for n in _lengths(p["case"]["lens"])[0]))
    c = torch.arange(NC, device=dev)
    seq = torch.bucketize(c, first + chunks, right=True)
    at = (c - first[seq])[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    rows = torch.where(at < lens[seq][:, None], cu[seq][:, None] + at, B * T)
    count = (lens[seq] - (c - first[seq]) * CHUNK).clamp(max=CHUNK)
    return rows, seq, c == first[seq], c == first[seq] + chunks[seq] - 1, count, lens


def _chunked(t, rows, group=1):
    """[B, T, heads, D] -> [NC, heads * group, CHUNK, D] in fp32, zeros where there is no token."""
    t = torch.cat([t.flatten(0, 1).float(), torch.zeros_like(t.flatten(0, 1)[:1], dtype=torch.float32)])
    return t[rows].transpose(1, 2).repeat_interleave(group, 1)


def _power(g, n):
    """exp(g n) [.., heads] of whole numbers n, the exponents in 64 bits."""
    return torch.exp(g.double() * n[..., None]).float()


def _carry(a, u):
    """s_c = a_c s_{c-1} + u_c along the first axis by doubling; both are consumed."""
    k = 1
    while k < a.shape[0]:
        u[k:] += a[k:] * u[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return u


def _states(p, a, b, left, entering, some, grid, back):
    """States [NC, HV, Ka, Vb] before each chunk (behind it, going back), and the last of each sequence: of products
    a^T b of rows `left` factors [NC, HV, CHUNK], from `entering` [N, HV, Ka, Vb]."""
    rows, seq, head, tail, count, lens = grid
    u = (a * left[..., None]).transpose(-1, -2) @ b
    decay = _power(p["g"], count)[..., None, None]
    start, end = (tail, head) if back else (head, tail)
    if back:
        u, decay, seq, start, end = u.flip(0), decay.flip(0), seq.flip(0), start.flip(0), end.flip(0)
    begin = torch.where(start[:, None, None, None], entering[seq], torch.zeros_like(u[:1]))
    after = _carry(torch.where(start[:, None, None, None], torch.zeros_like(decay), decay), u + decay * begin)
    before = torch.where(start[:, None, None, None], begin, torch.cat([torch.zeros_like(after[:1]), after[:-1]]))
    out = entering.clone()
    out[some] = after[end] if not back else after[end].flip(0)
    return (before.flip(0) if back else before), out


def _factors(p, grid):
    """exp(g |i - j|) [HV, CHUNK, CHUNK]; exp(g (i + 1)) [HV, CHUNK]; exp(g (count - 1 - i)) and exp(g (count - i - 1))
    [NC, HV, CHUNK] (zero behind the count)."""
    i = torch.arange(CHUNK, device=p["g"].device)
    near = _power(p["g"], (i[:, None] - i).abs()).permute(2, 0, 1)
    left = grid[4][:, None] - 1 - i
    rest = torch.where((left >= 0)[..., None], _power(p["g"], left.clamp(min=0)), 0.0).transpose(1, 2)
    return near, _power(p["g"], i + 1).t(), rest


def _flat(t, rows, like, dtype, group=1):
    """[NC, HV, CHUNK, D] -> [B, T, HV / group, D] like `like`, summed over groups of heads."""
    t = t.transpose(1, 2).unflatten(2, (-1, group)).sum(3)
    out = torch.empty(like.shape[0] * like.shape[1] + 1, *t.shape[2:], device=t.device)
    out[rows] = t
    return out[:-1].view(*like.shape[:2], *t.shape[2:]).to(dtype)


def _plain_attn_fwd(p):
    grid = _grid(p)
    rows, group = grid[0], p["case"]["HV"] // p["case"]["H"]
    q, k, v = _chunked(p["q"], rows, group), _chunked(p["k"], rows, group), _chunked(p["v"], rows)
    near, up, rest = _factors(p, grid)
    before, ht = _states(p, k, v, rest, p["h0"], grid[5] > 0, grid, False)
    o = ((q @ k.transpose(-1, -2)) * near.tril()) @ v + (q * up[..., None]) @ before
    return {"o": _flat(o * p["scale"], rows, p["v"], p["v"].dtype), "ht": ht}


def _plain_attn_bwd(p):
    grid = _grid(p)
    rows, group = grid[0], p["case"]["HV"] // p["case"]["H"]
    q, k, v = _chunked(p["q"], rows, group), _chunked(p["k"], rows, group), _chunked(p["v"], rows)
    do = _chunked(p["do"], rows) * p["scale"]
    near, up, rest = _factors(p, grid)
    before, _ = _states(p, k, v, rest, p["h0"], grid[5] > 0, grid, False)
    there = grid[0] < p["v"].shape[0] * p["v"].shape[1]
    # the gradient of the state behind each chunk; a query i tokens in passes i + 1 decays on its way to the front
    behind, dh0 = _states(p, q, do, up * there[:, None], p["dht"], grid[5] > 0, grid, True)
    pair = (do @ v.transpose(-1, -2)) * near.tril()
    score = (q @ k.transpose(-1, -2)) * near.tril()
    dq = pair @ k + (do * up[..., None]) @ before.transpose(-1, -2)
    dk = pair.transpose(-1, -2) @ q + (v * rest[..., None]) @ behind.transpose(-1, -2)
    dv = score.transpose(-1, -2) @ do + (k * rest[..., None]) @ behind
    return {"dq": _flat(dq, rows, p["q"], p["q"].dtype, group), "dk": _flat(dk, rows, p["k"], p["k"].dtype, group),
            "dv": _flat(dv, rows, p["v"], p["v"].dtype), "dh0": dh0}


def _plain_attn_step(p):
    slots, group = p["slots"].long(), p["case"]["HV"] // p["case"]["H"]
    q, k = (p[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    s = torch.exp(p["g"])[:, None, None] * p["state"][slots] + k[..., None] * p["v"].float()[:, :, None]
    p["state"][slots] = s
    return {"o": ((q[..., None] * s).sum(2) * p["scale"]).to(p["v"].dtype), "state": p["state"]}


# ------------------------------------------------------------------------------------------- own calls
def _own(p):
    import chunked_gated_delta_08_gb300 as gdr
    op = p["op"]
    if op.startswith("head"):
        kw = dict(cos=p["cos"], sin=p["sin"], positions=p["positions"], eps=EPS,
                  interleaved=p["case"]["style"] == "interleaved")
        if op == "head_fwd":
            return dict(zip(("yq", "yk"), gdr.qk_norm_fwd(p["q"], p["k"], p["wq"], p["wk"], **kw)))
        got = gdr.qk_norm_bwd(p["dyq"], p["dyk"], p["q"], p["k"], p["wq"], p["wk"], **kw)
        return dict(zip(("dq", "dk", "dwq", "dwk"), got))
    if op == "attn_fwd":
        o, ht = gdr.la_fwd(p["q"], p["k"], p["v"], p["g"], h0=p["h0"], cu_seqlens=p["cu"], scale=p["scale"])
        return {"o": o, "ht": ht}
    if op == "attn_bwd":
        got = gdr.la_bwd(p["q"], p["k"], p["v"], p["g"], p["do"], h0=p["h0"], dht=p["dht"], cu_seqlens=p["cu"],
                         scale=p["scale"])
        return dict(zip(("dq", "dk", "dv", "dh0"), got))
    o = gdr.la_step(p["q"], p["k"], p["v"], p["g"], p["state"], slots=p["slots"], scale=p["scale"])
    return {"o": o, "state": p["state"]}


_PLAIN = {"head_fwd": _plain_head_fwd, "head_bwd": _plain_head_bwd, "attn_fwd": _plain_attn_fwd,
          "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, K = case["op"], case["K"]
    el = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("head"):
        n = case["M"] * (case["H"] + case["HK"]) * K
        # each position's cosines and sines, once; of the weights and their gradients next to nothing
        table = case["M"] * (case["rot"] * 4 + 8) if case["rot"] else 0
        if op == "head_fwd":
            return {"bytes": 2 * n * el + table + 2 * K * el, "flops": 8 * n}
        return {"bytes": 3 * n * el + table + 2 * K * (el + 4), "flops": 18 * n}
    lens, _ = _lengths(case["lens"])
    step = op == "attn_step"
    M, N = (lens[0], lens[0]) if step else (sum(lens), len(lens))
    H, HV, V = case["H"], case["HV"], case["V"]
    state, qk, vo = 4 * N * HV * K * V, M * H * K * el, M * HV * V * el
    if op == "attn_bwd":
        return {"bytes": 4 * qk + 3 * vo + 3 * state, "flops": 10 * M * HV * K * V}
    return {"bytes": 2 * qk + 2 * vo + 2 * state, "flops": 4 * M * HV * K * V}


# ----------------------------------------------------------------------------------------------- exact
def _exact_heads(p):
    R, bwd = p["case"]["rot"] // 2, p["op"] == "head_bwd"
    half = p["case"]["style"] == "half"
    ia = torch.arange(R, device="cuda") if half else 2 * torch.arange(R, device="cuda")
    ib = ia + (R if half else 1)
    if R:
        c, s = (p[n].double()[p["positions"]].unsqueeze(1) for n in ("cos", "sin"))
    out = {}
    for n in ("q", "k"):
        x, w = p[n].double(), p["w" + n].double()
        root = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        unit = x / root
        if not bwd:
            y = unit * w
            if R:
                a, b = y[..., ia], y[..., ib]
                y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
            out["y" + n] = y
            continue
        t = p["dy" + n].double()
        if R:
            a, b = t[..., ia], t[..., ib]
            t[..., ia], t[..., ib] = a * c + b * s, b * c - a * s
        out["dw" + n] = (t * unit).sum((0, 1))
        t = t * w
        out["d" + n] = (t - unit * (t * unit).mean(-1, keepdim=True)) / root
    return {k: out[k] for k in (("dq", "dk", "dwq", "dwk") if bwd else ("yq", "yk"))}


def _exact_attn(p):
    """Token by token: the states forwards, their gradients backwards; a dense batch side by side."""
    H, HV = p["case"]["H"], p["case"]["HV"]
    f = torch.exp(p["g"].double())[:, None, None]
    q, k, v = p["q"].double(), p["k"].double(), p["v"].double()
    wide = lambda t: t.repeat_interleave(HV // H, -2)  # noqa: E731
    if p["op"] == "attn_step":
        new, o = p["state"].double(), torch.empty_like(v)
        for r, slot in enumerate(p["slots"].tolist()):
            new[slot] = f * new[slot] + wide(k[r])[:, :, None] * v[r][:, None]
            o[r] = torch.einsum("hk,hkv->hv", wide(q[r]), new[slot]) * p["scale"]
        return {"o": o, "state": new}
    lens, dense = _lengths(p["case"]["lens"])
    runs, at = [], 0
    if dense:
        runs = [(slice(None), slice(None), 0, lens[0])]
    else:
        for n, length in enumerate(lens):
            runs.append((slice(n, n + 1), slice(0, 1), at, at + length))
            at += length
    bwd = p["op"] == "attn_bwd"
    last, o, dq, dk, dv = p["h0"].double(), torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), \
        torch.zeros_like(v)
    do = p["do"].double() * p["scale"] if bwd else None
    dh0 = p["dht"].double() if bwd else None
    narrow = lambda t: t.unflatten(-2, (H, HV // H)).sum(-2)  # noqa: E731
    for n, b, i, j in runs:
        s = last[n]
        for t in range(i, j):
            s = f * s + wide(k[b, t])[..., None] * v[b, t][..., None, :]
            if bwd:
                dq[b, t] = narrow((s @ do[b, t][..., None])[..., 0])
            else:
                o[b, t] = (wide(q[b, t])[..., None, :] @ s)[..., 0, :] * p["scale"]
        last[n] = s
        if bwd:
            r = dh0[n]
            for t in range(j - 1, i - 1, -1):
                r = r + wide(q[b, t])[..., None] * do[b, t][..., None, :]
                dk[b, t] = narrow((r @ v[b, t][..., None])[..., 0])
                dv[b, t] = (wide(k[b, t])[..., None, :] @ r)[..., 0, :]
                r = f * r
            dh0[n] = r
    return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0} if bwd else {"o": o, "ht": last}


def exact(case, seed):
    p = prepare(case, seed)
    return _exact_heads(p) if p["op"].startswith("head") else _exact_attn(p)
