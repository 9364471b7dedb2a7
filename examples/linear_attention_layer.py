"""A linear attention layer built from the library's operators: norm with the
residual's addition, one projection to queries, keys and values, norm and
rotation of queries and keys, linear attention with a decay for each head, norm
of each head's output, output projection.  One class serves a packed prefill,
single-token decode with states in a pool of slots, and a training step.

    python examples/linear_attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_08_gb300 as gdr  # noqa: E402


class LinearAttentionLayer:
    """Parameters as plain tensors; ``heads`` query and key heads, ``value_heads`` a multiple of them."""

    def __init__(self, width=256, heads=4, value_heads=8, K=64, V=64, rotated=32, positions=4096, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def randn(*shape, k):
            return (torch.randn(*shape, generator=g) * k).to(device=device, dtype=dtype)

        self.H, self.HV, self.K, self.V, self.dtype, self.device = heads, value_heads, K, V, dtype, device
        self.scale = K ** -0.5
        self.p = {
            "norm": torch.ones(width, dtype=dtype, device=device),
            "w_in": randn(2 * heads * K + value_heads * V, width, k=width ** -0.5),
            "norm_q": torch.ones(K, dtype=dtype, device=device),
            "norm_k": torch.ones(K, dtype=dtype, device=device),
            "norm_o": torch.ones(V, dtype=dtype, device=device),
            "w_out": randn(width, value_heads * V, k=(value_heads * V) ** -0.5),
        }
        # constants of the layer: decays, slow and fast heads side by side, and the rotation's table
        self.decay = -torch.exp2(-8.0 * torch.arange(1, value_heads + 1, device=device) / value_heads)
        self.cos, self.sin = gdr.rotation_table(positions, rotated, device=device)

    def empty_states(self, n):
        """States of n sequences, or slots."""
        return torch.zeros(n, self.HV, self.K, self.V, device=self.device)

    def _project(self, n, positions):
        """q and k normed and turned; v, like the raw q and k, stays a part of the one projection."""
        hk = self.H * self.K
        qkv = n @ self.p["w_in"].t()
        q, k = (qkv[..., i:i + hk].unflatten(-1, (self.H, self.K)) for i in (0, hk))
        v = qkv[..., 2 * hk:].unflatten(-1, (self.HV, self.V))
        qn, kn = gdr.qk_norm_fwd(q, k, self.p["norm_q"], self.p["norm_k"], cos=self.cos, sin=self.sin,
                                 positions=positions)
        return q, k, qn, kn, v

    def prefill(self, x, residual, positions, states=None, cu_seqlens=None):
        """x, residual [B, T, width] (packed: [1, T, width]) -> output, new residual, states, what backward needs."""
        p = self.p
        n, s = gdr.norm_fwd(x, p["norm"], residual)
        q, k, qn, kn, v = self._project(n, positions)
        o, st = gdr.la_fwd(qn, kn, v, self.decay, h0=states, cu_seqlens=cu_seqlens, scale=self.scale)
        on, _ = gdr.norm_fwd(o, p["norm_o"])
        return on.flatten(-2) @ p["w_out"].t(), s, st, (s, n, q, k, qn, kn, v, o, on, positions, states, cu_seqlens)

    def step(self, x, residual, positions, states, slots):
        """One token of each running sequence: x, residual [R, width]; its state is updated in its slot."""
        p = self.p
        n, s = gdr.norm_fwd(x, p["norm"], residual)
        _, _, qn, kn, v = self._project(n, positions)
        o = gdr.la_step(qn, kn, v, self.decay, states, slots=slots, scale=self.scale)
        on, _ = gdr.norm_fwd(o, p["norm_o"])
        return on.flatten(-2) @ p["w_out"].t(), s

    def backward(self, saved, dout, ds):
        """Gradients of sum(output * dout) + sum(new residual * ds): of x (the residual's is the same), and by name."""
        p = self.p
        s, n, q, k, qn, kn, v, o, on, positions, states, cu = saved
        rows = lambda t: t.flatten(0, -2)  # noqa: E731
        g = {"w_out": rows(dout).t() @ rows(on.flatten(-2))}
        don = (dout @ p["w_out"]).unflatten(-1, (self.HV, self.V))
        do, _, g["norm_o"] = gdr.norm_bwd(don, o, p["norm_o"])
        dqn, dkn, dv, _ = gdr.la_bwd(qn, kn, v, self.decay, do, h0=states, cu_seqlens=cu, scale=self.scale)
        dq, dk, g["norm_q"], g["norm_k"] = gdr.qk_norm_bwd(dqn, dkn, q, k, p["norm_q"], p["norm_k"], cos=self.cos,
                                                           sin=self.sin, positions=positions)
        dqkv = torch.cat([t.flatten(-2) for t in (dq, dk, dv)], -1)
        g["w_in"] = rows(dqkv).t() @ rows(n)
        _, dres, g["norm"] = gdr.norm_bwd(dqkv @ p["w_in"], s, p["norm"], ds=ds)
        return dres, g


def main():
    torch.manual_seed(0)
    layer, width = LinearAttentionLayer(), 256
    lens = [300, 1, 77, 160]
    cu = torch.tensor([0, 300, 301, 378, 538], device="cuda")
    positions = torch.cat([torch.arange(n) for n in lens]).cuda()[None]
    x, residual = (torch.randn(1, 538, width, device="cuda").bfloat16() for _ in range(2))
    out, _, st, _ = layer.prefill(x, residual, positions, cu_seqlens=cu)
    print("prefill of", lens, "->", tuple(out.shape))

    # decode: the four sequences go on, their states in slots of a larger pool
    pool = layer.empty_states(16)
    slots = torch.tensor([3, 9, 0, 12], dtype=torch.int32, device="cuda")
    pool[slots.long()] = st
    tokens, at = torch.randn(8, 4, width, device="cuda").bfloat16(), torch.tensor(lens, device="cuda")
    for t in range(8):
        y, _ = layer.step(tokens[t], tokens[t], at + t, pool, slots)
    more = tokens[:, 3][None]
    whole, _, _, _ = layer.prefill(torch.cat([x[:, 378:], more], 1), torch.cat([residual[:, 378:], more], 1),
                                   torch.arange(168, device="cuda")[None])
    err = float((y[3] - whole[0, -1]).float().norm() / whole[0, -1].float().norm())
    print("eight decoded tokens against a longer prompt: relative difference %.1e" % err)

    # training: a few steps down the gradient on a fixed target, each parameter by a few thousandths of its size
    target = torch.randn_like(out)
    for it in range(5):
        out, res, _, saved = layer.prefill(x, residual, positions, cu_seqlens=cu)
        print("step", it, "loss %.4f" % float((out - target).float().square().mean()))
        _, grads = layer.backward(saved, (out - target) * (2 / out.numel()), torch.zeros_like(res))
        for k, gk in grads.items():
            now = layer.p[k].float()
            size = 0.003 * now.norm().clamp_min(1e-2) / gk.float().norm().clamp_min(1e-20)
            layer.p[k] = (now - size * gk.float()).to(layer.p[k].dtype)
    status = gdr.device_status()
    assert status == 0, gdr.last_error()


if __name__ == "__main__":
    main()
