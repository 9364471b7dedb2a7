"""A selective state space layer built from the library's operators: norm with
the residual's addition, input projection, short convolution, selective scan,
output projection.  One class serves a packed prefill, single-token decode with
states in a pool of slots, and a training step.

    python examples/ssm_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_08_gb300 as gdr  # noqa: E402


class SsmLayer:
    """Parameters as plain tensors; ``width`` is the residual stream's, ``inner`` the scan's channels."""

    def __init__(self, width=256, inner=512, states=16, rank=16, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def randn(*shape, k):
            return (torch.randn(*shape, generator=g) * k).to(device=device, dtype=dtype)

        self.inner, self.states, self.rank, self.taps, self.dtype, self.device = inner, states, rank, taps, dtype, device
        delta = torch.exp(torch.rand(inner, generator=g) * 4.6 - 6.9)  # 1e-3 to 1e-1 at rest
        self.p = {
            "norm": torch.ones(width, dtype=dtype, device=device),
            "w_in": randn(2 * inner, width, k=width ** -0.5),
            "conv_w": randn(inner, taps, k=taps ** -0.5),
            "conv_b": torch.zeros(inner, dtype=dtype, device=device),
            "w_bc": randn(rank + 2 * states, inner, k=inner ** -0.5),
            "w_dt": randn(inner, rank, k=rank ** -0.5),
            "dt_bias": (delta + torch.log(-torch.expm1(-delta))).to(device),
            "a": -torch.arange(1.0, states + 1, device=device).repeat(inner, 1),
            "d": torch.ones(inner, device=device),
            "w_out": randn(width, inner, k=inner ** -0.5),
        }

    def empty_states(self, n):
        """(inputs of the convolution, states of the scan) of n sequences, or slots."""
        return (torch.zeros(n, self.taps - 1, self.inner, dtype=self.dtype, device=self.device),
                torch.zeros(n, self.inner, self.states, device=self.device))

    def _scan_inputs(self, u):
        """dt, b and c of the convolved input; b and c stay parts of the one projection."""
        r, s = self.rank, self.states
        dbc = u @ self.p["w_bc"].t()
        return (dbc, dbc[..., :r] @ self.p["w_dt"].t(), dbc[..., r:r + s].unflatten(-1, (1, s)),
                dbc[..., r + s:].unflatten(-1, (1, s)))

    def prefill(self, x, residual, states=None, cu_seqlens=None):
        """x, residual [B, T, width] (packed: [1, T, width]) -> output, new residual, states, what backward needs."""
        p = self.p
        s0, h0 = states if states is not None else (None, None)
        n, s = gdr.norm_fwd(x, p["norm"], residual)
        xz = n @ p["w_in"].t()
        xi, z = xz[..., :self.inner], xz[..., self.inner:]  # slices: no copies
        u, st = gdr.conv_fwd(xi, p["conv_w"], bias=p["conv_b"], s0=s0, cu_seqlens=cu_seqlens)
        dbc, dt, b, c = self._scan_inputs(u)
        y, ht = gdr.ssm_fwd(u, dt, p["a"], b, c, d=p["d"], z=z, dt_bias=p["dt_bias"], h0=h0, cu_seqlens=cu_seqlens)
        return y @ p["w_out"].t(), s, (st, ht), (s, n, xi, z, u, dbc, dt, b, c, y, s0, h0, cu_seqlens)

    def step(self, x, residual, states, slots):
        """One token of each running sequence: x, residual [R, width]; its states are updated in their slots."""
        p = self.p
        n, s = gdr.norm_fwd(x, p["norm"], residual)
        xz = n @ p["w_in"].t()
        u = gdr.conv_step(xz[:, :self.inner], states[0], p["conv_w"], bias=p["conv_b"], slots=slots)
        _, dt, b, c = self._scan_inputs(u)
        y = gdr.ssm_step(u, dt, p["a"], b, c, states[1], d=p["d"], z=xz[:, self.inner:], dt_bias=p["dt_bias"],
                         slots=slots)
        return y @ p["w_out"].t(), s

    def backward(self, saved, dout, ds):
        """Gradients of sum(output * dout) + sum(new residual * ds): of x (the residual's is the same), and by name."""
        p, r, st = self.p, self.rank, self.states
        s, n, xi, z, u, dbc, dt, b, c, y, s0, h0, cu = saved
        rows = lambda t: t.flatten(0, -2)  # noqa: E731
        g = {"w_out": rows(dout).t() @ rows(y)}
        du, ddt, g["a"], db, dc, g["d"], dz, g["dt_bias"], _ = gdr.ssm_bwd(
            u, dt, p["a"], b, c, dout @ p["w_out"], d=p["d"], z=z, dt_bias=p["dt_bias"], h0=h0, cu_seqlens=cu)
        g["w_dt"] = rows(ddt).t() @ rows(dbc[..., :r])
        ddbc = torch.cat([ddt @ p["w_dt"], db.flatten(-2), dc.flatten(-2)], -1)
        g["w_bc"] = rows(ddbc).t() @ rows(u)
        dxi, g["conv_w"], g["conv_b"], _ = gdr.conv_bwd(xi, p["conv_w"], du + ddbc @ p["w_bc"], bias=p["conv_b"], s0=s0,
                                                       cu_seqlens=cu)
        dxz = torch.cat([dxi, dz], -1)
        g["w_in"] = rows(dxz).t() @ rows(n)
        _, dres, g["norm"] = gdr.norm_bwd(dxz @ p["w_in"], s, p["norm"], ds=ds)
        return dres, g


def main():
    torch.manual_seed(0)
    layer, width = SsmLayer(), 256
    lens = [300, 1, 77, 160]
    cu = torch.tensor([0, 300, 301, 378, 538], device="cuda")
    x = torch.randn(1, 538, width, device="cuda").bfloat16()
    residual = torch.randn(1, 538, width, device="cuda").bfloat16()
    out, res, (st, ht), saved = layer.prefill(x, residual, cu_seqlens=cu)
    print("prefill of", lens, "->", tuple(out.shape))

    # decode: the four sequences go on, their states in slots of a larger pool
    conv_pool, scan_pool = layer.empty_states(16)
    slots = torch.tensor([3, 9, 0, 12], dtype=torch.int32, device="cuda")
    conv_pool[slots.long()], scan_pool[slots.long()] = st, ht
    tokens = torch.randn(8, 4, width, device="cuda").bfloat16()
    for t in range(8):
        y, _ = layer.step(tokens[t], tokens[t], (conv_pool, scan_pool), slots)
    whole, _, _, _ = layer.prefill(torch.cat([x[:, 378:], tokens[:, 3][None]], 1),
                                   torch.cat([residual[:, 378:], tokens[:, 3][None]], 1))
    err = float((y[3] - whole[0, -1]).float().norm() / whole[0, -1].float().norm())
    print("eight decoded tokens against a longer prompt: relative difference %.1e" % err)

    # training: a few steps down the gradient on a fixed target, each parameter by a few thousandths of its size
    target = torch.randn_like(out)
    for it in range(5):
        out, res, _, saved = layer.prefill(x, residual, cu_seqlens=cu)
        dout = (out - target) * (2 / out.numel())
        print("step", it, "loss %.4f" % float((out - target).float().square().mean()))
        _, grads = layer.backward(saved, dout, torch.zeros_like(res))
        for k, gk in grads.items():
            now = layer.p[k].float()
            size = 0.003 * now.norm().clamp_min(1e-2) / gk.float().norm().clamp_min(1e-20)
            layer.p[k] = (now - size * gk.float()).to(layer.p[k].dtype)
    status = gdr.device_status()
    assert status == 0, gdr.last_error()


if __name__ == "__main__":
    main()
