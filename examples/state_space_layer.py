"""A state-space layer, from packed prompts to single tokens and through a training step.

Residual addition and RMS norm, a projection, the short causal convolution, projections to step sizes and to write and read
vectors, the selective scan with its gate, a projection back: norm, convolution and scan run on this library, the
projections on torch.  A sequence's memory is one convolution state and one scan state, kept in slots.  `main` checks that
tokens decoded one by one from the slots come out as they do when the whole sequence is run as a prompt, that an 8-bit norm
stands for the norm, and that a training step's gradients agree with torch's.

    python examples/state_space_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_recurrence_delta_gb300 as gdn  # noqa: E402

BF16, EPS = torch.bfloat16, 1e-6


class StateSpaceLayer:
    """res + x joins the residual stream, whose norm is mixed: W_out . scan(conv(W_in . norm))."""

    def __init__(self, g, dim, D, N=16, W=4, rank=None):
        self.dim, self.D, self.N, self.W = dim, D, N, W
        self.R = rank or 8 * max(1, dim // 128)
        weight = lambda *s: (torch.randn(s, generator=g, device="cuda") / math.sqrt(s[-1])).to(BF16)  # noqa: E731
        self.w_in, self.w_out = weight(2 * D, dim), weight(dim, D)
        self.w_bc, self.w_dt = weight(self.R + 2 * N, D), weight(D, self.R)
        self.norm = 1.0 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        self.taps = torch.randn(D, W, generator=g, device="cuda") / math.sqrt(W)
        self.conv_bias = 0.1 * torch.randn(D, generator=g, device="cuda")
        self.A_log = torch.log(torch.arange(1, N + 1, device="cuda").float()).expand(D, N).contiguous()
        self.skip = torch.ones(D, device="cuda")
        size = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(0.01), math.log(0.1), generator=g))
        self.dt_bias = size + torch.log(-torch.expm1(-size))

    def empty(self, rows, width):
        return torch.empty((rows, width), dtype=BF16, device="cuda")

    def normed(self, x, res):
        """The residual stream with x added, in place, and its norm."""
        y = self.empty(*x.shape)
        gdn.check(gdn.gdn_norm_fwd(gdn.make_norm(*x.shape, eps=EPS), x, res, self.norm, y, None, res))
        return y

    def normed8(self, x, res, group=128):
        """The same with an 8-bit result and a scale for each `group` values."""
        rows, dim = x.shape
        y = torch.empty((rows, dim), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty((rows, dim // group), device="cuda")
        gdn.check(gdn.gdn_norm_fwd(gdn.make_norm(rows, dim, out="e4m3", group=group, eps=EPS), x, res, self.norm, y, scale, res))
        return y, scale

    def vectors(self, u):
        """Step sizes before their bias and softplus, and the scan's write and read vectors, as slices of a projection."""
        bc = u @ self.w_bc.T
        return bc[:, : self.R] @ self.w_dt.T, bc[:, None, self.R: self.R + self.N], bc[:, None, self.R + self.N:], bc

    def prompt(self, x, res, cu, longest, conv_state=None, scan_state=None, slots=None, train=False):
        """Packed rows: the layer's output; the sequences' states go to their slots."""
        rows, B = x.shape[0], cu.numel() - 1
        n = self.normed(x, res)
        xz = n @ self.w_in.T
        u, y = self.empty(rows, self.D), self.empty(rows, self.D)
        sT = torch.empty((B, self.W - 1, self.D), dtype=BF16, device="cuda")
        hT = torch.empty((B, self.D, self.N), device="cuda")
        c = gdn.make_conv(B, longest, self.D, self.W, rows=rows)
        gdn.check(gdn.gdn_conv_fwd(c, xz[:, : self.D], self.taps, self.conv_bias, cu, None, u, sT))
        dt, Bm, Cm, bc = self.vectors(u)
        s = gdn.make_scan(B, longest, self.D, self.N, rows=rows)
        ws = torch.empty(gdn.gdn_scan_workspace_bytes(s, 0), dtype=torch.uint8, device="cuda")
        saved = torch.empty(gdn.gdn_scan_saved_bytes(s), dtype=torch.uint8, device="cuda") if train else None
        gdn.check(gdn.gdn_scan_fwd(s, u, dt, xz[:, self.D:], Bm, Cm, self.A_log, self.skip, self.dt_bias, cu, None, y, hT, saved, ws))
        if slots is not None:
            conv_state[slots.long()], scan_state[slots.long()] = sT, hT
        out = y @ self.w_out.T
        return (out, n, xz, u, dt, bc, y, saved, c, s) if train else out

    def step(self, x, res, conv_state, scan_state, slots, T=1):
        """T new tokens of each sequence, from and to its slot."""
        B = slots.numel()
        xz = self.normed(x, res) @ self.w_in.T
        u, y = self.empty(B * T, self.D), self.empty(B * T, self.D)
        c = gdn.make_conv_step(B, T, self.D, self.W, conv_state.shape[0])
        gdn.check(gdn.gdn_conv_step(c, xz[:, : self.D], self.taps, self.conv_bias, conv_state, slots, None, u))
        dt, Bm, Cm, _ = self.vectors(u)
        s = gdn.make_scan_step(B, T, self.D, self.N, scan_state.shape[0])
        gdn.check(gdn.gdn_scan_step(s, u, dt, xz[:, self.D:], Bm, Cm, self.A_log, self.skip, self.dt_bias, scan_state, slots, None, y))
        return y @ self.w_out.T

    def gradients(self, x, res, cu, longest, dout, dsum):
        """Gradients of a training step, from those of the layer's output and of the residual stream behind the addition."""
        total, D, N, R = res.clone(), self.D, self.N, self.R
        out, n, xz, u, dt, bc, y, saved, c, s = self.prompt(x, total, cu, longest, train=True)
        rows = x.shape[0]
        dy, dxz, du, ddt, dbc = dout @ self.w_out, torch.empty_like(xz), torch.empty_like(u), torch.empty_like(dt), torch.empty_like(bc)
        dA, dskip, dbias = torch.empty_like(self.A_log), torch.empty_like(self.skip), torch.empty_like(self.skip)
        ws = torch.empty(gdn.gdn_scan_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
        gdn.check(gdn.gdn_scan_bwd(s, u, dt, xz[:, D:], bc[:, None, R: R + N], bc[:, None, R + N:], self.A_log, self.skip, self.dt_bias,
                                   cu, saved, dy, None, du, ddt, dxz[:, D:], dbc[:, None, R: R + N], dbc[:, None, R + N:], dA, dskip,
                                   dbias, None, ws))
        dbc[:, :R] = ddt @ self.w_dt
        du = du + dbc @ self.w_bc
        dtaps, dcb = torch.empty_like(self.taps), torch.empty_like(self.conv_bias)
        wc = torch.empty(gdn.gdn_conv_workspace_bytes(c), dtype=torch.uint8, device="cuda")
        gdn.check(gdn.gdn_conv_bwd(c, xz[:, :D], self.taps, self.conv_bias, cu, None, du, None, dxz[:, :D], dtaps, dcb, None, wc))
        dn, dx, dnorm = dxz @ self.w_in, self.empty(rows, self.dim), torch.empty_like(self.norm)
        p = gdn.make_norm(rows, self.dim, eps=EPS)
        wn = torch.empty(gdn.gdn_norm_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        gdn.check(gdn.gdn_norm_bwd(p, total, self.norm, dn, dsum, dx, None, dnorm, wn))
        return {"x": dx, "norm": dnorm, "taps": dtaps, "conv_bias": dcb, "A_log": dA, "skip": dskip, "dt_bias": dbias,
                "w_in": dxz.T @ n, "w_bc": dbc.T @ u, "w_dt": ddt.T @ bc[:, :R], "w_out": dout.T @ y}

    def gradients_by_torch(self, x, res, lens, dout, dsum):
        """The same from torch's reverse mode in 32 bits, token by token."""
        names = ("norm", "taps", "conv_bias", "A_log", "skip", "dt_bias", "w_in", "w_bc", "w_dt", "w_out")
        w = {k: getattr(self, k).float().detach().requires_grad_() for k in names}
        total = (x.float() + res.float()).to(BF16).float().requires_grad_()
        n = total * torch.rsqrt(total.square().mean(-1, keepdim=True) + EPS) * w["norm"]
        xz = n @ w["w_in"].T
        outs, at = [], 0
        for length in lens:
            part = xz[at: at + length]
            v = torch.nn.functional.pad(part[:, : self.D].T, (self.W - 1, 0))
            v = (v.unfold(1, self.W, 1) * w["taps"][:, None]).sum(-1).T + w["conv_bias"]
            u = torch.nn.functional.silu(v)
            bc = u @ w["w_bc"].T
            size = torch.nn.functional.softplus(bc[:, : self.R] @ w["w_dt"].T + w["dt_bias"])
            h = torch.zeros(self.D, self.N, device="cuda")
            for t in range(length):
                h = torch.exp(-size[t][:, None] * w["A_log"].exp()) * h + (size[t] * u[t])[:, None] * bc[t, self.R: self.R + self.N]
                outs.append(((h * bc[t, self.R + self.N:]).sum(-1) + w["skip"] * u[t]) * torch.nn.functional.silu(part[t, self.D:]))
            at += length
        loss = ((torch.stack(outs) @ w["w_out"].T) * dout.float()).sum() + (total * dsum.float()).sum()
        return dict(zip(("x",) + names, torch.autograd.grad(loss, [total] + [w[k] for k in names])))


def main(dim=256, D=512, N=16, lens=(70, 33, 128), steps=6, say=print):
    g = torch.Generator(device="cuda").manual_seed(0)
    layers = [StateSpaceLayer(g, dim, D, N) for _ in range(2)]
    B, slots = len(lens), len(lens) + 2
    slot = torch.randperm(slots, generator=g, device="cuda")[:B].int()
    tokens = [torch.randn(n + steps, dim, generator=g, device="cuda").to(BF16) for n in lens]
    pools = [(torch.zeros(slots, layer.W - 1, D, dtype=BF16, device="cuda"), torch.zeros(slots, D, N, device="cuda")) for layer in layers]
    offsets = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    worst = {}

    def far(a, b):
        return ((a.float() - b.float()).norm() / b.float().norm()).item()

    def run(upto, pools=None):
        x = torch.cat([tokens[b][: upto[b]] for b in range(B)])
        res = torch.zeros_like(x)
        for k, layer in enumerate(layers):
            x = layer.prompt(x, res, offsets(upto), max(upto), *(pools[k] + (slot,) if pools else ()))
        return x + res

    run(list(lens), pools)
    got, one = [], torch.zeros(B, dim, dtype=BF16, device="cuda")
    for t in range(steps):
        x, res = torch.stack([tokens[b][lens[b] + t] for b in range(B)]), one.clone()
        for k, layer in enumerate(layers):
            x = layer.step(x, res, *pools[k], slot)
        got.append(x + res)
    whole = run([n + steps for n in lens]).split([n + steps for n in lens])
    worst["decoded tokens"] = far(torch.stack(got), torch.stack([torch.stack([whole[b][lens[b] + t] for b in range(B)]) for t in range(steps)]))

    layer, cu = layers[0], offsets(lens)
    x, res = torch.cat([tokens[b][: lens[b]] for b in range(B)]), torch.randn(sum(lens), dim, generator=g, device="cuda").to(BF16)
    y8, scale = layer.normed8(x, res.clone())
    worst["8-bit norm"] = far(y8.float() * scale.repeat_interleave(128, 1), layer.normed(x, res.clone()))
    dout, dsum = (torch.randn(sum(lens), dim, generator=g, device="cuda").to(BF16) for _ in range(2))
    ours, theirs = layer.gradients(x, res, cu, max(lens), dout, dsum), layer.gradients_by_torch(x, res, lens, dout, dsum)
    for k in theirs:
        worst["gradient of " + k] = far(ours[k], theirs[k])
    for k, v in worst.items():
        say(f"{k}: relative difference {v:.2e}")
    return worst


if __name__ == "__main__":
    main()
