"""Two layers of a GDN/MLA hybrid, from prompt to single tokens and through a training step.

A gated-delta-rule layer keeps one state a head; a latent-attention layer keeps one row of dc + dr values a token in a
paged cache.  Both run on this library, the projections around them on torch.  `main` checks that tokens decoded one
by one from the state and the cache come out as they do when the whole sequence is run as a prompt, and that the
attention layer's gradients of a training step agree with torch's.

    python examples/hybrid_layers.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_recurrence_delta_gb300 as gdn  # noqa: E402

BF16, EPS = torch.bfloat16, 1e-6


def weight(g, *shape):
    return (torch.randn(shape, generator=g, device="cuda") / math.sqrt(shape[-1])).to(BF16)


class DeltaLayer:
    """x + W_o . gated delta rule(W x): one state [d, d] a head and sequence."""

    def __init__(self, g, dim, H, d):
        self.H, self.d = H, d
        self.w_vbc, self.w_gate, self.w_out = weight(g, 3 * H * d, dim), weight(g, 2 * H, dim), weight(g, dim, H * d)
        self.A_log = torch.rand(H, d, generator=g, device="cuda") * math.log(16.0)

    def __call__(self, x, state, fresh):
        """x [B, T, dim]; state [B, H, d, d] fp32 is read unless `fresh` and holds the last token's state afterwards."""
        B, T, _ = x.shape
        v, b, c = (x @ self.w_vbc.T).view(B, T, 3, self.H, self.d).unbind(2)
        v, b, c = v.contiguous(), b.contiguous(), c.contiguous()
        gate, beta = ((x @ self.w_gate.T).view(B, T, 2, self.H).unbind(2))
        s = gdn.make_shape(B, self.H, T, self.d, self.d, "delta", "bf16", gate_logits=True, norm_bc=True)
        o, ws = torch.empty_like(v), torch.empty(gdn.gdn_workspace_bytes(s, 0), dtype=torch.uint8, device="cuda")
        gdn.check(gdn.gdn_fwd(s, v, b, c, gate.contiguous(), beta.contiguous(), self.A_log, None if fresh else state, o, state, ws))
        return x + o.flatten(2) @ self.w_out.T


class LatentLayer:
    """x + W_o . latent attention: queries of H heads over keys and values that come from one latent a token."""

    def __init__(self, g, dim, H, Hkv, dc, dn, dr, dv, positions):
        self.H, self.Hkv, self.dc, self.dn, self.dr, self.dv, self.npos = H, Hkv, dc, dn, dr, dv, positions
        self.w_q, self.w_down = weight(g, H * (dn + dr), dim), weight(g, dc + dr, dim)
        self.w_up, self.w_out = weight(g, Hkv * (dn + dv), dc), weight(g, dim, H * dv)
        self.norm = 1.0 + 0.1 * torch.randn(dc, generator=g, device="cuda")
        a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -2.0 * torch.arange(dr // 2, device="cuda", dtype=torch.float64) / dr)
        self.rot = torch.cat([a.cos(), a.sin()], 1).float()
        self.scale = 1.0 / math.sqrt(dn + dr)

    def project(self, x):
        return x @ self.w_down.T, (x @ self.w_q.T).view(-1, self.H, self.dn + self.dr)

    def attend(self, q, qr, lat, kr, cu, longest, train=False):
        """Packed queries over their own sequences' latents, expanded: o (and lse, workspace and keys for the gradients)."""
        N = q.shape[0]
        kv = (lat @ self.w_up.T).view(N, self.Hkv, self.dn + self.dv)
        s = gdn.make_mla_attn(cu.numel() - 1, self.H, self.Hkv, longest, longest, self.dn, self.dr, self.dv, "bf16", self.scale,
                              Nq=N, Nk=N)
        o = torch.empty(N, self.H, self.dv, dtype=BF16, device="cuda")
        lse = torch.empty(self.H, N, device="cuda") if train else None
        ws = torch.empty(gdn.gdn_mla_workspace_bytes(s, int(train)), dtype=torch.uint8, device="cuda")
        gdn.check(gdn.gdn_mla_fwd(s, q[..., : self.dn], qr, kv[..., : self.dn], kr, kv[..., self.dn:], cu, cu, o, lse, ws))
        return (o, lse, kv, s, ws) if train else o

    def prompt(self, x, cache, rows, pos, cu, longest):
        """x [N, dim], packed prompts; `rows` of the cache receive the latents and the rotated keys for later steps."""
        N = x.shape[0]
        down, q = self.project(x)
        qr = torch.empty(N, self.H, self.dr, dtype=BF16, device="cuda")
        lat, kr = (torch.empty(N, d, dtype=BF16, device="cuda") for d in (self.dc, self.dr))
        p = gdn.make_mla_prep(N, self.H, self.dc, self.dr, "bf16", self.npos, EPS)
        gdn.check(gdn.gdn_mla_prep(p, down, self.norm, self.rot, pos, None, None, q[..., self.dn:], lat, kr, qr))
        cache.view(-1, self.dc + self.dr)[rows] = torch.cat([lat, kr], 1)
        return x + self.attend(q, qr, lat, kr, cu, longest).flatten(1) @ self.w_out.T

    def step(self, x, cache, table, lens):
        """x [B, dim], one new token a sequence at position lens - 1: into the cache, then over it without expanding it."""
        B = x.shape[0]
        down, q = self.project(x)
        qr = torch.empty(B, self.H, self.dr, dtype=BF16, device="cuda")
        pages, page = cache.shape[:2]
        p = gdn.make_mla_prep(B, self.H, self.dc, self.dr, "bf16", self.npos, EPS, B=B, page=page, npages=pages,
                              maxpages=table.shape[1])
        gdn.check(gdn.gdn_mla_prep(p, down, self.norm, self.rot, lens - 1, torch.arange(B, device="cuda", dtype=torch.int32), table,
                                   q[..., self.dn:], cache, None, qr))
        # the up projection moves into the query, and behind the output
        G = self.H // self.Hkv
        up = self.w_up.view(self.Hkv, self.dn + self.dv, self.dc)
        qc = torch.einsum("bgid,gdc->bgic", q[..., : self.dn].reshape(B, self.Hkv, G, self.dn), up[:, : self.dn])
        qc = qc.reshape(B, 1, self.H, self.dc)
        s = gdn.make_mla_cache(B, 1, self.H, self.dc, self.dr, page, pages, table.shape[1], "bf16", self.scale)
        ws = torch.empty(gdn.gdn_mla_decode_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(qc)
        gdn.check(gdn.gdn_mla_decode(s, qc, qr.view(B, 1, self.H, self.dr), cache, table, lens, o, None, ws))
        o = torch.einsum("bgic,gvc->bgiv", o.view(B, self.Hkv, G, self.dc), up[:, self.dn:])
        return x + o.reshape(B, self.H * self.dv) @ self.w_out.T

    def gradients(self, x, pos, cu, longest, dy):
        """Gradients of the down projection's rows, the queries and the norm's weight for one sequence batch, from the
        gradient dy of the attention's output."""
        N = x.shape[0]
        down, q = self.project(x)
        qr = torch.empty(N, self.H, self.dr, dtype=BF16, device="cuda")
        lat, kr = (torch.empty(N, d, dtype=BF16, device="cuda") for d in (self.dc, self.dr))
        p = gdn.make_mla_prep(N, self.H, self.dc, self.dr, "bf16", self.npos, EPS)
        gdn.check(gdn.gdn_mla_prep(p, down, self.norm, self.rot, pos, None, None, q[..., self.dn:], lat, kr, qr))
        o, lse, kv, s, ws = self.attend(q, qr, lat, kr, cu, longest, train=True)
        dq, dkv, dkr = torch.empty_like(q), torch.empty_like(kv), torch.empty_like(kr)
        gdn.check(gdn.gdn_mla_bwd(s, q[..., : self.dn], qr, kv[..., : self.dn], kr, kv[..., self.dn:], cu, cu, o, lse, dy,
                                  dq[..., : self.dn], dq[..., self.dn:], dkv[..., : self.dn], dkr, dkv[..., self.dn:], ws))
        gdn.check(gdn.gdn_last_device_status(ws))
        dlat = dkv.flatten(1) @ self.w_up
        ddown, dnorm = torch.empty_like(down), torch.empty_like(self.norm)
        wp = torch.empty(gdn.gdn_mla_prep_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        turned = dq[..., self.dn:]                               # turned back in place
        gdn.check(gdn.gdn_mla_prep_bwd(p, down, self.norm, self.rot, pos, dlat, dkr, turned, ddown, dnorm, turned, wp))
        return {"down": ddown, "q": dq, "norm": dnorm}

    def gradients_by_torch(self, x, pos, lens, dy):
        """The same from torch's reverse mode in 32 bits, a sequence at a time."""
        down, q = (t.float().requires_grad_() for t in self.project(x))
        norm = self.norm.clone().requires_grad_()
        r = self.rot[pos.long()]
        cos, sin = r[:, : self.dr // 2], r[:, self.dr // 2:]

        def turn(t, c, s):
            a, b = t.chunk(2, -1)
            return torch.cat([a * c - b * s, a * s + b * c], -1)

        z = down[:, : self.dc]
        lat = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * norm
        kr = turn(down[:, self.dc:], cos, sin)
        qq = torch.cat([q[..., : self.dn], turn(q[..., self.dn:], cos[:, None], sin[:, None])], -1)
        kv = (lat @ self.w_up.float().T).view(-1, self.Hkv, self.dn + self.dv).repeat_interleave(self.H // self.Hkv, 1)
        k = torch.cat([kv[..., : self.dn], kr[:, None].expand(-1, self.H, -1)], -1)
        loss, at = 0.0, 0
        for n in lens:
            i = slice(at, at + n)
            w = torch.einsum("ihd,jhd->hij", qq[i], k[i]) * self.scale
            w = w.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf).softmax(-1)
            loss, at = loss + (torch.einsum("hij,jhv->ihv", w, kv[i][..., self.dn:]) * dy[i].float()).sum(), at + n
        return dict(zip(("down", "q", "norm"), torch.autograd.grad(loss, [down, q, norm])))


def main(dim=512, lens=(150, 77, 300), steps=5, page=64, say=print):
    g = torch.Generator(device="cuda").manual_seed(0)
    B, total = len(lens), [n + steps for n in lens]
    delta = DeltaLayer(g, dim, 8, 64)
    latent = LatentLayer(g, dim, 8, 2, 128, 64, 32, 64, positions=max(total))
    per = [-(-n // page) for n in total]
    cache = torch.zeros(sum(per) + 1, page, latent.dc + latent.dr, dtype=BF16, device="cuda")
    table = torch.full((B, max(per)), -1, dtype=torch.int32)
    for b in range(B):       # the last sequence's pages first, to have a table that matters
        table[b, : per[b]] = torch.arange(per[b]) + sum(per[b + 1:])
    tokens = [torch.randn(n, dim, generator=g, device="cuda").to(BF16) for n in total]

    def run(upto, into):
        """Both layers over the first upto[b] tokens of each sequence as prompts: outputs and the delta layer's states."""
        states = torch.empty(B, delta.H, delta.d, delta.d, device="cuda")
        mid = torch.cat([delta(tokens[b][None, : upto[b]], states[b:b + 1], fresh=True)[0] for b in range(B)])
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in upto])
        seq = torch.tensor([b for b, n in enumerate(upto) for _ in range(n)])
        rows = (table[seq, pos.long() // page].long() * page + pos.long() % page).cuda()
        cu = torch.tensor([sum(upto[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        return latent.prompt(mid, into, rows, pos.cuda(), cu, max(upto)), states, mid, pos.cuda(), cu

    _, states, mid, pos, cu = run(list(lens), cache)
    dy = torch.randn(sum(lens), latent.H, latent.dv, generator=g, device="cuda").to(BF16)
    worst = {}
    ours, theirs = latent.gradients(mid, pos, cu, max(lens), dy), latent.gradients_by_torch(mid, pos, lens, dy)
    for k in ours:
        worst["gradient of " + k] = ((ours[k].float() - theirs[k]).norm() / theirs[k].norm()).item()
    got = []
    for t in range(steps):
        x = torch.stack([tokens[b][lens[b] + t] for b in range(B)])
        x = delta(x[:, None], states, fresh=False)[:, 0]
        got.append(latent.step(x, cache, table.cuda(), torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device="cuda")))
    whole = run(total, torch.zeros_like(cache))[0].split(total)
    want = torch.stack([torch.stack([whole[b][lens[b] + t] for b in range(B)]) for t in range(steps)])
    worst["decoded tokens"] = ((torch.stack(got).float() - want.float()).norm() / want.float().norm()).item()
    for k, v in worst.items():
        say(f"{k}: relative difference {v:.2e}")
    return worst


if __name__ == "__main__":
    main()
