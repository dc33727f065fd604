"""Latent attention in 64 bits on the CPU, and seeded inputs for it: what the tests of ``gdn_mla_*`` compare against.

The definitions are written per sequence and head with plain torch operations; gradients come from torch's reverse
mode on those definitions and, where a test asks for it, from central differences of them.
"""
import math

import torch

import linear_attention_recurrence_delta_gb300 as gdn

EPS = 1e-6

# A bf16 result is rounded once (2^-9 of its size at most), and on the way the weights, or the scores' gradients, are
# rounded to bf16 before a matrix product (2^-9 each again); a gradient also sees o's own rounding through
# rowsum(dO o).  Against the largest value of the result that is 2 roundings forward and 3 backward, with half as
# much again for sums in which rounded terms cancel; in norm the roundings are independent and add in squares.
# f32 results go through sums of up to a few thousand fp32 products.
U = 2.0 ** -9
TOL_MAX = {("bf16", "fwd"): 3 * U, ("bf16", "bwd"): 5 * U, ("f32", "fwd"): 1e-5, ("f32", "bwd"): 2e-5}
TOL_NORM = {("bf16", "fwd"): 1.5 * U, ("bf16", "bwd"): 2 * U, ("f32", "fwd"): 5e-6, ("f32", "bwd"): 1e-5}


def tdtype(io):
    return torch.float32 if io == "f32" else torch.bfloat16


def close(got, ref, io, way, name):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    if ref.numel() == 0:
        return
    top, norm = ref.abs().max().item(), ref.norm().item()
    d = (got - ref).abs()
    if top == 0.0:
        assert d.max().item() == 0.0, f"{name}: {d.max().item():.3e} where zero is exact"
        return
    assert d.max().item() <= TOL_MAX[io, way] * top, f"{name}: max {d.max().item() / top:.3e} > {TOL_MAX[io, way]:.1e}"
    assert (got - ref).norm().item() <= TOL_NORM[io, way] * norm, \
        f"{name}: norm {(got - ref).norm().item() / norm:.3e} > {TOL_NORM[io, way]:.1e}"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, io, std=1.0):
    """Values exactly representable in the I/O type, as a CPU tensor of it."""
    return (torch.randn(shape, generator=g) * std).to(tdtype(io))


# ---------------------------------------------------------------- attention over expanded keys and values

def offsets(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def attn_one(q, k, v, scale, causal):
    """One head of one sequence: o and lse; rows that see nothing give 0 and -inf."""
    a, b = q.shape[0], k.shape[0]
    x = (q @ k.T) * scale
    if causal:
        i, j = torch.arange(a)[:, None], torch.arange(b)[None]
        x = x.masked_fill(j > i + b - a, -math.inf)
    empty = max(0, min(a, a - b)) if causal else (a if b == 0 else 0)
    lse = torch.full((a,), -math.inf, dtype=q.dtype)
    o = torch.zeros(a, v.shape[1], dtype=q.dtype)
    if empty < a:
        w = torch.softmax(x[empty:], -1)
        o = torch.cat([o[:empty], w @ v])
        lse = torch.cat([lse[:empty], torch.logsumexp(x[empty:], -1)])
    return o, lse


def attn_ref(x, nq, nk, scale, causal, dO=None):
    """x: dict of qn, qr, kn, kr, v (CPU, any float type; qr, kr may be None) -> o, lse [H, Nq], gradients."""
    x = {k: (None if t is None else t.double().requires_grad_(dO is not None)) for k, t in x.items()}
    Nq, H = x["qn"].shape[:2]
    Hkv = x["kn"].shape[1]
    oq, ok = offsets(nq), offsets(nk)
    os, ls = [], []
    for b in range(len(nq)):
        heads, lses = [], []
        for h in range(H):
            g = h // (H // Hkv)
            qs, ks = slice(oq[b], oq[b + 1]), slice(ok[b], ok[b + 1])
            q, k = x["qn"][qs, h], x["kn"][ks, g]
            if x["qr"] is not None:
                q, k = torch.cat([q, x["qr"][qs, h]], -1), torch.cat([k, x["kr"][ks]], -1)
            o, lse = attn_one(q, k, x["v"][ks, g], scale, causal)
            heads.append(o)
            lses.append(lse)
        os.append(torch.stack(heads, 1))
        ls.append(torch.stack(lses, 0))
    o, lse = torch.cat(os, 0), torch.cat(ls, 1)
    if dO is None:
        return o, lse, None
    names = [k for k, t in x.items() if t is not None]
    g = torch.autograd.grad((o * dO.double()).sum(), [x[k] for k in names], allow_unused=True)
    return o.detach(), lse.detach(), {k: (torch.zeros_like(x[k]) if d is None else d) for k, d in zip(names, g)}


def attn_inputs(seed, nq, nk, H, Hkv, dn, dr, dv, io, joined=True):
    """Inputs on the CPU; joined: keys and values (and the queries' parts) are slices of one tensor."""
    g = gen(seed)
    q = normal(g, (sum(nq), H, dn + dr), io, 1.5)
    kv = normal(g, (sum(nk), Hkv, dn + dv), io)
    x = {"qn": q[..., :dn], "qr": q[..., dn:] if dr else None, "kn": kv[..., :dn],
         "kr": normal(g, (sum(nk), dr), io) if dr else None, "v": kv[..., dn:]}
    return x, normal(g, (sum(nq), H, dv), io)


def attn_run(x, nq, nk, scale, causal, io, dO=None, cu=True, Tq=None, Tk=None, stream=None, shape=None):
    """gdn_mla_fwd (and gdn_mla_bwd): device results; every output buffer starts as NaN."""
    dev = {k: (None if t is None else (t if t.is_cuda else t.cuda())) for k, t in x.items()}
    Nq, H, dn = dev["qn"].shape
    Nk, Hkv, dv = dev["v"].shape
    dr = 0 if dev["qr"] is None else dev["qr"].shape[-1]
    B = len(nq)
    s = shape or gdn.make_mla_attn(B, H, Hkv, Tq if Tq is not None else max(nq), Tk if Tk is not None else max(nk), dn, dr, dv,
                                   io, scale, causal, Nq=Nq, Nk=Nk)
    cu_q = torch.tensor(offsets(nq), dtype=torch.int32, device="cuda") if cu else None
    cu_k = torch.tensor(offsets(nk), dtype=torch.int32, device="cuda") if cu else None
    nan = lambda shape, dt=tdtype(io): torch.full(shape, math.nan, dtype=dt, device="cuda")  # noqa: E731
    o, lse = nan((Nq, H, dv)), nan((H, Nq), torch.float32)
    args = (dev["qn"], dev["qr"], dev["kn"], dev["kr"], dev["v"], cu_q, cu_k)
    ws = torch.full((gdn.gdn_mla_workspace_bytes(s, 1 if dO is not None else 0),), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_mla_fwd(s, *args, o, lse, ws, stream=stream), "gdn_mla_fwd")
    gdn.check(gdn.gdn_last_device_status(ws, stream=stream), "forward status")
    if dO is None:
        return o, lse, None
    dq, dkv, dkr = nan((Nq, H, dn + dr)), nan((Nk, Hkv, dn + dv)), nan((Nk, dr)) if dr else None
    d = {"qn": dq[..., :dn], "qr": dq[..., dn:] if dr else None, "kn": dkv[..., :dn], "kr": dkr, "v": dkv[..., dn:]}
    gdn.check(gdn.gdn_mla_bwd(s, *args, o, lse, dO.cuda(), *d.values(), ws, stream=stream), "gdn_mla_bwd")
    gdn.check(gdn.gdn_last_device_status(ws, stream=stream), "backward status")
    return o, lse, {k: t for k, t in d.items() if t is not None}


# ---------------------------------------------------------------- norm, rotation, cache write

def rotation(rows, dr, base=10000.0):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-2.0 * torch.arange(dr // 2, dtype=torch.float64) / max(dr, 1))
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate_ref(x, rot, interleaved):
    """x [N, ..., d] with rot's rows [N, d], in 64 bits."""
    d = x.shape[-1]
    at = torch.arange(d // 2)
    one, two = (2 * at, 2 * at + 1) if interleaved else (at, at + d // 2)
    r = rot.double().reshape([x.shape[0]] + [1] * (x.dim() - 2) + [d])
    c, s = r[..., : d // 2], r[..., d // 2:]
    out = torch.zeros_like(x)
    out[..., one] = x[..., one] * c - x[..., two] * s
    out[..., two] = x[..., one] * s + x[..., two] * c
    return out


def prep_ref(kv, w, dc, rot_rows, qr, interleaved, eps=EPS):
    x = kv[:, :dc]
    lat = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    kr = rotate_ref(kv[:, dc:], rot_rows, interleaved)
    return lat, kr, (None if qr is None else rotate_ref(qr, rot_rows, interleaved))


# ---------------------------------------------------------------- the paged cache

def block_table(g, n, page, spare=3, width=None):
    """A table of scattered pages for lengths n; entries past a sequence's end are -1 (no page is shared)."""
    per = [-(-k // page) for k in n]
    order = torch.randperm(sum(per) + spare, generator=g).tolist()
    width = width or max(1, max(per))
    t = torch.full((len(n), width), -1, dtype=torch.int32)
    for b, k in enumerate(per):
        for i in range(k):
            t[b, i] = order.pop()
    return t, sum(per) + spare


def decode_ref(qc, qr, rows, scale):
    """One sequence: qc [T, H, dc], qr [T, H, dr] or None, its cache rows [n, dc + dr] -> o [T, H, dc], lse [T, H]."""
    T, H, dc = qc.shape
    q = qc.double() if qr is None else torch.cat([qc, qr], -1).double()
    rows = rows.double()
    o, lse = torch.zeros(T, H, dc, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    for t in range(T):
        m = rows.shape[0] - (T - 1 - t)
        if m <= 0:
            continue
        x = (q[t] @ rows[:m].T) * scale
        o[t], lse[t] = torch.softmax(x, -1) @ rows[:m, :dc], torch.logsumexp(x, -1)
    return o, lse
