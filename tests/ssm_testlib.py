"""The state-space operators in 64 bits on the CPU, and seeded inputs for them: what the tests of ``gdn_norm_*``,
``gdn_conv_*`` and ``gdn_scan_*`` compare against.

The definitions are written per sequence and token with plain torch operations; gradients come from torch's reverse mode
on them.  `close` allows two things, both fixed by arithmetic:

* the result's one rounding to its type, at most half a step: eps / 2 of the value (bf16 2^-8, e4m3 2^-4, f32 2^-24);
* the fp32 arithmetic before it, `work` of the result's largest value.  Norm and convolution: sums of at most a few
  thousand fp32 products of mixed sign, and functions good to 2^-21: 1e-5.  The scan: each step's factor is exp2 of a
  rounded product, good to 2^-22 + 2^-24 |argument|, and the test inputs' step sizes (0.01 and up, rates 0.8 and up) forget
  a state over at most 125 tokens, so a state is within 125 x 2^-21.5 = 4.2e-5 of the largest one; a gradient multiplies
  two such sequences: 9e-5.
"""
import math

import torch

import linear_attention_recurrence_delta_gb300 as gdn

EPS = 1e-6
WORK = {"sum": 1e-5, "scan": 4.2e-5, "scan_bwd": 9e-5}


def tdtype(io):
    return torch.float32 if io == "f32" else torch.bfloat16


def close(got, ref, what, name, seen=None):
    """`seen`: rows that count (the others may hold anything)."""
    if seen is not None:
        got, ref = got.cpu()[seen], ref[seen]
    step = torch.finfo(got.dtype).eps / 2
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: non-finite values"
    if ref.numel() == 0:
        return
    top = ref.abs().max().item()
    over = ((got - ref).abs() - step * ref.abs()).max().item()
    assert over <= WORK[what] * top, f"{name}: {over / max(top, 1e-300):.2e} of the largest value over a rounding"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, io, std=1.0):
    """Values exactly representable in the I/O type, as a CPU tensor of it."""
    return (torch.randn(shape, generator=g) * std).to(tdtype(io))


def nan(shape, dtype):
    return torch.full(shape, math.nan, dtype=dtype, device="cuda")


def offsets(lens, gap=0):
    """Row offsets of packed sequences behind `gap` rows of nobody."""
    return torch.tensor([gap + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


# ---------------------------------------------------------------- convolution

def conv_ref(x, w, bias, s0, silu):
    """One sequence [n, D] behind its state [W - 1, D]: outputs and the new state."""
    n, W = x.shape[0], w.shape[1]
    seq = torch.cat([s0, x])
    y = sum(w[:, k] * seq[k: k + n] for k in range(W))
    y = y if bias is None else y + bias
    return (y * torch.sigmoid(y) if silu else y), seq[n:]


def conv_all(x, w, bias, s0, lens, silu, gap=0):
    """Packed rows -> y (zeros in rows of nobody), states."""
    ys, states, at = [x.new_zeros(gap, x.shape[1])], [], gap
    for b, n in enumerate(lens):
        y, s = conv_ref(x[at: at + n], w, bias, s0[b], silu)
        ys.append(y)
        states.append(s)
        at += n
    ys.append(x.new_zeros(x.shape[0] - at, x.shape[1]))
    return torch.cat(ys), torch.stack(states)


# ---------------------------------------------------------------- scan

def scan_one(x, dt, z, Bm, Cm, A_log, skip, bias, h, softplus):
    """One sequence: x, dt, z [n, D], Bm, Cm [n, G, N], h [D, N] -> y, last state."""
    each, ys = x.shape[1] // Bm.shape[1], []
    for t in range(x.shape[0]):
        v = dt[t] if bias is None else dt[t] + bias
        delta = torch.nn.functional.softplus(v, threshold=100) if softplus else v
        b, c = (m[t].repeat_interleave(each, 0) for m in (Bm, Cm))
        h = torch.exp(-delta[:, None] * torch.exp(A_log)) * h + (delta * x[t])[:, None] * b
        y = (h * c).sum(-1)
        if skip is not None:
            y = y + skip * x[t]
        ys.append(y if z is None else y * z[t] * torch.sigmoid(z[t]))
    return (torch.stack(ys) if ys else x.new_zeros(0, x.shape[1])), h


def scan_all(i, lens, softplus=True, gap=0):
    """Packed inputs (dict of 64-bit tensors or None) -> y (zeros in rows of nobody), last states."""
    rows, D = i["x"].shape
    ys, states, at = [i["x"].new_zeros(gap, D)], [], gap
    for b, n in enumerate(lens):
        part = [None if i[k] is None else i[k][at: at + n] for k in ("x", "dt", "z", "Bm", "Cm")]
        y, h = scan_one(*part, i["A_log"], i["skip"], i["bias"], i["h0"][b], softplus)
        ys.append(y)
        states.append(h)
        at += n
    ys.append(i["x"].new_zeros(rows - at, D))
    return torch.cat(ys), torch.stack(states)


def scan_inputs(seed, lens, D, N, G, io, gate=True, skip=True, bias=True, softplus=True, h0=True, gap=0, pad=0):
    """Inputs on the CPU: x, z halves and Bm, Cm slices of wider rows, as projections leave them."""
    g, rows = gen(seed), sum(lens) + gap + pad
    xz, bc = normal(g, (rows, 2 * D), io), normal(g, (rows, 16 + 2 * G * N), io)
    raw = normal(g, (rows, D), io, 0.5)
    size = torch.exp(torch.empty(D).uniform_(math.log(0.03), math.log(0.3), generator=g))
    if not softplus:
        raw = (raw.abs() * 0.1 + 0.02).to(tdtype(io))
    elif bias:
        raw = raw.clamp(min=-0.8)
    else:
        raw = (raw - 2.0).clamp(min=-3.5).to(tdtype(io))
    return {"x": xz[:, :D], "z": xz[:, D:] if gate else None, "dt": raw,
            "Bm": bc[:, 16: 16 + G * N].unflatten(1, (G, N)), "Cm": bc[:, 16 + G * N:].unflatten(1, (G, N)),
            "A_log": torch.log(torch.arange(1, N + 1).float()) + 0.05 * torch.randn((D, N), generator=g).clamp(-3, 3),
            "skip": 1 + 0.1 * torch.randn(D, generator=g) if skip else None,
            "bias": (size + torch.log(-torch.expm1(-size)) if softplus else 0.01 + 0.0 * size) if bias else None,
            "h0": 0.5 * torch.randn((len(lens), D, N), generator=g) if h0 else None,
            "dy": normal(g, (rows, D), io), "dhT": torch.randn((len(lens), D, N), generator=g)}


ORDER = ("x", "dt", "z", "Bm", "Cm", "A_log", "skip", "bias")


def cuda(i):
    """The inputs on the GPU, with slices still slices."""
    out = {}
    for k, t in i.items():
        out[k] = None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)
    return out


def scan_run(i, lens, io, softplus=True, cu=None, T=None, train=False, dhT=True, stream=None):
    """gdn_scan_fwd (and gdn_scan_bwd) on device inputs; every output starts as NaN."""
    rows, D = i["x"].shape
    G, N = i["Bm"].shape[1:]
    B, dt = len(lens), tdtype(io)
    s = gdn.make_scan(B, max(lens) if T is None else T, D, N, G, io, softplus, rows)
    ws, saved = (torch.full((n,), 255, dtype=torch.uint8, device="cuda")      # NaN, to see that all is written before it is read
                 for n in (gdn.gdn_scan_workspace_bytes(s, 0), gdn.gdn_scan_saved_bytes(s)))
    args = [i[k] for k in ORDER]
    out = {"y": nan((rows, D), dt), "hT": nan((B, D, N), torch.float32)}
    gdn.check(gdn.gdn_scan_fwd(s, *args, cu, i["h0"], out["y"], out["hT"], saved if train else None, ws, stream=stream))
    if not train:
        return out
    wb = torch.full((gdn.gdn_scan_workspace_bytes(s, 1),), 255, dtype=torch.uint8, device="cuda")
    grad = {k: None if i[k] is None else nan(i[k].shape, dt if k in ("x", "dt", "z", "Bm", "Cm") else torch.float32)
            for k in ORDER + ("h0",)}
    gdn.check(gdn.gdn_scan_bwd(s, *args, cu, saved, i["dy"], i["dhT"] if dhT else None, *[grad[k] for k in ORDER], grad["h0"], wb,
                               stream=stream))
    out.update({"d" + k: t for k, t in grad.items()})
    return out


def scan_grads(i, lens, softplus=True, gap=0, dhT=True):
    """y, last states and gradients in 64 bits."""
    names = [k for k in ORDER + ("h0",) if i[k] is not None]
    x = {k: None if t is None else t.double() for k, t in i.items()}
    for k in names:
        x[k] = x[k].clone().requires_grad_()
    if x["h0"] is None:
        x["h0"] = torch.zeros(i["dhT"].shape, dtype=torch.float64)
    y, hT = scan_all(x, lens, softplus, gap)
    loss = (y * x["dy"]).sum() + ((hT * x["dhT"]).sum() if dhT else 0.0)
    if not loss.requires_grad:
        return y, hT, {}
    grads = torch.autograd.grad(loss, [x[k] for k in names], allow_unused=True)
    return y.detach(), hT.detach(), {k: torch.zeros_like(x[k]) if d is None else d for k, d in zip(names, grads)}
