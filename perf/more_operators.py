"""A state-space layer's operators on cases of real use: inputs, one pass through each, and what a pass cannot do without.

Three operators, in ten kinds of case:

  norm         the residual's addition and an RMS norm, its result in 8 bits with scales (serving) or in the I/O type
  norm_train   the same step in the I/O type and its gradients
  conv         short causal convolution of packed prompts, from and to the states of their slots
  conv_step    the same for one to a few new tokens of each sequence, its states in a pool of slots
  conv_train   whole sequences and their gradients
  scan         selective state-space scan of packed prompts, or of one long prompt
  scan_step    the same for one to a few new tokens of each sequence, its states in a pool of slots
  scan_train   whole sequences and their gradients

With `own` false a pass is elementary torch operations in 32 bits; with `own` true it is the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TOP = 448.0          # the largest e4m3 value
TINY = 1e-30         # a scale's group counts as at least this large


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 24 running requests: latency is all that counts
        {"name": "norm step", "kind": "norm", "rows": 24, "D": 2048, "io": "bf16", "res": "bf16", "group": 0},
        # prompts in front of an 8-bit projection with a scale for each 128 values; the residual stream in 32 bits
        {"name": "norm prompt", "kind": "norm", "rows": 5371, "D": 4096, "io": "bf16", "res": "f32", "group": 128},
        # a training batch of 8 x 4096 tokens, and back
        {"name": "norm train", "kind": "norm_train", "rows": 32768, "D": 2048, "io": "bf16", "res": "bf16"},
        # one decoding step of 24 running requests among 40 slots
        {"name": "conv step", "kind": "conv_step", "B": 24, "T": 1, "slots": 40, "D": 4096, "W": 4, "io": "bf16"},
        # nine prompts of uneven length, each continuing from its slot's state
        {"name": "conv prompt", "kind": "conv", "B": 9, "T": 1500, "D": 2048, "W": 4, "io": "bf16", "ragged": True},
        # a training batch of 8 x 4096 tokens, and back
        {"name": "conv train", "kind": "conv_train", "B": 8, "T": 4096, "D": 2048, "W": 4, "io": "bf16", "ragged": False},
        # one token of one request: the latency of a single stream
        {"name": "scan step", "kind": "scan_step", "B": 1, "T": 1, "slots": 4, "D": 2048, "N": 16, "G": 1, "io": "bf16"},
        # a large serving batch: the states' bytes count
        {"name": "scan batch", "kind": "scan_step", "B": 512, "T": 1, "slots": 600, "D": 2048, "N": 16, "G": 1, "io": "bf16"},
        # nine prompts of uneven length, each continuing from its slot's state
        {"name": "scan prompt", "kind": "scan", "B": 9, "T": 1500, "D": 2048, "N": 16, "G": 1, "io": "bf16", "ragged": True},
        # one prompt of odd length: few channels, many tokens
        {"name": "scan long", "kind": "scan", "B": 1, "T": 16001, "D": 1536, "N": 16, "G": 1, "io": "bf16", "ragged": False},
        # a small model trained in 32 bits: odd length, few states, two groups
        {"name": "scan train f32", "kind": "scan_train", "B": 2, "T": 333, "D": 208, "N": 8, "G": 2, "io": "f32", "ragged": False},
        # a training batch of 8 x 2048 tokens, and back
        {"name": "scan train", "kind": "scan_train", "B": 8, "T": 2048, "D": 2048, "N": 16, "G": 1, "io": "bf16", "ragged": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "conv", "conv_step", "conv_train", "scan", "scan_step", "scan_train", "scan_train"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    D = 8 * _spread(rng, 8, 512)
    if kind == "norm":
        group = rng.choice([0, 32, 64, 128])
        D = max(1, D // max(group, 8)) * max(group, 8)
        return {"kind": kind, "rows": _spread(rng, 1, 8000), "D": D, "io": io, "res": rng.choice([io, "f32"]), "group": group}
    if kind == "norm_train":
        res = rng.choice([io, "f32"])
        most = 67000000 // D // (1 if res == "bf16" else 2)
        return {"kind": kind, "rows": _spread(rng, 1, most), "D": D, "io": io, "res": res}
    if kind in ("conv_step", "scan_step"):
        B = _spread(rng, 1, 500)
        c = {"kind": kind, "B": B, "T": rng.choice([1, 1, 1, 2, 3, 5, 8]), "slots": B + rng.randrange(90), "io": io}
        if kind == "conv_step":
            return dict(c, D=D, W=rng.choice([2, 3, 4]))
        return dict(c, **_states(rng, min(D, 2048)))
    B = _spread(rng, 1, 12)
    c = {"kind": kind, "B": B, "io": io, "ragged": rng.random() < 0.6}
    if kind in ("conv", "conv_train"):
        return dict(c, T=_spread(rng, 1, 32000000 // D // B // (2 if kind == "conv_train" else 1)), D=D, W=rng.choice([2, 3, 4]))
    c = dict(c, **_states(rng, min(D, 2048)))
    most = (2.6e8 if kind == "scan" else 2e8) / (c["D"] * c["N"] * B)
    return dict(c, T=_spread(rng, 1, max(1, min(16384, int(most)))))


def _states(rng, D):
    G = rng.choice([1, 1, 2, 4])
    return {"D": max(8 * G, D // (8 * G) * (8 * G)), "N": rng.choice([8, 16, 16, 32, 64]), "G": G}


# ---------------------------------------------------------------------------------------------------- lengths

def _lengths(case):
    """One length a sequence, the case's own and no seed's: T each, or uneven ones with the longest among them."""
    B, T = case["B"], case["T"]
    if not case["ragged"] or T <= 1:
        return [T] * B
    r = random.Random("%d %d" % (B, T))
    n = [max(1, int(T * r.random())) for _ in range(B)]
    n[r.randrange(B)] = T
    return n


def _rows(case):
    if "rows" in case:
        return case["rows"]
    return case["B"] * case["T"] if case["kind"].endswith("step") else sum(_lengths(case))


def work(case):
    e, kind, D, rows = 2 if case["io"] == "bf16" else 4, case["kind"], case["D"], _rows(case)
    if kind.startswith("norm"):
        r = 2 if case["res"] == "bf16" else 4
        if kind == "norm":       # x and the residual in; the new residual, 8-bit values and their scales out
            scales = rows * (D // case["group"] if case["group"] else 1)
            return {"bytes": rows * D * (e + 2 * r + 1) + 4 * (D + scales), "flops": rows * D * 7}
        # in: x, residual, then the gradients of the norm's output and of the new residual; out: norm, new residual, gradients
        gradients = e if r == e else e + r
        return {"bytes": rows * D * (e + r + e + r + e + r + gradients) + 8 * D, "flops": rows * D * 16}
    if kind.startswith("conv"):
        W, B = case["W"], case["B"]
        weights, states = 4 * D * (W + 1), B * (W - 1) * D * e
        if kind == "conv_train":
            return {"bytes": rows * D * 4 * e + 2 * weights, "flops": rows * D * (6 * W + 20)}
        return {"bytes": rows * D * 2 * e + weights + 2 * states, "flops": rows * D * (2 * W + 5)}
    N, G, B = case["N"], case["G"], case["B"]
    weights, states, ins = 4 * D * (N + 2), 4 * B * D * N, rows * (3 * D + 2 * G * N) * e
    if kind == "scan_train":     # the inputs once, y out, its gradient in, the gradients of all inputs out
        return {"bytes": 2 * ins + 2 * rows * D * e + 2 * weights, "flops": rows * D * (22 * N + 50)}
    return {"bytes": ins + rows * D * e + weights + 2 * states, "flops": rows * D * (7 * N + 15)}


# ---------------------------------------------------------------------------------------------------- inputs

def _type(io):
    return torch.bfloat16 if io == "bf16" else torch.float32


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _slots(g, case):
    """A slot for each sequence of the batch, scattered over the pool, none twice."""
    return torch.randperm(case["slots"], generator=g, device=DEV)[: case["B"]].int()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind, D, dt, rows = case["kind"], case["D"], _type(case["io"]), _rows(case)
    s = {"case": case}
    if kind.startswith("norm"):
        s["x"] = _normal(g, (rows, D), dt)
        s["res"] = _normal(g, (rows, D), _type(case["res"]), 3.0)
        s["w"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        if kind == "norm_train":
            s["dy"], s["dsum"] = _normal(g, (rows, D), dt), _normal(g, (rows, D), _type(case["res"]))
        return s
    B, step, train = case["B"], kind.endswith("step"), kind.endswith("train")
    if not step:
        n = _lengths(case)
        s["cu"] = torch.tensor([sum(n[:i]) for i in range(B + 1)], device=DEV, dtype=torch.int32) if case["ragged"] else None
    if step:
        s["slot"] = _slots(g, case)
    if kind.startswith("conv"):
        W = case["W"]
        s["x"] = _normal(g, (rows, 2 * D), dt)[:, :D]            # the value half of a projection whose other half gates
        s["w"] = torch.randn((D, W), generator=g, device=DEV) / math.sqrt(W)
        s["bias"] = 0.1 * torch.randn(D, generator=g, device=DEV)
        if step:
            s["state"] = _normal(g, (case["slots"], W - 1, D), dt)
        elif train:
            s["dy"] = _normal(g, (rows, D), dt)
        else:
            s["s0"] = _normal(g, (B, W - 1, D), dt)
        return s
    N, G, R = case["N"], case["G"], 8 * max(1, D // 128)
    s["x"] = _normal(g, (rows, D), dt)
    s["z"] = _normal(g, (rows, 2 * D), dt)[:, D:]                # the gating half of the first projection
    s["dt"] = _normal(g, (rows, D), dt, 0.5)
    bc = _normal(g, (rows, R + 2 * G * N), dt)                   # low-rank step sizes, write and read vectors side by side
    s["Bm"] = bc[:, R: R + G * N].unflatten(1, (G, N))
    s["Cm"] = bc[:, R + G * N:].unflatten(1, (G, N))
    s["A_log"] = torch.log(torch.arange(1, N + 1, device=DEV, dtype=torch.float32)) + 0.05 * torch.randn((D, N), generator=g, device=DEV)
    s["D"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
    size = torch.exp(torch.empty(D, device=DEV).uniform_(math.log(1e-3), math.log(0.1), generator=g))
    s["bias"] = size + torch.log(-torch.expm1(-size))            # softplus(bias) is a step size between 0.001 and 0.1
    if step:
        s["state"] = 0.5 * torch.randn((case["slots"], D, N), generator=g, device=DEV)
    else:
        s["h0"] = None if train else 0.5 * torch.randn((B, D, N), generator=g, device=DEV)
    if train:
        s["dy"] = _normal(g, (rows, D), dt)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _plain_norm(s):
    c = s["case"]
    dt, w = s["x"].dtype, s["w"]
    total = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    t = total.float()
    inv = torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
    y = t * inv * w
    if c["kind"] == "norm":
        parts = y.unflatten(1, (-1, c["group"] or c["D"]))
        scale = parts.abs().amax(-1).clamp(min=TINY) / TOP
        q = (parts / scale[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).flatten(1)
        return {"y": q, "scale": scale, "sum": total}
    dy = s["dy"].float()
    gw = dy * w
    d = inv * (gw - t * inv.square() * (gw * t).mean(-1, keepdim=True)) + s["dsum"].float()
    out = {"y": y.to(dt), "sum": total, "dx": d.to(dt), "dw": (dy * t * inv).sum(0)}
    if c["res"] != c["io"]:
        out["dres"] = d.to(s["res"].dtype)
    return out


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _bounds(s):
    """Rows where the sequences begin and end."""
    c = s["case"]
    if s["cu"] is None:
        first = torch.arange(c["B"], device=DEV) * c["T"]
        return first, first + c["T"]
    return s["cu"][:-1].long(), s["cu"][1:].long()


def _history(s, x, s0):
    """Each sequence's rows behind its W - 1 earlier ones (zeros if it has none), and where its own rows lie there."""
    c = s["case"]
    first, end = _bounds(s)
    W, B = c["W"], c["B"]
    row = torch.arange(x.shape[0], device=DEV)
    seq = torch.searchsorted(end, row, right=True)
    at = row + (seq + 1) * (W - 1)
    whole = torch.zeros((x.shape[0] + B * (W - 1), x.shape[1]), device=DEV)
    whole[at] = x
    if s0 is not None:
        whole[(first + torch.arange(B, device=DEV) * (W - 1))[:, None] + torch.arange(W - 1, device=DEV)] = s0
    return whole, at, end


def _plain_conv(s):
    c = s["case"]
    W, B, w, dt = c["W"], c["B"], s["w"], s["x"].dtype
    back = torch.arange(W, device=DEV) - (W - 1)
    if c["kind"] == "conv_step":
        slot = s["slot"].long()
        whole = torch.cat([s["state"][slot].float(), s["x"].float().view(B, c["T"], -1)], 1)
        pre = (whole.unfold(1, W, 1) * w).sum(-1) + s["bias"]
        s["state"][slot] = whole[:, c["T"]:].to(dt)
        return {"y": (pre * _sigmoid(pre)).flatten(0, 1).to(dt), "state": s["state"]}
    whole, at, end = _history(s, s["x"].float(), None if "s0" not in s else s["s0"].float())
    taps = whole[at[:, None] + back]                              # [rows, W, D]
    pre = (taps * w.T).sum(1) + s["bias"]
    gate = _sigmoid(pre)
    out = {"y": (pre * gate).to(dt)}
    if c["kind"] == "conv":
        last = (end + torch.arange(1, B + 1, device=DEV) * (W - 1))[:, None] + back[1:] - 1
        return dict(out, state=whole[last].to(dt))
    d = s["dy"].float() * gate * (1.0 + pre * (1.0 - gate))
    out["dw"], out["dbias"] = (d[:, None] * taps).sum(0).T, d.sum(0)
    dwhole = torch.zeros((whole.shape[0] + W - 1, whole.shape[1]), device=DEV)
    dwhole[at] = d                                                # zeros behind and between the sequences
    out["dx"] = (dwhole[at[:, None] + torch.arange(W, device=DEV)] * w.flip(1).T).sum(1).to(dt)
    return out


def _running(a, u, most):
    """h[t] = a[t] h[t-1] + u[t] over the first axis, by doubling; a is zero where a sequence begins and none is over `most` long."""
    k = 1
    while k < most:
        u = torch.cat([u[:k], torch.addcmul(u[k:], a[k:], u[:-k])])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return u


def _parts(s):
    """x, step sizes, gate, write and read vectors for every channel's group, in 32 bits."""
    c = s["case"]
    each = c["D"] // c["G"]
    v = s["dt"].float() + s["bias"]
    size = torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
    return s["x"].float(), v, size, s["z"].float(), s["Bm"].float(), s["Cm"].float(), each


def _read(h, C, each):
    """Sum over the states of h [rows, D, N] and the read vectors [rows, G, N]."""
    return (h.unflatten(1, (-1, each)) * C[:, :, None]).sum(-1).flatten(1)


def _plain_scan(s):
    c = s["case"]
    dt, A = s["x"].dtype, -torch.exp(s["A_log"])
    x, v, size, z, Bm, Cm, each = _parts(s)
    wide = lambda t: t.repeat_interleave(each, 1)  # noqa: E731
    first, end = _bounds(s)
    a = torch.exp(size[..., None] * A)
    u = (size * x)[..., None] * wide(Bm)
    if s["h0"] is not None:
        u[first] += a[first] * s["h0"]
    starts = a[first]
    a[first] = 0
    h = _running(a, u, c["T"])
    core = _read(h, Cm, each) + s["D"] * x
    gate = _sigmoid(z)
    out = {"y": (core * z * gate).to(dt)}
    if c["kind"] == "scan":
        return dict(out, state=h[end - 1])
    dy = s["dy"].float()
    g = dy * z * gate
    out["dz"] = (dy * core * gate * (1.0 + z * (1.0 - gate))).to(dt)
    out["dD"] = (g * x).sum(0)
    out["dC"] = (g[..., None] * h).unflatten(1, (-1, each)).sum(2).to(dt)
    later = torch.cat([a[1:], torch.zeros_like(a[:1])])           # a is zero at the starts: nothing crosses them
    dh = _running(later.flip(0), (g[..., None] * wide(Cm)).flip(0), c["T"]).flip(0)
    del later
    out["dB"] = (dh * (size * x)[..., None]).unflatten(1, (-1, each)).sum(2).to(dt)
    du = _read(dh, Bm, each)
    out["dx"] = (du * size + g * s["D"]).to(dt)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    a[first] = starts
    before[first] = 0
    dh *= before
    dh *= a                                                       # the gradient of size * A
    dv = (du * x + (dh * A).sum(-1)) * _sigmoid(v)
    out["dA_log"] = (dh * size[..., None]).sum(0) * A
    out["ddt"], out["dbias"] = dv.to(dt), dv.sum(0)
    return out


def _plain_scan_step(s):
    c = s["case"]
    B, T, dt, A, slot = c["B"], c["T"], s["x"].dtype, -torch.exp(s["A_log"]), s["slot"].long()
    x, v, size, z, Bm, Cm, each = _parts(s)
    a = torch.exp(size[..., None] * A).unflatten(0, (B, T))
    u = ((size * x)[..., None] * Bm.repeat_interleave(each, 1)).unflatten(0, (B, T))
    u[:, 0] += a[:, 0] * s["state"][slot]
    a[:, 0] = 0
    h = _running(a.transpose(0, 1), u.transpose(0, 1), T).transpose(0, 1)
    s["state"][slot] = h[:, -1]
    core = _read(h.flatten(0, 1), Cm, each) + s["D"] * x
    return {"y": (core * z * _sigmoid(z)).to(dt), "state": s["state"]}


# ---------------------------------------------------------------------------------------------------- the library's calls

def _own_norm(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    rows, D, train, other = s["x"].shape[0], c["D"], c["kind"] == "norm_train", c["res"] != c["io"]
    if "plan" not in s:     # what a user's program keeps for its passes
        s["plan"] = gdn.make_norm(rows, D, c["io"], res=c["res"], out=c["io"] if train else "e4m3", group=0 if train else c["group"], eps=EPS)
        s["ws"] = torch.empty(gdn.gdn_norm_workspace_bytes(s["plan"]), dtype=torch.uint8, device=DEV) if train else None
    total = torch.empty_like(s["res"])
    if not train:
        y = torch.empty((rows, D), dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.empty((rows, D // c["group"] if c["group"] else 1), device=DEV)
        gdn.check(gdn.gdn_norm_fwd(s["plan"], s["x"], s["res"], s["w"], y, scale, total))
        return {"y": y, "scale": scale, "sum": total}
    y, dx, dw = torch.empty_like(s["x"]), torch.empty_like(s["x"]), torch.empty(D, device=DEV)
    dres = torch.empty_like(s["res"]) if other else None
    gdn.check(gdn.gdn_norm_fwd(s["plan"], s["x"], s["res"], s["w"], y, None, total))
    gdn.check(gdn.gdn_norm_bwd(s["plan"], total, s["w"], s["dy"], s["dsum"], dx, dres, dw, s["ws"]))
    out = {"y": y, "sum": total, "dx": dx, "dw": dw}
    return dict(out, dres=dres) if other else out


def _own_conv(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    kind, B, T, D, W, rows, dt = c["kind"], c["B"], c["T"], c["D"], c["W"], s["x"].shape[0], s["x"].dtype
    y = torch.empty((rows, D), dtype=dt, device=DEV)
    if kind == "conv_step":
        if "plan" not in s:
            s["plan"] = gdn.make_conv_step(B, T, D, W, c["slots"], c["io"])
        gdn.check(gdn.gdn_conv_step(s["plan"], s["x"], s["w"], s["bias"], s["state"], s["slot"], None, y))
        return {"y": y, "state": s["state"]}
    if "plan" not in s:
        s["plan"] = gdn.make_conv(B, T, D, W, c["io"], rows=rows)
        s["ws"] = torch.empty(gdn.gdn_conv_workspace_bytes(s["plan"]), dtype=torch.uint8, device=DEV) if kind == "conv_train" else None
    state = torch.empty_like(s["s0"]) if kind == "conv" else None
    gdn.check(gdn.gdn_conv_fwd(s["plan"], s["x"], s["w"], s["bias"], s["cu"], s.get("s0"), y, state))
    if kind == "conv":
        return {"y": y, "state": state}
    dx, dw, dbias = torch.empty((rows, D), dtype=dt, device=DEV), torch.empty((D, W), device=DEV), torch.empty(D, device=DEV)
    gdn.check(gdn.gdn_conv_bwd(s["plan"], s["x"], s["w"], s["bias"], s["cu"], None, s["dy"], None, dx, dw, dbias, None, s["ws"]))
    return {"y": y, "dx": dx, "dw": dw, "dbias": dbias}


def _own_scan(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    kind, B, T, D, N, G, rows, dt = c["kind"], c["B"], c["T"], c["D"], c["N"], c["G"], s["x"].shape[0], s["x"].dtype
    y = torch.empty((rows, D), dtype=dt, device=DEV)
    args = (s["x"], s["dt"], s["z"], s["Bm"], s["Cm"], s["A_log"], s["D"], s["bias"])
    if kind == "scan_step":
        if "plan" not in s:
            s["plan"] = gdn.make_scan_step(B, T, D, N, c["slots"], G, c["io"])
        gdn.check(gdn.gdn_scan_step(s["plan"], *args, s["state"], s["slot"], None, y))
        return {"y": y, "state": s["state"]}
    train = kind == "scan_train"
    if "plan" not in s:
        p = s["plan"] = gdn.make_scan(B, T, D, N, G, c["io"], rows=rows)
        s["ws"] = torch.empty(gdn.gdn_scan_workspace_bytes(p, int(train)), dtype=torch.uint8, device=DEV)
        s["saved"] = torch.empty(gdn.gdn_scan_saved_bytes(p), dtype=torch.uint8, device=DEV) if train else None
    state = None if train else torch.empty_like(s["h0"])
    gdn.check(gdn.gdn_scan_fwd(s["plan"], *args, s["cu"], s["h0"], y, state, s["saved"], s["ws"]))
    if not train:
        return {"y": y, "state": state}
    dx, ddt, dz = (torch.empty((rows, D), dtype=dt, device=DEV) for _ in range(3))
    dB, dC = (torch.empty((rows, G, N), dtype=dt, device=DEV) for _ in range(2))
    dA_log, dD, dbias = torch.empty((D, N), device=DEV), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    gdn.check(gdn.gdn_scan_bwd(s["plan"], *args, s["cu"], s["saved"], s["dy"], None, dx, ddt, dz, dB, dC, dA_log, dD, dbias, None,
                               s["ws"]))
    return {"y": y, "dx": dx, "ddt": ddt, "dz": dz, "dB": dB, "dC": dC, "dA_log": dA_log, "dD": dD, "dbias": dbias}


def run(state):
    kind = state["case"]["kind"]
    if kind.startswith("norm"):
        return _own_norm(state) if own else _plain_norm(state)
    if kind.startswith("conv"):
        return _own_conv(state) if own else _plain_conv(state)
    if own:
        return _own_scan(state)
    return _plain_scan_step(state) if kind == "scan_step" else _plain_scan(state)


# ---------------------------------------------------------------------------------------------------- the definitions in 64 bits

def _silu(x):
    return x / (1 + torch.exp(-x))


def _exact_norm(case, s):
    D = case["D"]
    total = (s["x"].double() + s["res"].double())
    kept = total.to(s["res"].dtype).double().requires_grad_()      # the norm sees the residual as it is kept
    w = s["w"].double().requires_grad_()
    y = kept / ((kept ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w
    if case["kind"] == "norm":
        group = case["group"] or D
        v = y.detach().view(-1, D // group, group)
        scale = torch.clamp(v.abs().max(-1).values, min=TINY) / TOP
        return {"y": (v / scale.unsqueeze(-1)).view(-1, D), "scale": scale, "sum": total}
    dw, d = torch.autograd.grad((y * s["dy"].double()).sum() + (kept * s["dsum"].double()).sum(), [w, kept])
    out = {"y": y.detach(), "sum": total, "dx": d, "dw": dw}
    return dict(out, dres=d) if case["res"] != case["io"] else out


def _exact_conv(case, s):
    W, B, D, kind = case["W"], case["B"], case["D"], case["kind"]
    n = [case["T"]] * B if kind == "conv_step" else _lengths(case)
    train = kind == "conv_train"
    x, w, b = s["x"].double().requires_grad_(train), s["w"].double().requires_grad_(train), s["bias"].double().requires_grad_(train)
    if kind == "conv_step":
        pool, slot = s["state"].double(), [int(k) for k in s["slot"]]
    at, ys, states = 0, [], []
    for i, length in enumerate(n):
        if kind == "conv_step":
            before = pool[slot[i]].clone()
        else:
            before = torch.zeros(W - 1, D, dtype=torch.float64, device=DEV) if train else s["s0"][i].double()
        seq = torch.cat([before, x[at: at + length]])
        at += length
        ys.append(_silu(b + sum(w[:, k] * seq[k: k + length] for k in range(W))))
        states.append(seq[length:].detach())
    y = torch.cat(ys)
    if not train:
        if kind == "conv":
            return {"y": y, "state": torch.stack(states)}
        for k, v in zip(slot, states):
            pool[k] = v
        return {"y": y, "state": pool}
    dx, dw, db = torch.autograd.grad((y * s["dy"].double()).sum(), [x, w, b])
    return {"y": y.detach(), "dx": dx, "dw": dw, "dbias": db}


def _recur(h, p, each):
    """One token: the state [B, D, N] and the token's p (x, dt, z, B, C of all sequences) to the new state and the output."""
    x, v, z, b, c, A_log, skip, bias = p
    size = torch.nn.functional.softplus(v + bias, threshold=100)
    b, c = (t.repeat_interleave(each, 1) for t in (b, c))
    h = torch.exp(-size.unsqueeze(-1) * torch.exp(A_log)) * h + (size * x).unsqueeze(-1) * b
    return h, ((h * c).sum(-1) + skip * x) * _silu(z)


def _exact_scan(case, s):
    kind, B, T, D, N, G = case["kind"], case["B"], case["T"], case["D"], case["N"], case["G"]
    n = [T] * B if kind == "scan_step" else _lengths(case)
    train = kind == "scan_train"
    if train and (T * B * D * N > 6e8 or T > 5000):
        return None
    first = [sum(n[:i]) for i in range(B)]
    names = ("x", "dt", "z", "Bm", "Cm")
    if kind == "scan_step":
        h = s["state"].double()[s["slot"].long()]
    else:
        h = torch.zeros(B, D, N, dtype=torch.float64, device=DEV) if train else s["h0"].double()
    order = sorted(range(B), key=lambda i: -n[i])                  # longest first: those still running are a front part
    h, start = h[order], torch.tensor([first[i] for i in order], device=DEV)
    running = [sum(1 for i in range(B) if n[i] > t) for t in range(T)]
    weights = [s[k].double() for k in ("A_log", "D", "bias")]
    rows = sum(n)
    if not train:
        y, x = torch.zeros(rows, D, dtype=torch.float64, device=DEV), [s[k].double() for k in names]
        for t in range(T):
            m = running[t]
            at = start[:m] + t
            h[:m], y[at] = _recur(h[:m], [v[at] for v in x] + weights, D // G)
        if kind == "scan_step":
            pool = s["state"].double()
            pool[s["slot"].long()[order]] = h
            return {"y": y, "state": pool}
        out = torch.empty_like(h)
        out[order] = h
        return {"y": y, "state": out}
    # gradients from torch's reverse mode, a block of one group's channels at a time
    x = [s[k].double() for k in names]
    grads = [torch.zeros_like(v) for v in x + weights]
    y, each = torch.zeros(rows, D, dtype=torch.float64, device=DEV), D // G
    block = max(8, min(each, int(2.5e8 / (rows * N))))
    for g in range(G):
        for d0 in range(g * each, (g + 1) * each, block):
            ch = slice(d0, min(d0 + block, (g + 1) * each))
            place = [(slice(None), ch)] * 3 + [(slice(None), slice(g, g + 1))] * 2 + [(ch,)] * 3
            leaf = [v[p].clone().requires_grad_() for v, p in zip(x + weights, place)]
            seqs = [leaf[k][(start[:, None] + torch.arange(T, device=DEV)).clamp(max=rows - 1)].unbind(1) for k in range(5)]
            state, loss = h[:, ch], 0.0
            for t in range(T):
                m = running[t]
                state, out = _recur(state[:m], [q[t][:m] for q in seqs] + leaf[5:], ch.stop - ch.start)
                at = start[:m] + t
                y[at, ch] = out.detach()
                loss = loss + (out * s["dy"][at, ch].double()).sum()
            for total, p, d in zip(grads, place, torch.autograd.grad(loss, leaf)):
                total[p] += d
    return dict(zip(("y", "dx", "ddt", "dz", "dB", "dC", "dA_log", "dD", "dbias"), [y] + grads))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("norm"):
        return _exact_norm(case, s)
    return _exact_conv(case, s) if case["kind"].startswith("conv") else _exact_scan(case, s)
