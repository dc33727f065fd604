"""The latent-attention operators on cases of real use: inputs, one pass through each, and what a pass cannot do without.

Three operators, in five kinds of case:

  prep        new tokens enter a paged latent cache: RMS norm of the latent, rotation of the shared position key and of
              the queries' position part, rows written at the places that a block table gives
  prep_train  the same step on dense rows and its gradients
  decode      one to a few new tokens of each sequence attend over its paged latent cache (absorbed form)
  fwd         causal attention over expanded keys and values (prompts, whole or in chunks after a cached prefix)
  train       that attention with the gradients of all its inputs

With `own` false a pass is elementary torch operations in 32 bits; with `own` true it is the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 24 running requests: each writes one cache row; latency is all that counts
        {"name": "prep step", "kind": "prep", "B": 24, "most": 1, "H": 16, "dc": 256, "dn": 64, "dr": 64, "page": 64,
         "past": 1500, "io": "bf16", "pairs": False},
        # six prompts of uneven length enter a cache of wide latents in small pages
        {"name": "prep prompt", "kind": "prep", "B": 6, "most": 2300, "H": 16, "dc": 512, "dn": 128, "dr": 64, "page": 16,
         "past": 0, "io": "bf16", "pairs": True},
        # a training batch of 8 x 4096 tokens through the norm and the rotation, and back
        {"name": "prep train", "kind": "prep_train", "N": 32768, "H": 16, "dc": 256, "dn": 64, "dr": 64, "io": "bf16",
         "pairs": False},
        # one request, one token: the latency of a single stream
        {"name": "decode one", "kind": "decode", "B": 1, "most": 777, "T": 1, "H": 16, "dc": 256, "dr": 64, "page": 64,
         "ragged": False, "io": "bf16"},
        # a serving batch of 64 slots with lengths up to 4096, some slots without a request
        {"name": "decode batch", "kind": "decode", "B": 64, "most": 4096, "T": 1, "H": 16, "dc": 256, "dr": 64, "page": 64,
         "ragged": True, "io": "bf16"},
        # eight long contexts of 32768 tokens with wide latents: the cache's bytes count
        {"name": "decode long", "kind": "decode", "B": 8, "most": 32768, "T": 1, "H": 16, "dc": 512, "dr": 64, "page": 64,
         "ragged": False, "io": "bf16"},
        # checking four drafted tokens of each request with 40 heads: 160 query rows share each cache row
        {"name": "decode draft", "kind": "decode", "B": 32, "most": 6000, "T": 4, "H": 40, "dc": 512, "dr": 64, "page": 16,
         "ragged": True, "io": "bf16"},
        # a handful of short prompts, packed: launch and tail latency
        {"name": "prompt short", "kind": "fwd", "B": 12, "Tq": 700, "Tk": 700, "H": 16, "Hkv": 4, "dn": 64, "dr": 64,
         "dv": 128, "ragged": True, "io": "bf16"},
        # the last 2048 tokens of two prompts of 8192: queries against a longer prefix
        {"name": "prompt chunk", "kind": "fwd", "B": 2, "Tq": 2048, "Tk": 8192, "H": 16, "Hkv": 4, "dn": 64, "dr": 64,
         "dv": 128, "ragged": False, "io": "bf16"},
        # a small model trained in 32 bits, odd length and narrow heads
        {"name": "train f32", "kind": "train", "B": 2, "Tq": 333, "Tk": 333, "H": 4, "Hkv": 2, "dn": 32, "dr": 16, "dv": 48,
         "ragged": False, "io": "f32"},
        # packed documents of uneven length, a key and a value for every head, wide keys
        {"name": "train packed", "kind": "train", "B": 6, "Tq": 1900, "Tk": 1900, "H": 16, "Hkv": 16, "dn": 128, "dr": 64,
         "dv": 128, "ragged": True, "io": "bf16"},
        # the training step of the 16-head layers: 8 x 4096 tokens, four key heads
        {"name": "train full", "kind": "train", "B": 8, "Tq": 4096, "Tk": 4096, "H": 16, "Hkv": 4, "dn": 64, "dr": 64,
         "dv": 128, "ragged": False, "io": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    n = 3072
    while n == 3072:
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["prep", "prep_train", "decode", "decode", "fwd", "train"])
    io = "f32" if rng.random() < 0.2 else "bf16"
    dc, dr = rng.choice([64, 128, 192, 256, 384, 512]), rng.choice([32, 64])
    if kind == "prep":
        return {"kind": kind, "B": _spread(rng, 1, 100), "most": rng.choice([1, _spread(rng, 2, 1500)]),
                "H": rng.choice([1, 4, 12, 16, 40]), "dc": dc, "dn": rng.choice([32, 64, 128]), "dr": dr,
                "page": rng.choice([16, 32, 64, 128]), "past": _spread(rng, 1, 4000), "io": io, "pairs": rng.random() < 0.5}
    if kind == "prep_train":
        return {"kind": kind, "N": _spread(rng, 1, 32768), "H": rng.choice([1, 4, 12, 16, 40]), "dc": dc,
                "dn": rng.choice([32, 64, 128]), "dr": dr, "io": io, "pairs": rng.random() < 0.5}
    if kind == "decode":
        B = _spread(rng, 1, 100)
        top = max(64, min(32768, 300000 // B)) if io == "bf16" else max(64, min(4096, 20000 // B))
        return {"kind": kind, "B": B, "most": _spread(rng, 1, top), "T": rng.choice([1, 1, 1, 2, 3, 4]),
                "H": rng.choice([4, 12, 16, 40, 64]), "dc": dc, "dr": dr, "page": rng.choice([16, 32, 64, 128]),
                "ragged": rng.random() < 0.7, "io": io}
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4])
    dn, dr, dv = rng.choice([(32, 32, 64), (64, 64, 128), (96, 32, 128), (128, 64, 128), (56, 16, 56), (64, 0, 64)])
    B = _spread(rng, 1, 12)
    top = int(math.sqrt((4e8 if io == "bf16" else 1.2e7) / (B * H)))
    Tk = _spread(rng, 1, max(1, min(8192, top)))
    Tq = Tk if kind == "train" or rng.random() < 0.5 else max(1, min(Tk, _spread(rng, 1, Tk)))
    return {"kind": kind, "B": B, "Tq": Tq, "Tk": Tk, "H": H, "Hkv": Hkv, "dn": dn, "dr": dr, "dv": dv,
            "ragged": rng.random() < 0.6, "io": io}


# ---------------------------------------------------------------------------------------------------- lengths

def _lengths(case, what, most):
    """One length a sequence, the case's own and no seed's: `most` each, or uneven ones with the longest among them."""
    B = case["B"]
    if not case.get("ragged", True) or most <= 1:
        return [most] * B
    r = random.Random("%s %d %d" % (what, B, most))
    n = [max(1, int(most * r.random())) for _ in range(B)]
    n[r.randrange(B)] = most
    return n


def _attn_lengths(case):
    nk = _lengths(case, "keys", case["Tk"])
    if case["Tq"] == case["Tk"]:
        return nk, nk
    return [max(1, min(case["Tq"], k * case["Tq"] // case["Tk"])) for k in nk], nk


def _cache_lengths(case):
    n = _lengths(case, "cache", case["most"])
    if case["ragged"] and case["B"] >= 4:     # slots of the batch that hold no request
        n[[i for i in range(case["B"]) if n[i] < case["most"] or n.count(case["most"]) > 1][0]] = 0
    return n


def _pairs(nq, nk):
    """Pairs of a query and a key that it sees."""
    return sum(sum(max(0, k - q + i + 1) for i in range(q)) if k < q else q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    kind = case["kind"]
    if kind in ("prep", "prep_train"):
        N = case["N"] if kind == "prep_train" else sum(_lengths(case, "new", case["most"]))
        row = case["dc"] + case["dr"] + case["H"] * case["dr"]
        if kind == "prep":
            return {"bytes": 2 * N * row * e + N * case["dr"] * 4, "flops": N * (4 * case["dc"] + 3 * (case["H"] + 1) * case["dr"])}
        return {"bytes": 4 * N * row * e + N * case["dc"] * e + N * case["dr"] * 4,
                "flops": N * (14 * case["dc"] + 6 * (case["H"] + 1) * case["dr"])}
    if kind == "decode":
        n, T, H, dc, dr = _cache_lengths(case), case["T"], case["H"], case["dc"], case["dr"]
        seen = sum(max(0, k - t) for k in n for t in range(T))
        return {"bytes": sum(n) * (dc + dr) * e + case["B"] * T * H * (2 * dc + dr) * e, "flops": 2 * seen * H * (2 * dc + dr)}
    nq, nk = _attn_lengths(case)
    H, Hkv, dn, dr, dv = (case[k] for k in ("H", "Hkv", "dn", "dr", "dv"))
    q, k, o = sum(nq) * H * (dn + dr), sum(nk) * (Hkv * (dn + dv) + dr), sum(nq) * H * dv
    pairs = _pairs(nq, nk) * H
    if kind == "fwd":
        return {"bytes": (q + k + o) * e, "flops": 2 * pairs * (dn + dr + dv)}
    return {"bytes": (2 * q + 2 * k + 2 * o) * e, "flops": 2 * pairs * (4 * (dn + dr) + 3 * dv)}


# ---------------------------------------------------------------------------------------------------- inputs

def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _rotation(rows, dr):
    """Rows of cos and sin of position times 10000^(-2 i / dr)."""
    f = torch.arange(dr // 2, device=DEV, dtype=torch.float64)
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * torch.pow(10000.0, -2.0 * f / dr)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _table(g, n, page):
    """A block table whose pages lie scattered in the cache, some pages of it nobody's; entries past a sequence's end are -1."""
    per = [-(-k // page) for k in n]
    free = torch.randperm(sum(per) + 5, generator=g, device=DEV).int()
    width = max(1, max(per))
    at = torch.tensor([sum(per[:i]) for i in range(len(per))], device=DEV)[:, None] + torch.arange(width, device=DEV)
    used = torch.arange(width, device=DEV) < torch.tensor(per, device=DEV)[:, None]
    t = torch.where(used, free[at.clamp(max=sum(per) + 4)], torch.full_like(at, -1, dtype=torch.int32))
    return t.contiguous(), sum(per) + 5


def _offsets(n):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], device=DEV, dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    s = {"case": case}
    kind = case["kind"]
    if kind in ("prep", "prep_train"):
        dc, dr, dn, H = case["dc"], case["dr"], case["dn"], case["H"]
        if kind == "prep":
            new = _lengths(case, "new", case["most"])
            past = [case["past"] * (i + 1) // len(new) for i in range(len(new))]
            N = sum(new)
            s["pos"] = torch.tensor([p + i for n, p in zip(new, past) for i in range(n)], device=DEV, dtype=torch.int32)
            s["seq"] = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], device=DEV, dtype=torch.int32)
            s["table"], pages = _table(g, [n + p for n, p in zip(new, past)], case["page"])
            s["cache"] = _normal(g, (pages, case["page"], dc + dr), dt)
            rows = max(n + p for n, p in zip(new, past))
        else:
            N, rows = case["N"], 4096
            s["pos"] = (torch.arange(N, device=DEV) % rows).int()
            s["dlat"], s["dkr"] = _normal(g, (N, dc), dt), _normal(g, (N, dr), dt)
            s["dqr"] = _normal(g, (N, H, dn + dr), dt)[..., dn:]     # a slice of the whole query's gradient
        s["rot"] = _rotation(rows, dr)
        s["kv"] = _normal(g, (N, dc + dr), dt, 0.7)                  # the down projection's rows
        s["w"] = 1.0 + 0.2 * torch.randn(dc, generator=g, device=DEV)
        s["qr"] = _normal(g, (N, H, dn + dr), dt)[..., dn:]          # a slice of the whole query
        return s
    if kind == "decode":
        n, T, H, dc, dr = _cache_lengths(case), case["T"], case["H"], case["dc"], case["dr"]
        s["table"], pages = _table(g, n, case["page"])
        s["cache"] = _normal(g, (pages, case["page"], dc + dr), dt)
        s["lens"] = torch.tensor(n, device=DEV, dtype=torch.int32)
        s["qc"] = _normal(g, (case["B"], T, H, dc), dt, 1.5 * math.sqrt(64.0 / dc))   # absorbed queries
        s["qr"] = _normal(g, (case["B"], T, H, dr), dt, 1.5)
        s["scale"] = 1.0 / math.sqrt(64.0 + dr)
        return s
    nq, nk = _attn_lengths(case)
    H, Hkv, dn, dr, dv = (case[k] for k in ("H", "Hkv", "dn", "dr", "dv"))
    q = _normal(g, (sum(nq), H, dn + dr), dt, 1.5)
    kv = _normal(g, (sum(nk), Hkv, dn + dv), dt)                     # the up projection's rows: key and value side by side
    s["qn"], s["qr"] = q[..., :dn], q[..., dn:] if dr else None
    s["kn"], s["v"] = kv[..., :dn], kv[..., dn:]
    s["kr"] = _normal(g, (sum(nk), dr), dt) if dr else None
    s["cu_q"], s["cu_k"] = (_offsets(nq), _offsets(nk)) if case["ragged"] else (None, None)
    s["scale"] = 1.0 / math.sqrt(dn + dr)
    if kind == "train":
        s["dO"] = _normal(g, (sum(nq), H, dv), dt)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, pairs, back=False):
    sin = -sin if back else sin
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :h], x[..., h:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)


def _plain_prep(s):
    c = s["case"]
    dc, dr = c["dc"], c["dr"]
    dt, kv, q = s["kv"].dtype, s["kv"].float(), s["qr"].float()
    r = s["rot"][s["pos"].long()]
    cos, sin = r[:, : dr // 2], r[:, dr // 2:]
    x = kv[:, :dc]
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    lat = (x * inv * s["w"]).to(dt)
    kr = _rotate(kv[:, dc:], cos, sin, c["pairs"]).to(dt)
    qr = _rotate(q, cos[:, None], sin[:, None], c["pairs"]).to(dt)
    if c["kind"] == "prep":
        pos = s["pos"].long()
        page = s["table"][s["seq"].long(), pos // c["page"]].long()
        s["cache"][page, pos % c["page"]] = torch.cat([lat, kr], 1)
        return {"cache": s["cache"], "qr": qr}
    dy = s["dlat"].float()
    gw = dy * s["w"]
    dx = inv * (gw - x * inv.square() * (gw * x).mean(-1, keepdim=True))
    dk = _rotate(s["dkr"].float(), cos, sin, c["pairs"], back=True)
    dq = _rotate(s["dqr"].float(), cos[:, None], sin[:, None], c["pairs"], back=True)
    return {"lat": lat, "kr": kr, "qr": qr, "dkv": torch.cat([dx, dk], 1).to(dt), "dw": (dy * x * inv).sum(0), "dqr": dq.to(dt)}


def _softmax(scores, seen):
    """Weights over the last axis of what is seen; zero in a row that sees nothing."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(s):
    c = s["case"]
    B, T, H, dc = c["B"], c["T"], c["H"], c["dc"]
    rows = s["cache"][s["table"].clamp(min=0).long()].flatten(1, 2).float()      # [B, places, dc + dr]
    q = torch.cat([s["qc"], s["qr"]], -1).float().flatten(1, 2)                  # [B, T * H, dc + dr]
    at = torch.arange(rows.shape[1], device=DEV)
    last = s["lens"][:, None] - (T - 1 - torch.arange(T, device=DEV))            # what token t sees ends here
    seen = (at < last[..., None])[:, :, None].expand(-1, -1, H, -1).flatten(1, 2)
    p = _softmax(torch.matmul(q, rows.transpose(1, 2)) * s["scale"], seen)
    return torch.matmul(p, rows[..., :dc]).view(B, T, H, dc).to(s["qc"].dtype)


def _padded(x, cu, B, T):
    """Packed rows [N, heads, d] as [B, heads, T, d] in 32 bits, with where they are and which are real."""
    if cu is None:
        cu = torch.arange(B + 1, device=DEV, dtype=torch.int32) * T
    cu = cu.long()
    at = cu[:-1, None] + torch.arange(T, device=DEV)
    real = at < cu[1:, None]
    return x.float()[at.clamp(max=x.shape[0] - 1)].transpose(1, 2), real, cu[1:] - cu[:-1]


def _plain_attention(s):
    c = s["case"]
    B, Tq, Tk, H, Hkv, dn = (c[k] for k in ("B", "Tq", "Tk", "H", "Hkv", "dn"))
    G, dt = H // Hkv, s["qn"].dtype
    q = torch.cat([s["qn"], s["qr"]], -1) if c["dr"] else s["qn"]
    k = torch.cat([s["kn"], s["kr"][:, None].expand(-1, Hkv, -1)], -1) if c["dr"] else s["kn"]
    q, realq, nq = _padded(q, s["cu_q"], B, Tq)
    k, realk, nk = _padded(k, s["cu_k"], B, Tk)
    v = _padded(s["v"], s["cu_k"], B, Tk)[0]
    q, k, v = q.reshape(B, Hkv, G * Tq, -1), k.contiguous(), v.contiguous()         # a key head's queries, one below another
    i, j = torch.arange(Tq, device=DEV)[:, None], torch.arange(Tk, device=DEV)
    seen = (j <= i + (nk - nq)[:, None, None]) & (j < nk[:, None, None])
    seen = seen[:, None, None].expand(B, Hkv, G, Tq, Tk)
    scores = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).view(B, Hkv, G, Tq, Tk)
    p = _softmax(scores, seen).view(B, Hkv, G * Tq, Tk)
    del scores
    o = torch.matmul(p, v)
    rows = lambda x, d: x.reshape(B, H, Tq, d).transpose(1, 2)[realq].to(dt)  # noqa: E731
    out = {"o": rows(o, c["dv"])}
    if c["kind"] == "fwd":
        return out
    do = _padded(s["dO"], s["cu_q"], B, Tq)[0] * realq[:, None, :, None]
    do = do.reshape(B, Hkv, G * Tq, -1)
    keys = lambda x: x.transpose(1, 2)[realk].to(dt)  # noqa: E731
    out["dv"] = keys(torch.matmul(p.transpose(-1, -2), do))
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * s["scale"]
    del p
    dq, dk = rows(torch.matmul(ds, k), q.shape[-1]), torch.matmul(ds.transpose(-1, -2), q)
    out["dqn"], out["dkn"] = dq[..., :dn], keys(dk[..., :dn])
    if c["dr"]:
        out["dqr"], out["dkr"] = dq[..., dn:], dk[..., dn:].sum(1)[realk].to(dt)
    return out


# ---------------------------------------------------------------------------------------------------- the library's calls

def _own_prep(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    N, H, dc, dr = s["kv"].shape[0], c["H"], c["dc"], c["dr"]
    dt = s["kv"].dtype
    qr = torch.empty((N, H, dr), dtype=dt, device=DEV)
    if c["kind"] == "prep":
        if "plan" not in s:     # what a serving loop keeps for its steps
            s["plan"] = gdn.make_mla_prep(N, H, dc, dr, c["io"], s["rot"].shape[0], EPS, interleaved=c["pairs"], B=c["B"],
                                          page=c["page"], npages=s["cache"].shape[0], maxpages=s["table"].shape[1])
        gdn.check(gdn.gdn_mla_prep(s["plan"], s["kv"], s["w"], s["rot"], s["pos"], s["seq"], s["table"], s["qr"], s["cache"],
                                   None, qr))
        return {"cache": s["cache"], "qr": qr}
    if "plan" not in s:
        s["plan"] = gdn.make_mla_prep(N, H, dc, dr, c["io"], s["rot"].shape[0], EPS, interleaved=c["pairs"])
        s["ws"] = torch.empty(gdn.gdn_mla_prep_workspace_bytes(s["plan"]), dtype=torch.uint8, device=DEV)
    lat, kr, dkv = (torch.empty((N, d), dtype=dt, device=DEV) for d in (dc, dr, dc + dr))
    dw, dqr = torch.empty(dc, device=DEV), torch.empty((N, H, dr), dtype=dt, device=DEV)
    gdn.check(gdn.gdn_mla_prep(s["plan"], s["kv"], s["w"], s["rot"], s["pos"], None, None, s["qr"], lat, kr, qr))
    gdn.check(gdn.gdn_mla_prep_bwd(s["plan"], s["kv"], s["w"], s["rot"], s["pos"], s["dlat"], s["dkr"], s["dqr"], dkv, dw, dqr,
                                   s["ws"]))
    return {"lat": lat, "kr": kr, "qr": qr, "dkv": dkv, "dw": dw, "dqr": dqr}


def _own_decode(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    if "plan" not in s:
        s["plan"] = gdn.make_mla_cache(c["B"], c["T"], c["H"], c["dc"], c["dr"], c["page"], s["cache"].shape[0],
                                       s["table"].shape[1], c["io"], s["scale"])
        s["ws"] = torch.empty(gdn.gdn_mla_decode_workspace_bytes(s["plan"]), dtype=torch.uint8, device=DEV)
    o = torch.empty_like(s["qc"])
    gdn.check(gdn.gdn_mla_decode(s["plan"], s["qc"], s["qr"], s["cache"], s["table"], s["lens"], o, None, s["ws"]))
    return o


def _own_attention(s):
    import linear_attention_recurrence_delta_gb300 as gdn
    c = s["case"]
    train = c["kind"] == "train"
    Nq, Nk, H, dv = s["qn"].shape[0], s["kn"].shape[0], c["H"], c["dv"]
    if "plan" not in s:
        s["plan"] = gdn.make_mla_attn(c["B"], H, c["Hkv"], c["Tq"], c["Tk"], c["dn"], c["dr"], dv, c["io"], s["scale"],
                                      causal=True, Nq=Nq, Nk=Nk)
        s["ws"] = torch.empty(gdn.gdn_mla_workspace_bytes(s["plan"], int(train)), dtype=torch.uint8, device=DEV)
    args = (s["qn"], s["qr"], s["kn"], s["kr"], s["v"], s["cu_q"], s["cu_k"])
    dt = s["qn"].dtype
    o = torch.empty((Nq, H, dv), dtype=dt, device=DEV)
    lse = torch.empty((H, Nq), device=DEV) if train else None
    gdn.check(gdn.gdn_mla_fwd(s["plan"], *args, o, lse, s["ws"]))
    if not train:
        return {"o": o}
    dq = torch.empty((Nq, H, c["dn"] + c["dr"]), dtype=dt, device=DEV)
    dkv = torch.empty((Nk, c["Hkv"], c["dn"] + dv), dtype=dt, device=DEV)
    dkr = torch.empty((Nk, c["dr"]), dtype=dt, device=DEV) if c["dr"] else None
    out = {"o": o, "dqn": dq[..., : c["dn"]], "dkn": dkv[..., : c["dn"]], "dv": dkv[..., c["dn"]:]}
    dqr = dq[..., c["dn"]:] if c["dr"] else None
    gdn.check(gdn.gdn_mla_bwd(s["plan"], *args, o, lse, s["dO"], out["dqn"], dqr, out["dkn"], dkr, out["dv"], s["ws"]))
    if c["dr"]:
        out["dqr"], out["dkr"] = dqr, dkr
    return out


def run(state):
    kind = state["case"]["kind"]
    if kind in ("prep", "prep_train"):
        return _own_prep(state) if own else _plain_prep(state)
    if kind == "decode":
        return _own_decode(state) if own else _plain_decode(state)
    return _own_attention(state) if own else _plain_attention(state)


# ---------------------------------------------------------------------------------------------------- the definitions in 64 bits

def _turned(x, pos, pairs):
    """x [N, ..., d] rotated by the angles of the rows' positions, as products of complex numbers."""
    d = x.shape[-1]
    at = torch.arange(d // 2, device=DEV)
    one, two = (2 * at, 2 * at + 1) if pairs else (at, at + d // 2)
    r = _rotation(int(pos.max()) + 1, d).double()[pos.long()]      # the table is an input of the operator
    turn = torch.complex(r[:, : d // 2], r[:, d // 2:]).view([x.shape[0]] + [1] * (x.dim() - 2) + [d // 2])
    z = torch.complex(x[..., one], x[..., two]) * turn
    out = torch.empty_like(x)
    out[..., one], out[..., two] = z.real, z.imag
    return out


def _attend(q, k, v, scale):
    """One head's queries, the last of the sequence, over its keys and values in 64 bits."""
    a, b = q.shape[0], k.shape[0]
    x = (q @ k.T) * scale
    x = x.masked_fill(torch.ones(a, b, dtype=torch.bool, device=DEV).triu(b - a + 1), -math.inf)
    empty = max(0, a - b)                                          # the first queries precede every key
    return torch.cat([torch.zeros(empty, v.shape[1], dtype=v.dtype, device=DEV), torch.softmax(x[empty:], -1) @ v])


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("prep", "prep_train"):
        dc = case["dc"]
        kv, w, qr = s["kv"].double().requires_grad_(), s["w"].double().requires_grad_(), s["qr"].double().requires_grad_()
        rms = (kv[:, :dc] ** 2).sum(-1, keepdim=True).div(dc).add(EPS).sqrt()
        lat, kr, q = kv[:, :dc] / rms * w, _turned(kv[:, dc:], s["pos"], case["pairs"]), _turned(qr, s["pos"], case["pairs"])
        if kind == "prep":
            cache = s["cache"].double().flatten(0, 1)
            places = [int(x) for x in (s["table"].cpu()[s["seq"].cpu().long(), s["pos"].cpu().long() // case["page"]].long() *
                                       case["page"] + s["pos"].cpu().long() % case["page"])]
            cache[torch.tensor(places, device=DEV)] = torch.cat([lat, kr], 1).detach()
            return {"cache": cache.view(s["cache"].shape), "qr": q.detach()}
        loss = (lat * s["dlat"].double()).sum() + (kr * s["dkr"].double()).sum() + (q * s["dqr"].double()).sum()
        dkv, dw, dq = torch.autograd.grad(loss, [kv, w, qr])
        return {"lat": lat.detach(), "kr": kr.detach(), "qr": q.detach(), "dkv": dkv, "dw": dw, "dqr": dq}
    if kind == "decode":
        T, H, dc, page = case["T"], case["H"], case["dc"], case["page"]
        o = torch.zeros(s["qc"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_cache_lengths(case)):
            if n == 0:
                continue
            rows = torch.cat([s["cache"][int(p)] for p in s["table"][b, : -(-n // page)]])[:n].double()
            for h in range(H):
                q = torch.cat([s["qc"][b, :, h], s["qr"][b, :, h]], -1).double()
                o[b, :, h] = _attend(q, rows, rows[:, :dc], s["scale"])
        return o
    H, Hkv, dr = case["H"], case["Hkv"], case["dr"]
    names = [k for k in ("qn", "qr", "kn", "kr", "v") if s[k] is not None]
    x = {k: s[k].double() for k in names}
    o = torch.zeros(x["qn"].shape[:2] + (case["dv"],), dtype=torch.float64, device=DEV)
    grad = {k: torch.zeros_like(x[k]) for k in names} if kind == "train" else {}
    q0 = k0 = 0
    for nq, nk in zip(*_attn_lengths(case)):
        qs, ks = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        for h in range(H):
            place = {"qn": (qs, h), "qr": (qs, h), "kn": (ks, h * Hkv // H), "kr": (ks,), "v": (ks, h * Hkv // H)}
            a = {k: x[k][place[k]].clone().requires_grad_(kind == "train") for k in names}
            q = torch.cat([a["qn"], a["qr"]], -1) if dr else a["qn"]
            k = torch.cat([a["kn"], a["kr"]], -1) if dr else a["kn"]
            y = _attend(q, k, a["v"], s["scale"])
            o[qs, h] = y.detach()
            if kind == "train":
                for name, d in zip(names, torch.autograd.grad((y * s["dO"][qs, h].double()).sum(), [a[k] for k in names])):
                    grad[name][place[name]] += d
    out = {"o": o}
    out.update({"d" + k: v for k, v in grad.items()})
    return out
