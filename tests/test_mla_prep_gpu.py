"""gdn_mla_prep and its gradients against 64 bits: paged and dense rows, both pairings, skipped tokens, strides."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.mla_testlib import EPS, block_table, close, gen, normal, prep_ref, rotation, tdtype

pytestmark = pytest.mark.gpu


def inputs(seed, N, H, dc, dr, io, npos, pad=0):
    g = gen(seed)
    kv = normal(g, (N, dc + dr + pad), io, 0.7)[:, : dc + dr]
    w = 1.0 + 0.2 * torch.randn(dc, generator=g)
    q = normal(g, (N, H, 32 + dr), io)
    pos = torch.randint(0, npos, (N,), generator=g, dtype=torch.int32)
    return g, kv, w, q[..., 32:], pos


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,dc,dr,pad", [(1, 1, 8, 16, 0), (24, 16, 256, 64, 0), (37, 5, 520, 48, 8), (130, 3, 1024, 128, 0),
                                           (9, 2, 64, 0, 8), (7, 0, 192, 32, 0)])
def test_dense_and_gradients(io, interleaved, N, H, dc, dr, pad):
    g, kv, w, qr, pos = inputs(N + dc, N, H, dc, dr, io, 500, pad)
    rot = rotation(500, dr)
    queries = H > 0 and dr > 0
    s = gdn.make_mla_prep(N, H, dc, dr, io, 500, EPS, interleaved)
    nan = lambda *shape: torch.full(shape, math.nan, dtype=tdtype(io), device="cuda")  # noqa: E731
    lat, kr, qo = nan(N, dc), nan(N, dr) if dr else None, nan(N, H, dr) if queries else None
    dev = lambda t: t.cuda()  # noqa: E731
    args = (dev(kv), dev(w), dev(rot) if dr else None, dev(pos))
    gdn.check(gdn.gdn_mla_prep(s, *args, None, None, dev(qr) if queries else None, lat, kr, qo))
    x = [t.double().requires_grad_() for t in (kv, w, qr)]
    want = prep_ref(x[0], x[1], dc, rot[pos.long()], x[2] if queries else None, interleaved)
    close(lat, want[0], io, "fwd", "lat")
    if dr:
        close(kr, want[1], io, "fwd", "kr")
    if queries:
        close(qo, want[2], io, "fwd", "qr")
    dlat, dkr, dqr = normal(g, (N, dc), io), normal(g, (N, dr), io), normal(g, (N, H, 40 + dr), io)[..., 40:]
    loss = (want[0] * dlat.double()).sum() + (want[1] * dkr.double()).sum()
    if queries:
        loss = loss + (want[2] * dqr.double()).sum()
    ref = torch.autograd.grad(loss, x, allow_unused=True)
    dkv, dw, dqo = nan(N, dc + dr), torch.full((dc,), math.nan, device="cuda"), nan(N, H, dr) if queries else None
    ws = torch.empty(gdn.gdn_mla_prep_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    call = lambda: gdn.check(gdn.gdn_mla_prep_bwd(  # noqa: E731
        s, *args, dev(dlat), dev(dkr) if dr else None, dev(dqr) if queries else None, dkv, dw, dqo, ws))
    call()
    close(dkv, ref[0], io, "bwd", "dkv")
    close(dw, ref[1], "f32", "bwd", "dw")
    if queries:
        close(dqo, ref[2], io, "bwd", "dqr")
    first = dw.clone()
    call()
    assert torch.equal(first, dw)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 64, 100])
def test_paged_write(io, page):
    """Prompts and single tokens in one call; tokens with a bad position, sequence or page leave the cache alone."""
    H, dc, dr, npos = 4, 192, 32, 400
    first, new = [0, 77, 399, 5], [130, 1, 1, 20]
    n = [a + b for a, b in zip(first, new)]
    N = sum(new) + 4
    g, kv, w, qr, _ = inputs(page, N, H, dc, dr, io, npos)
    table, pages = block_table(g, n, page, width=max(-(-k // page) for k in n) + 1)
    at = [(b, first[b] + i) for b in range(4) for i in range(new[b])] + [(0, -1), (4, 3), (3, npos + 2), (1, page * (-(-n[1] // page)))]
    seq = torch.tensor([b for b, _ in at], dtype=torch.int32)
    pos = torch.tensor([p for _, p in at], dtype=torch.int32)
    cache = normal(g, (pages, page, dc + dr), io)
    rot = rotation(npos, dr)
    s = gdn.make_mla_prep(N, H, dc, dr, io, npos, EPS, B=4, page=page, npages=pages, maxpages=table.shape[1])
    got, qo = cache.cuda(), torch.full((N, H, dr), 7.0, dtype=tdtype(io), device="cuda")
    gdn.check(gdn.gdn_mla_prep(s, kv.cuda(), w.cuda(), rot.cuda(), pos.cuda(), seq.cuda(), table.cuda(), qr.cuda(), got, None, qo))
    ok = sum(new)
    lat, kr, q = prep_ref(kv.double(), w.double(), dc, rot[pos.long().clamp(0, npos - 1)], qr.double(), False)
    want = cache.double().clone()
    touched = torch.zeros(pages, page, dtype=torch.bool)
    for i in range(ok):
        b, p = at[i]
        want[table[b, p // page], p % page] = torch.cat([lat[i], kr[i]])
        touched[table[b, p // page], p % page] = True
    close(got, want, io, "fwd", "cache")
    assert torch.equal(got.cpu()[~touched], cache[~touched])
    fine = torch.tensor([0 <= p < npos for _, p in at])
    close(qo.cpu()[fine], q[fine], io, "fwd", "qr")
    assert (qo.cpu()[~fine] == 7.0).all()


def test_in_place_queries_and_zero_latent():
    """qr_out may be the very view of qr; a latent of zeros stays zero (eps keeps the division finite)."""
    N, H, dc, dr = 19, 6, 64, 64
    g, kv, w, qr, pos = inputs(3, N, H, dc, dr, "bf16", 50)
    kv[4] = 0
    rot = rotation(50, dr)
    s = gdn.make_mla_prep(N, H, dc, dr, "bf16", 50, EPS)
    whole = torch.zeros(N, H, 32 + dr, dtype=torch.bfloat16, device="cuda")
    q = whole[..., 32:]
    q.copy_(qr)
    lat, kr = (torch.empty(N, d, dtype=torch.bfloat16, device="cuda") for d in (dc, dr))
    gdn.check(gdn.gdn_mla_prep(s, kv.cuda(), w.cuda(), rot.cuda(), pos.cuda(), None, None, q, lat, kr, q))
    want = prep_ref(kv.double(), w.double(), dc, rot[pos.long()], qr.double(), False)
    close(q, want[2], "bf16", "fwd", "qr in place")
    close(lat, want[0], "bf16", "fwd", "lat")
    assert (lat[4] == 0).all() and (whole[..., :32] == 0).all()


def test_bad_positions_give_zero_gradients():
    N, H, dc, dr = 11, 2, 64, 32
    g, kv, w, qr, pos = inputs(5, N, H, dc, dr, "bf16", 50)
    pos[2], pos[7] = -3, 50
    s = gdn.make_mla_prep(N, H, dc, dr, "bf16", 50, EPS)
    dlat, dkr, dqr = normal(g, (N, dc), "bf16"), normal(g, (N, dr), "bf16"), normal(g, (N, H, dr), "bf16")
    rot = rotation(50, dr)
    dkv, dqo = (torch.full(t.shape, math.nan, dtype=torch.bfloat16, device="cuda") for t in (kv, dqr))
    dw = torch.empty(dc, device="cuda")
    ws = torch.empty(gdn.gdn_mla_prep_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_mla_prep_bwd(s, kv.cuda(), w.cuda(), rot.cuda(), pos.cuda(), dlat.cuda(), dkr.cuda(), dqr.cuda(), dkv, dw,
                                   dqo, ws))
    bad = torch.tensor([2, 7])
    assert (dkv[bad.cuda()] == 0).all() and (dqo[bad.cuda()] == 0).all()
    keep = torch.tensor([i for i in range(N) if i not in (2, 7)])
    x, ww = kv[keep].double(), w.double().requires_grad_()
    loss = (prep_ref(x, ww, dc, rot[pos[keep].long()], None, False)[0] * dlat[keep].double()).sum()
    close(dw, torch.autograd.grad(loss, ww)[0], "f32", "bwd", "dw")


def test_no_tokens():
    s = gdn.make_mla_prep(0, 4, 64, 32, "bf16", 10, EPS)
    assert gdn.gdn_mla_prep(s, None, None, None, None, None, None, None, None, None, None) == gdn.GDN_OK
    dw = torch.full((64,), math.nan, device="cuda")
    ws = torch.empty(gdn.gdn_mla_prep_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_mla_prep_bwd(s, None, None, None, None, None, None, None, None, dw, None, ws))
    assert (dw == 0).all()
