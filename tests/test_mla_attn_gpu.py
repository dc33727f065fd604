"""gdn_mla_fwd and gdn_mla_bwd against 64 bits: lengths, head groups, widths, masks, packed rows, isolation."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.mla_testlib import attn_inputs, attn_ref, attn_run, close, gen, normal, offsets

pytestmark = pytest.mark.gpu

WIDTHS = [(64, 64, 128), (128, 64, 128), (56, 16, 56), (64, 0, 64), (128, 0, 72), (8, 8, 8), (96, 32, 128)]


def compare(x, dO, nq, nk, causal, io, **kw):
    scale = 1.0 / math.sqrt(x["qn"].shape[-1] + (0 if x["qr"] is None else x["qr"].shape[-1]))
    ro, rl, rd = attn_ref(x, nq, nk, scale, causal, dO)
    o, lse, d = attn_run(x, nq, nk, scale, causal, io, dO, **kw)
    close(o, ro, io, "fwd", "o")
    none = rl == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, none)
    assert torch.isfinite(lse.cpu()[~none]).all()
    if (~none).any():
        assert (lse.cpu()[~none] - rl[~none]).abs().max() <= 2e-5 * max(1.0, rl[~none].abs().max().item())
    for k in rd:
        close(d[k], rd[k], io, "bwd", f"d{k}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dn,dr,dv", WIDTHS)
def test_widths(io, causal, dn, dr, dv):
    nq = nk = [150, 3, 97]
    x, dO = attn_inputs(dn + dr + dv, nq, nk, 4, 2, dn, dr, dv, io)
    compare(x, dO, nq, nk, causal, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (6, 2), (5, 1)])
def test_head_groups(io, H, Hkv):
    nq = nk = [130, 70]
    x, dO = attn_inputs(H, nq, nk, H, Hkv, 64, 32, 64, io)
    compare(x, dO, nq, nk, True, io)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_lengths(n):
    x, dO = attn_inputs(n, [n], [n], 2, 1, 64, 64, 128, "bf16")
    compare(x, dO, [n], [n], True, "bf16")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_after_a_prefix(io, causal):
    """Fewer queries than keys (a chunk after a prefix), and more: those rows that see no key give zeros."""
    nq, nk = [1, 40, 200, 150, 130], [300, 170, 200, 20, 1]
    x, dO = attn_inputs(9, nq, nk, 4, 2, 64, 32, 64, io)
    compare(x, dO, nq, nk, causal, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_empty_sequences(io):
    """Sequences without queries, without keys, or without either; keys that no query sees get zero gradients."""
    nq, nk = [0, 70, 0, 5, 66], [40, 0, 0, 5, 66]
    x, dO = attn_inputs(10, nq, nk, 2, 2, 64, 0, 64, io)
    compare(x, dO, nq, nk, True, io)
    compare(x, dO, nq, nk, False, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_dense_batch(io):
    """Without offsets the sequences lie one after another, [B, T, heads, d]."""
    nq, nk = [100] * 3, [140] * 3
    x, dO = attn_inputs(11, nq, nk, 4, 4, 32, 16, 48, io)
    compare(x, dO, nq, nk, True, io, cu=False)


def test_longer_bf16():
    """Many tiles a row, uneven lengths, four query heads a key head."""
    nq = nk = [1111, 700]
    x, dO = attn_inputs(12, nq, nk, 4, 1, 64, 64, 128, "bf16")
    compare(x, dO, nq, nk, True, "bf16")


@pytest.mark.parametrize("scale", [6.0, 0.0])
def test_sharp_and_flat_scores(scale):
    """Scores of hundreds (one weight of almost one, the rest far below fp32's range) and of zero."""
    nq = nk = [260]
    x, dO = attn_inputs(13, nq, nk, 2, 2, 64, 64, 128, "bf16")
    ro, rl, rd = attn_ref(x, nq, nk, scale, True, dO)
    o, lse, d = attn_run(x, nq, nk, scale, True, "bf16", dO)
    close(o, ro, "bf16", "fwd", "o")
    assert ((lse.cpu() - rl).abs() <= 2e-5 * rl.abs().max() + 1e-5).all()
    if scale == 0.0:   # all keys weigh the same: the queries get no gradient at all
        assert all((d[k] == 0).all() for k in ("qn", "qr", "kn", "kr"))
        close(d["v"], rd["v"], "bf16", "bwd", "dv")
    else:
        assert all(torch.isfinite(d[k]).all() for k in d)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_other_sequences_do_not_reach_a_result(io):
    """A NaN or Inf anywhere in a neighbouring sequence of the packed rows changes no bit of this one's results."""
    nq = nk = [70, 90, 201]
    x, dO = attn_inputs(14, nq, nk, 4, 2, 64, 32, 64, io)
    scale = 0.1
    o, lse, d = attn_run(x, nq, nk, scale, True, io, dO)
    a, b = offsets(nq)[1:3]
    for bad in (math.nan, math.inf):
        y = {k: t.clone() for k, t in x.items()}
        dP = dO.clone()
        for t in (*y.values(), dP):
            t[a:b] = bad
        po, pl, pd = attn_run(y, nq, nk, scale, True, io, dP)
        keep = torch.cat([torch.arange(0, a), torch.arange(b, sum(nq))]).cuda()
        assert torch.equal(po[keep], o[keep]) and torch.equal(pl[:, keep], lse[:, keep])
        for k in d:
            assert torch.equal(pd[k][keep], d[k][keep]), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_of_no_sequence_stay(io):
    """Offsets that leave rows out before, between and after the sequences (and lie outside the tensors): those rows'
    outputs are not written; a sequence longer than the shape says is cut."""
    N, H = 300, 2
    g = gen(15)
    x = {k: normal(g, (N, H, 64), io) for k in ("qn", "kn", "v")}
    x.update(qr=None, kr=None)
    dO = normal(g, (N, H, 64), io)
    cu = torch.tensor([10, 90, 400], dtype=torch.int32)       # the second sequence is cut to Tq rows and at the end
    T = 150
    s = gdn.make_mla_attn(2, H, H, T, T, 64, 0, 64, io, 0.125, True, Nq=N, Nk=N)
    dev = {k: None if t is None else t.cuda() for k, t in x.items()}
    fill = lambda: torch.full((N, H, 64), 3.0, dtype=x["qn"].dtype, device="cuda")  # noqa: E731
    o, lse = fill(), torch.full((H, N), 3.0, device="cuda")
    ws = torch.empty(gdn.gdn_mla_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
    a = (dev["qn"], None, dev["kn"], None, dev["v"], cu.cuda(), cu.cuda())
    gdn.check(gdn.gdn_mla_fwd(s, *a, o, lse, ws))
    d = {k: fill() for k in ("qn", "kn", "v")}
    gdn.check(gdn.gdn_mla_bwd(s, *a, o, lse, dO.cuda(), d["qn"], None, d["kn"], None, d["v"], ws))
    rows = [slice(10, 90), slice(90, 240)]
    ref = attn_ref({k: None if t is None else torch.cat([t[r] for r in rows]) for k, t in x.items()}, [80, 150], [80, 150], 0.125,
                   True, torch.cat([dO[r] for r in rows]))
    inside = torch.zeros(N, dtype=torch.bool)
    inside[10:240] = True
    close(o.cpu()[inside], ref[0], io, "fwd", "o")
    assert (o.cpu()[~inside] == 3.0).all() and (lse.cpu()[:, ~inside] == 3.0).all()
    for k in d:
        close(d[k].cpu()[inside], ref[2][k], io, "bwd", k)
        assert (d[k].cpu()[~inside] == 3.0).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strides_and_head_major(io):
    """Views of wider rows, and keys stored head by head: the row stride is the smaller one."""
    nq = nk = [77, 140]
    N, H, Hkv = sum(nq), 4, 2
    x, dO = attn_inputs(16, nq, nk, H, Hkv, 64, 16, 64, io)
    wide = {}
    for k, t in x.items():
        if t.dim() == 3:
            pad = torch.full((t.shape[1], N, t.shape[2] + 24), math.nan, dtype=t.dtype, device="cuda")
            wide[k] = pad[..., 8: 8 + t.shape[2]].transpose(0, 1)
        else:
            wide[k] = torch.full((N, t.shape[1] + 40), math.nan, dtype=t.dtype, device="cuda")[:, 16: 16 + t.shape[1]]
        wide[k].copy_(t)
    scale = 0.11
    o, lse, d = attn_run(x, nq, nk, scale, True, io, dO)
    po, pl, pd = attn_run(wide, nq, nk, scale, True, io, dO)
    assert torch.equal(o, po) and torch.equal(lse, pl)
    for k in d:
        assert torch.equal(d[k], pd[k]), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_same_call_same_bits_on_another_stream(io):
    nq = nk = [200, 333]
    x, dO = attn_inputs(17, nq, nk, 8, 2, 64, 64, 128, io)
    a = attn_run(x, nq, nk, 0.1, True, io, dO)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = attn_run(x, nq, nk, 0.1, True, io, dO)
    st.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for k in a[2]:
        assert torch.equal(a[2][k], b[2][k]), k


@pytest.mark.parametrize("io,tol", [("f32", 2e-3), ("bf16", 3e-2)])
def test_gradients_against_differences(io, tol):
    """Central differences of the 64-bit definition along random directions: step 1e-4, whose own error is of order
    1e-8; the gradient's is its type's (a direction mixes all its values, so its size is the norm's)."""
    nq = nk = [60, 33]
    x, dO = attn_inputs(18, nq, nk, 2, 1, 32, 16, 32, io)
    scale = 0.15
    _, _, d = attn_run(x, nq, nk, scale, True, io, dO)
    g = gen(19)
    for k in x:
        u = torch.randn(x[k].shape, generator=g, dtype=torch.float64)
        at = []
        for e in (1e-4, -1e-4):
            y = {n: t.double() for n, t in x.items()}
            y[k] = y[k] + e * u
            at.append((attn_ref(y, nq, nk, scale, True)[0] * dO.double()).sum().item())
        want, got = (at[0] - at[1]) / 2e-4, (d[k].double().cpu() * u).sum().item()
        assert abs(got - want) <= tol * d[k].double().norm().item(), k
