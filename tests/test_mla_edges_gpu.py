"""Latent attention at its edges: ends inside a warp, NaN and Inf and how far they reach, status words."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
import tests.test_mla_attn_gpu as attn
import tests.test_mla_decode_gpu as decode
from tests.mla_testlib import attn_inputs, attn_run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dn,dr,dv", [(64, 0, 64), (64, 64, 128), (128, 64, 128), (128, 0, 24)])
def test_ends_inside_a_warp(dn, dr, dv, causal):
    """The last row of a tile in each of its four warps, first, inner and last lane: the lanes past it store nothing while
    the warp reads on.  One, two and three 64-column blocks a key, and a value that one half of the columns holds."""
    n = [1, 31, 33, 50, 63, 65, 81, 96, 97, 127, 129, 190, 225]
    x, dO = attn_inputs(sum((dn, dr, dv)), n, n, 2, 1, dn, dr, dv, "bf16")
    attn.compare(x, dO, n, n, causal, "bf16")


@pytest.mark.parametrize("n", [[64] * 160 + [1], [20000, 70]])
@pytest.mark.parametrize("dc", [8, 24, 40, 104, 136, 200, 264, 488])
def test_latents_that_end_inside_a_warp(dc, n):
    """Widths whose last 32 columns are not all there, of sequences that one worker covers and of ones that many share."""
    decode.compare(dc + len(n), n, 1, 16, dc, 16, 16, "bf16")


@pytest.mark.parametrize("T,H", [(1, 3), (2, 40), (3, 30), (5, 33), (8, 128)])
def test_query_rows_that_end_inside_a_warp(T, H):
    """Rows that fill a part of a group's columns, in one group and in several, over enough tiles for a raised maximum."""
    decode.compare(T * H, [300, 1, 0, 2000, 64], T, H, 200, 32, 16, "bf16", std=4.0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 5), (1, 16), (2, 40), (8, 70)])
@pytest.mark.parametrize("where", ["latent", "position", "query"])
def test_nan_that_a_query_sees(where, T, H, io):
    """A NaN in a row that every query sees, or in the queries, makes o and lse NaN, in a piece of its own or in one of many;
    the other sequences keep their bits."""
    n, dc, dr, page = [5000, 40, 300, 700], 128, 32, 16
    table, pages, cache, rows, qc, qr = decode.setup(T + H, n, T, H, dc, dr, page, io)
    good = decode.call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, 0.1)
    bad = [0, 1]
    for b in bad:
        if where == "query":
            qc[b, :, :, 3] = math.nan
        else:
            cache[table[b, 1], 7, 5 if where == "latent" else dc + 5] = math.nan
    o, lse = decode.call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, 0.1)
    for b in range(len(n)):
        if b in bad:
            assert torch.isnan(lse[b]).all(), b
            assert torch.isnan(o[b]).all() if where != "latent" else torch.isnan(o[b]).any(-1).all(), b
        else:
            assert torch.equal(o[b], good[0][b]) and torch.equal(lse[b], good[1][b]), b


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,H", [(2, 5), (4, 40), (8, 16)])
def test_reach_of_a_drafted_row(T, H, bad, io):
    """A NaN or Inf in the last new token's row: the earlier tokens' lse and every other sequence keep their bits, the token
    itself gets a NaN or an Inf."""
    n, dc, dr, page = [3000, 70, 64, 300], 128, 32, 16
    table, pages, cache, rows, qc, qr = decode.setup(3 * T + H, n, T, H, dc, dr, page, io)
    good = decode.call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, 0.1)
    hit = [0, 1, 2]
    for b in hit:
        cache[table[b, (n[b] - 1) // page], (n[b] - 1) % page, :dc] = bad
    o, lse = decode.call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, 0.1)
    for b in range(len(n)):
        if b in hit:
            assert torch.equal(lse[b, :-1], good[1][b, :-1]), b
            assert (~torch.isfinite(o[b, -1])).all(), b
        else:
            assert torch.equal(o[b], good[0][b]) and torch.equal(lse[b], good[1][b]), b


@pytest.mark.parametrize("T,H", [(1, 5), (2, 9), (3, 30)])
def test_another_sequences_queries_change_no_bit(T, H):
    """The queries of the sequences behind, whose rows fill up a group's columns: large ones, whose scores rise from tile to
    tile, Inf and NaN leave every bit of the first sequence's results."""
    n, dc, dr, page = [6000, 500, 300], 128, 32, 16
    table, pages, cache, rows, qc, qr = decode.setup(T + 7 * H, n, T, H, dc, dr, page, "bf16", 4.0)
    good = decode.call(n, T, H, dc, dr, page, "bf16", table, pages, cache, qc, qr, 0.1)
    for factor in (30.0, math.inf, math.nan):
        c, r = qc.clone(), qr.clone()
        c[1:] *= factor
        r[1:] *= factor
        o, lse = decode.call(n, T, H, dc, dr, page, "bf16", table, pages, cache, c, r, 0.1)
        assert torch.equal(o[0], good[0][0]) and torch.equal(lse[0], good[1][0]), factor


def test_status_words():
    """What a kernel may leave in a workspace's first word, as the status reads it."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for word, status in ((0, gdn.GDN_OK), (1, 7), (2, 6), (0, gdn.GDN_OK)):     # timeout; shared memory not as compiled for
        ws[0] = word
        assert gdn.gdn_last_device_status(ws) == status


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dn,dr,dv", [(64, 32, 64), (128, 64, 128)])
@pytest.mark.parametrize("nq,nk,at", [(600, 600, 383), (600, 600, 300), (500, 731, 640), (700, 660, 511)])
def test_reach_of_a_nan_in_a_sequence(nq, nk, at, dn, dr, dv, io):
    """A NaN in a key: queries 255 positions and more before it keep the bits of their o and gradients.  One in a query's
    rows: so do the keys 255 positions and more behind it.  Every other head group keeps all."""
    H, Hkv = 4, 2
    x, dO = attn_inputs(nq + at, [nq], [nk], H, Hkv, dn, dr, dv, io)
    good = attn_run(x, [nq], [nk], 0.1, True, io, dO)
    off = nk - nq
    y = {k: t.clone() for k, t in x.items()}
    y["kn"][at, 0] = y["v"][at, 0] = math.nan
    o, lse, d = attn_run(y, [nq], [nk], 0.1, True, io, dO)
    far = max(0, at - 254 - off)                     # the queries before this one
    sees = max(0, at - off)                          # the first that sees the key
    assert torch.equal(o[:far], good[0][:far]) and torch.equal(lse[:, :sees], good[1][:, :sees])
    assert torch.equal(o[:, 2:], good[0][:, 2:]) and torch.isnan(o[sees:, :2]).all()
    for k in ("qn", "qr"):
        assert torch.equal(d[k][:far], good[2][k][:far]) and torch.equal(d[k][:, 2:], good[2][k][:, 2:]), k
    for k in ("kn", "v"):
        assert torch.equal(d[k][:, 1], good[2][k][:, 1]), k
    row = max(0, at - off - 200)
    y, dP = {k: t.clone() for k, t in x.items()}, dO.clone()
    y["qn"][row, 0] = dP[row, 0] = math.nan
    o, lse, d = attn_run(y, [nq], [nk], 0.1, True, io, dP)
    keep = torch.arange(nq, device="cuda") != row
    assert torch.equal(o[keep], good[0][keep]) and torch.equal(lse[:, keep], good[1][:, keep])
    for k in ("qn", "qr"):
        assert torch.equal(d[k][keep], good[2][k][keep]), k
    for k in ("kn", "v"):
        past = row + off + 255
        assert torch.equal(d[k][past:], good[2][k][past:]) and torch.equal(d[k][:, 1], good[2][k][:, 1]), k
