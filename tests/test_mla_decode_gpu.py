"""gdn_mla_decode against 64 bits: lengths from none to long, head counts, widths, pages, drafts, isolation."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.mla_testlib import block_table, close, decode_ref, gen, normal, tdtype

pytestmark = pytest.mark.gpu


def setup(seed, n, T, H, dc, dr, page, io, std=1.0):
    g = gen(seed)
    table, pages = block_table(g, n, page)
    # places that no length covers, and pages that no table names, hold NaN
    cache = torch.full((pages, page, dc + dr), math.nan, dtype=tdtype(io))
    rows = []
    for b, k in enumerate(n):
        r = normal(g, (k, dc + dr), io)
        for j in range(k):
            cache[table[b, j // page], j % page] = r[j]
        rows.append(r)
    qc = normal(g, (len(n), T, H, dc), io, std * 1.5 * math.sqrt(64.0 / dc))
    qr = normal(g, (len(n), T, H, dr), io, std * 1.5) if dr else None
    return table, pages, cache, rows, qc, qr


def call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, scale, stream=None, lens=None):
    s = gdn.make_mla_cache(len(n), T, H, dc, dr, page, pages, table.shape[1], io, scale)
    o = torch.full((len(n), T, H, dc), math.nan, dtype=tdtype(io), device="cuda")
    lse = torch.full((len(n), T, H), math.nan, device="cuda")
    ws = torch.full((gdn.gdn_mla_decode_workspace_bytes(s),), 0xFF, dtype=torch.uint8, device="cuda")
    dev = lambda t: None if t is None else (t if t.is_cuda else t.cuda())  # noqa: E731
    lens = torch.tensor(n if lens is None else lens, dtype=torch.int32)
    gdn.check(gdn.gdn_mla_decode(s, dev(qc), dev(qr), dev(cache), dev(table), dev(lens), o, lse, ws, stream=stream))
    gdn.check(gdn.gdn_last_device_status(ws, stream=stream))
    return o, lse


def compare(seed, n, T, H, dc, dr, page, io, std=1.0):
    table, pages, cache, rows, qc, qr = setup(seed, n, T, H, dc, dr, page, io, std)
    scale = 1.0 / math.sqrt(64 + dr)
    o, lse = call(n, T, H, dc, dr, page, io, table, pages, cache, qc, qr, scale)
    ref = [decode_ref(qc[b], None if qr is None else qr[b], rows[b], scale) for b in range(len(n))]
    ro, rl = torch.stack([r[0] for r in ref]), torch.stack([r[1] for r in ref])
    close(o, ro, io, "fwd", "o")
    none = rl == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, none)
    if (~none).any():
        assert (lse.cpu()[~none] - rl[~none]).abs().max() <= 2e-5 * max(1.0, rl[~none].abs().max().item())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (1, 5), (2, 16), (4, 40), (8, 3), (1, 64), (1, 128), (3, 24)])
def test_rows(io, T, H):
    compare(T * 100 + H, [130, 64, 7, 300], T, H, 128, 32, 16, io)


@pytest.mark.parametrize("dc,dr", [(512, 64), (256, 64), (448, 0), (72, 16)])
@pytest.mark.parametrize("T,H", [(2, 24), (1, 49), (5, 13), (2, 40), (1, 81), (2, 48), (3, 43), (2, 80), (7, 23)])
def test_group_sizes(T, H, dc, dr):
    """48 to 161 query rows: every size of a worker's group, alone and in pairs that share the cache's loads."""
    compare(T * 200 + H + dc, [300, 0, 65, 700], T, H, dc, dr, 16, "bf16")


@pytest.mark.parametrize("n", [[20000], [3000, 1, 12000, 0, 500]])
@pytest.mark.parametrize("T,H", [(2, 40), (4, 40)])
def test_long_drafts(n, T, H):
    """Many tiles a worker, so that every ring goes round, with a new piece in between."""
    compare(len(n) + T, n, T, H, 512, 64, 64, "bf16")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dc,dr", [(256, 64), (512, 64), (512, 0), (64, 16), (8, 8), (200, 24), (448, 48), (72, 0)])
def test_widths(io, dc, dr):
    compare(dc + dr, [100, 1, 257], 2, 16, dc, dr, 32, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 200])
def test_pages(io, page):
    compare(page, [65, 3, 200, 128, 127], 1, 16, 128, 64, page, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 4])
def test_lengths_from_none(io, T):
    """No rows, fewer rows than drafted tokens (their first ones see nothing), and every edge of a tile."""
    compare(T, [0, 1, 2, 3, 0, 63, 64, 65, 127, 128, 129, 0], T, 4, 64, 32, 16, io)


@pytest.mark.parametrize("n", [[20000], [9001, 1, 0, 12345, 4000], [64] * 200, [1] * 33, [0] * 5])
def test_split_and_join(n):
    """One long sequence over all workers, uneven ones, many that share a worker, none."""
    compare(len(n), n, 1, 16, 64, 32, 64, "bf16")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,T,H,dc", [([5000, 0, 3000], 1, 16, 512), ([2500, 1900, 0, 700], 8, 32, 200), ([150], 1, 5, 72),
                                      ([900, 0] + [700] * 6, 8, 9, 264)])
def test_both_joins(n, T, H, dc, io):
    """Rows x sequences on both sides of 4096, where the join of a sequence's pieces changes its form."""
    compare(T + H, n, T, H, dc, 16, 16, io)


def test_sharp_scores():
    """One row takes almost all the weight, and the largest score moves from tile to tile."""
    compare(77, [1000, 333], 1, 16, 256, 64, 64, "bf16", std=8.0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_shared_pages_and_bad_entries(io):
    """Two sequences share a prefix's pages; a page number outside the cache reads as rows of zeros; a length past the
    table is cut to it."""
    H, dc, dr, page = 4, 64, 32, 16
    g = gen(5)
    cache = normal(g, (6, page, dc + dr), io)
    table = torch.tensor([[3, 1, 0], [3, 1, 5], [2, 99, 4], [2, -7, 4]], dtype=torch.int32)
    n = [40, 48, 45, 48]
    qc, qr = normal(g, (4, 1, H, dc), io), normal(g, (4, 1, H, dr), io)
    o, _ = call(n, 1, H, dc, dr, page, io, table, 6, cache, qc, qr, 0.1, lens=[40, 1000, 45, 48])
    zero = torch.zeros(page, dc + dr, dtype=cache.dtype)
    for b in range(4):
        rows = torch.cat([cache[p] if 0 <= p < 6 else zero for p in table[b].tolist()])[: n[b]]
        close(o[b].cpu(), decode_ref(qc[b], qr[b], rows, 0.1)[0], io, "fwd", f"o {b}")


def test_strided_queries_streams_and_bits():
    """Queries as slices of wider rows; the same bits on another stream and in another call."""
    n, H, dc, dr, page = [500, 77, 3000], 16, 128, 64, 32
    table, pages, cache, rows, qc, qr = setup(6, n, 1, H, dc, dr, page, "bf16")
    a = call(n, 1, H, dc, dr, page, "bf16", table, pages, cache, qc, qr, 0.1)
    both = torch.full((3, 1, H, dc + dr + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    both[..., :dc], both[..., dc: dc + dr] = qc.cuda(), qr.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = call(n, 1, H, dc, dr, page, "bf16", table, pages, cache, both[..., :dc], both[..., dc: dc + dr], 0.1)
    st.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("past", [2, 3])
def test_long_cache_offsets(past):
    """Rows beyond 2^31 elements of the cache (offsets that pass 32 bits): pages at its far end."""
    dc, dr, page, H = 512, 64, 64, 8
    pages = past * (1 << 30) // (page * (dc + dr)) + 3
    cache = torch.empty((pages, page, dc + dr), dtype=torch.bfloat16, device="cuda")
    g = gen(7)
    n = [130]
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32)
    data = normal(g, (3, page, dc + dr), "bf16")
    for i in range(3):
        cache[table[0, i]] = data[i].cuda()
    qc, qr = normal(g, (1, 1, H, dc), "bf16", 0.5), normal(g, (1, 1, H, dr), "bf16")
    o, _ = call(n, 1, H, dc, dr, page, "bf16", table, pages, cache, qc, qr, 0.1)
    close(o[0], decode_ref(qc[0], qr[0], data.flatten(0, 1)[:130], 0.1)[0], "bf16", "fwd", "o")


@pytest.mark.parametrize("T,H", [(2, 6), (4, 40)])
def test_some_heads_of_a_wider_query(T, H):
    """Queries that are the first heads of a tensor with more: rows of one token lie apart from the next one's."""
    n, dc, dr, page = [500, 77, 130], 128, 64, 32
    table, pages, cache, rows, qc, qr = setup(8, n, T, H, dc, dr, page, "bf16")
    a = call(n, T, H, dc, dr, page, "bf16", table, pages, cache, qc, qr, 0.1)
    wide = torch.full((3, T, H + 3, dc + dr), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :H, :dc], wide[:, :, :H, dc:] = qc.cuda(), qr.cuda()
    b = call(n, T, H, dc, dr, page, "bf16", table, pages, cache, wide[:, :, :H, :dc], wide[:, :, :H, dc:], 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
