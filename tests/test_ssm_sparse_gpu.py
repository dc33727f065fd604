"""The convolution and the scan over batches of which T is far more than the average length: one long sequence among many, many
empty ones, T only a bound.  The calls then look up whose rows they work on."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import ORDER, close, conv_all, cuda, gen, nan, normal, offsets, scan_inputs, tdtype
from tests.test_ssm_scan_gpu import compare

pytestmark = pytest.mark.gpu

# lengths, rows of nobody in front and behind; T is all rows
BATCHES = [([0, 3, 0, 0, 1, 400, 0, 2, 9, 0, 0, 31, 32, 33, 0], 70, 40), ([1] * 150, 0, 0), ([0] * 20 + [257] + [0] * 19, 1, 0),
           ([90, 64, 64, 129, 128, 127], 0, 3), ([0] * 6 + [1], 33, 0), ([0] * 9, 0, 5), ([800] + [7] * 30, 0, 0), ([7] * 30 + [800], 600, 600)]


@pytest.mark.parametrize("io,D,N,G", [("f32", 40, 24, 1), ("bf16", 96, 16, 1), ("f32", 64, 8, 2), ("bf16", 16, 64, 1)])
@pytest.mark.parametrize("lens,gap,pad", BATCHES)
def test_scan(io, D, N, G, lens, gap, pad):
    rows = sum(lens) + gap + pad
    assert len(lens) * rows > 4 * rows
    compare(scan_inputs(rows, lens, D, N, G, io, gap=gap, pad=pad), lens, io, gap, pad, T=rows)


@pytest.mark.parametrize("io,D,W,silu", [("f32", 8, 4, True), ("bf16", 136, 3, False), ("bf16", 520, 4, True), ("f32", 24, 2, True)])
@pytest.mark.parametrize("lens,gap,pad", BATCHES)
def test_conv(io, D, W, silu, lens, gap, pad):
    rows, B, g = sum(lens) + gap + pad, len(lens), gen(D + W)
    x, w, b, dy = normal(g, (rows, D), io), torch.randn((D, W), generator=g) / math.sqrt(W), 0.1 * torch.randn(D, generator=g), normal(g, (rows, D), io)
    s0, dsT = normal(g, (B, W - 1, D), io), normal(g, (B, W - 1, D), io)
    own = torch.zeros(rows, dtype=torch.bool)
    own[gap: gap + sum(lens)] = True
    leaf = [t.double().requires_grad_() for t in (x, w, b, s0)]
    ref, refT = conv_all(*leaf, lens, silu, gap)
    loss = (ref[own] * dy.double()[own]).sum() + (refT * dsT.double()).sum()
    want = [torch.zeros_like(t) if d is None else d for t, d in zip(leaf, torch.autograd.grad(loss, leaf, allow_unused=True))]
    s = gdn.make_conv(B, rows, D, W, io, silu, rows)
    args = (x.cuda(), w.cuda(), b.cuda(), offsets(lens, gap).cuda(), s0.cuda())
    y, sT = nan((rows, D), tdtype(io)), nan(s0.shape, tdtype(io))
    gdn.check(gdn.gdn_conv_fwd(s, *args, y, sT))
    close(y, ref, "sum", "y", own)
    assert torch.equal(sT.cpu().double(), refT.detach())
    dx, dw, db, ds0 = nan(y.shape, y.dtype), nan(w.shape, torch.float32), nan((D,), torch.float32), nan(s0.shape, s0.dtype)
    ws = torch.full((gdn.gdn_conv_workspace_bytes(s),), 255, dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_conv_bwd(s, *args, dy.cuda(), dsT.cuda(), dx, dw, db, ds0, ws))
    close(dx, want[0], "sum", "dx", own)
    for t in (y, dx):
        assert t.cpu()[~own].isnan().all()
    for got, ref, name in ((dw, want[1], "dw"), (db, want[2], "dbias"), (ds0, want[3], "ds0")):
        close(got, ref, "sum", name)


def test_the_longest_length_and_a_bound_agree():
    """A sequence's results do not depend on T beyond its length: those of the convolution to the bit."""
    lens, D = [5, 900, 0, 44, 1, 1, 260, 3], 64
    g, rows = gen(1), sum(lens)
    x, w, cu = normal(g, (rows, D), "bf16").cuda(), torch.randn((D, 4), generator=g).cuda(), offsets(lens).cuda()
    out = []
    for T in (max(lens), rows):
        for B in (len(lens), len(lens) + 60):
            more = torch.cat([cu, torch.full((B - len(lens),), rows, dtype=torch.int32, device="cuda")])
            y, sT = nan((rows, D), torch.bfloat16), nan((B, 3, D), torch.bfloat16)
            gdn.check(gdn.gdn_conv_fwd(gdn.make_conv(B, T, D, 4, rows=rows), x, w, None, more, None, y, sT))
            out.append((y, sT[:len(lens)]))
    for y, sT in out[1:]:
        assert torch.equal(y, out[0][0]) and torch.equal(sT, out[0][1])


@pytest.mark.parametrize("lens,bound", [([700, 90, 260], False), ([900] + [3] * 30, True)])
def test_calls_behind_one_another_share_a_workspace(lens, bound):
    """Training steps of different inputs through one workspace and one `saved`, enqueued without a wait, give the bits of steps
    alone: a split call's launches overlap with one another, and with nothing else."""
    D, N, rows, B = 72, 16, sum(lens), len(lens)
    cu, T = offsets(lens).cuda(), rows if bound else max(lens)
    s = gdn.make_scan(B, T, D, N, 1, "bf16", rows=rows)
    ws, saved = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (gdn.gdn_scan_workspace_bytes(s, 1), gdn.gdn_scan_saved_bytes(s)))
    sets = [cuda(scan_inputs(k, lens, D, N, 1, "bf16")) for k in range(3)]

    def step(i):
        args = [i[k] for k in ORDER]
        out = {"y": nan((rows, D), torch.bfloat16), "hT": nan((B, D, N), torch.float32),
               **{k: nan(i[k].shape, i[k].dtype) for k in ORDER + ("h0",)}}
        gdn.check(gdn.gdn_scan_fwd(s, *args, cu, i["h0"], out["y"], out["hT"], saved, ws))
        gdn.check(gdn.gdn_scan_bwd(s, *args, cu, saved, i["dy"], i["dhT"], *[out[k] for k in ORDER], out["h0"], ws))
        return out

    alone = []
    for i in sets:
        alone.append(step(i))
        torch.cuda.synchronize()
    for _ in range(10):
        for got, want in zip([step(i) for i in sets], alone):
            for k in want:
                assert torch.isfinite(want[k]).all() and torch.equal(got[k], want[k]), k
