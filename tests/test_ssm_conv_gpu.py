"""gdn_conv_fwd, gdn_conv_bwd and gdn_conv_step against 64 bits: taps, lengths from zero on, states, slots, strides."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import close, conv_all, conv_ref, gen, nan, normal, offsets, tdtype

pytestmark = pytest.mark.gpu

LENS = [[1], [2, 0, 5], [63, 64, 65, 1], [200, 3, 0, 129], [0, 0]]


def inputs(lens, D, W, io, gap=0, pad=0, bias=True):
    g, rows = gen(D + W + sum(lens)), sum(lens) + gap + pad
    x = normal(g, (rows, 2 * D), io)[:, :D]
    return (g, x, torch.randn((D, W), generator=g) / math.sqrt(W), 0.1 * torch.randn(D, generator=g) if bias else None,
            normal(g, (len(lens), W - 1, D), io), normal(g, (rows, D), io), normal(g, (len(lens), W - 1, D), io))


def dev(t):
    return None if t is None else torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,silu,bias,state", [(8, True, True, True), (136, False, True, True), (520, True, False, False)])
@pytest.mark.parametrize("lens", LENS)
def test_sequences_and_gradients(io, W, D, silu, bias, state, lens):
    gap, pad = 2, 3
    g, x, w, b, s0, dy, dsT = inputs(lens, D, W, io, gap, pad, bias)
    rows, cu = x.shape[0], offsets(lens, gap)
    own = torch.zeros(rows, dtype=torch.bool)
    own[gap: gap + sum(lens)] = True
    leaf = [None if t is None else t.double().requires_grad_() for t in (x, w, b, s0 if state else torch.zeros_like(s0))]
    ref, refT = conv_all(*leaf, lens, silu, gap)
    s = gdn.make_conv(len(lens), max(lens), D, W, io, silu, rows) if max(lens) else gdn.make_conv(len(lens), 1, D, W, io, silu, rows)
    dx_, dw_, db_, ds_ = None, None, None, None
    args = (dev(x), dev(w), dev(b), cu.cuda(), dev(s0) if state else None)
    y, sT = nan((rows, D), tdtype(io)), nan(s0.shape, tdtype(io))
    gdn.check(gdn.gdn_conv_fwd(s, *args, y, sT))
    close(y, ref, "sum", "y", own)
    assert y.cpu()[~own].isnan().all()
    assert torch.equal(sT.cpu().double(), refT.detach())                       # inputs, moved
    used = [t for t in leaf if t is not None]
    loss = (ref[own] * dy.double()[own]).sum() + (refT * dsT.double()).sum()
    dx_, dw_, *db_, ds_ = [torch.zeros_like(t) if d is None else d
                           for t, d in zip(used, torch.autograd.grad(loss, used, allow_unused=True))]
    dx, dw, db = nan((rows, D), tdtype(io)), nan((D, W), torch.float32), nan((D,), torch.float32) if bias else None
    ds0 = nan(s0.shape, tdtype(io)) if state else None
    ws = torch.full((gdn.gdn_conv_workspace_bytes(s),), 255, dtype=torch.uint8, device="cuda")
    call = lambda: gdn.check(gdn.gdn_conv_bwd(s, *args, dev(dy), dev(dsT), dx, dw, db, ds0, ws))  # noqa: E731
    call()
    close(dx, dx_, "sum", "dx", own)
    assert dx.cpu()[~own].isnan().all()
    close(dw, dw_, "sum", "dw")
    if bias:
        close(db, db_[0], "sum", "dbias")
    if state:
        close(ds0, ds_, "sum", "ds0")
    first = dw.clone()
    call()
    assert torch.equal(first, dw)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_equal_sequences_without_offsets(io):
    """[B, T, D] tensors, no state in, no state gradient: a training batch."""
    B, T, D, W = 3, 70, 64, 4
    g, x, w, b, _, dy, _ = inputs([T] * B, D, W, io)
    leaf = [t.double().requires_grad_() for t in (x, w, b)]
    ref, _ = conv_all(*leaf, torch.zeros(B, W - 1, D, dtype=torch.float64), [T] * B, True)
    d = torch.autograd.grad((ref * dy.double()).sum(), leaf)
    s = gdn.make_conv(B, T, D, W, io)
    xs, y, dx = dev(x).unflatten(0, (B, T)), nan((B, T, D), tdtype(io)), nan((B, T, D), tdtype(io))
    dw, db = nan((D, W), torch.float32), nan((D,), torch.float32)
    gdn.check(gdn.gdn_conv_fwd(s, xs, dev(w), dev(b), None, None, y, None))
    ws = torch.empty(gdn.gdn_conv_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_conv_bwd(s, xs, dev(w), dev(b), None, None, dev(dy).view(B, T, D), None, dx, dw, db, None, ws))
    close(y.flatten(0, 1), ref, "sum", "y")
    for got, want, name in ((dx.flatten(0, 1), d[0], "dx"), (dw, d[1], "dw"), (db, d[2], "dbias")):
        close(got, want, "sum", name)


def test_cut_and_bad_offsets():
    """Sequences over T rows are cut there; offsets outside the tensor count as its bounds, descending ones as nothing."""
    D, W, rows = 16, 4, 40
    g, x, w, b, s0, _, _ = inputs([rows], D, W, "f32")
    s0 = normal(g, (4, W - 1, D), "f32")
    cu = torch.tensor([-5, 12, 30, 24, 99], dtype=torch.int32)
    s = gdn.make_conv(4, 10, D, W, "f32", rows=rows)
    y, sT = nan((rows, D), torch.float32), nan(s0.shape, torch.float32)
    gdn.check(gdn.gdn_conv_fwd(s, dev(x), dev(w), dev(b), cu.cuda(), dev(s0), y, sT))
    seen = torch.zeros(rows, dtype=torch.bool)
    for q, (at, n) in enumerate(((0, 10), (12, 10), (30, 0), (24, 10))):
        want, state = conv_ref(x[at: at + n].double(), w.double(), b.double(), s0[q].double(), True)
        close(y.cpu()[at: at + n], want, "sum", f"y of {q}")
        assert torch.equal(sT[q].cpu().double(), state)
        seen[at: at + n] = True
    assert y.cpu()[~seen].isnan().all()


def test_nothing_crosses_sequences():
    lens, D, W = [40, 33, 70], 24, 4
    g, x, w, b, s0, dy, dsT = inputs(lens, D, W, "bf16")
    x[40:73], s0[1], dy[40:73] = math.nan, math.inf, math.nan
    s = gdn.make_conv(3, 70, D, W, "bf16", rows=143)
    args = (dev(x), dev(w), dev(b), offsets(lens).cuda(), dev(s0))
    y, sT, dx, ds0 = nan((143, D), torch.bfloat16), nan(s0.shape, torch.bfloat16), nan((143, D), torch.bfloat16), nan(s0.shape, torch.bfloat16)
    dw, db = nan((D, W), torch.float32), nan((D,), torch.float32)
    ws = torch.empty(gdn.gdn_conv_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_conv_fwd(s, *args, y, sT))
    gdn.check(gdn.gdn_conv_bwd(s, *args, dev(dy), dev(dsT), dx, dw, db, ds0, ws))
    keep = torch.ones(143, dtype=torch.bool)
    keep[40:73] = False
    for t in (y, dx):
        assert torch.isfinite(t.cpu()[keep]).all()
    assert torch.isfinite(sT[[0, 2]]).all() and torch.isfinite(ds0[[0, 2]]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,W,silu", [(1, 1, 8, 4, True), (24, 1, 4096, 4, True), (7, 3, 136, 2, False), (5, 8, 64, 3, True)])
def test_new_tokens(io, B, T, D, W, silu):
    """States by slot: in place, from one slot to another, from none (zeros), to none (a place without a request)."""
    g = gen(B + T + D)
    x, w, b = normal(g, (B * T, 2 * D), io)[:, :D], torch.randn((D, W), generator=g) / 2, 0.1 * torch.randn(D, generator=g)
    slots = 2 * B + 3
    pool, order = normal(g, (slots, W - 1, D), io), torch.randperm(slots, generator=g).int()
    src, dst = order[:B].clone(), order[B: 2 * B].clone()
    s = gdn.make_conv_step(B, T, D, W, slots, io, silu)

    def check(src, dst):
        y, state = nan((B * T, D), tdtype(io)), pool.cuda()
        gdn.check(gdn.gdn_conv_step(s, dev(x), dev(w), dev(b), state, None if src is None else src.cuda(),
                                    None if dst is None else dst.cuda(), y))
        want = pool.clone().double()
        a = list(range(B)) if src is None else src.tolist()
        for q in range(B):
            before = pool[a[q]].double() if 0 <= a[q] < slots else torch.zeros(W - 1, D, dtype=torch.float64)
            ref, after = conv_ref(x[q * T: (q + 1) * T].double(), w.double(), b.double(), before, silu)
            close(y[q * T: (q + 1) * T], ref, "sum", f"y of {q}")
            to = a[q] if dst is None else dst.tolist()[q]
            if 0 <= to < slots:
                want[to] = after
        assert torch.equal(state.cpu().double(), want)

    check(None, None)
    check(src, None)
    check(src, dst)
    if B > 1:
        src[0], src[1] = -1, slots
        check(src, None)
        dst[0], dst[B - 1] = slots, -7
        check(src, dst)


def test_prompt_then_tokens():
    """A prompt's state goes on token by token as the whole sequence would have."""
    D, W, n, more = 40, 4, 21, 6
    g, x, w, b, _, _, _ = inputs([n + more], D, W, "f32")
    y, sT = nan((n, D), torch.float32), nan((1, W - 1, D), torch.float32)
    gdn.check(gdn.gdn_conv_fwd(gdn.make_conv(1, n, D, W, "f32"), dev(x[:n]), dev(w), dev(b), None, None, y, sT))
    step, rows = gdn.make_conv_step(1, 1, D, W, 1, "f32"), [y]
    for t in range(n, n + more):
        o = nan((1, D), torch.float32)
        gdn.check(gdn.gdn_conv_step(step, dev(x[t: t + 1]), dev(w), dev(b), sT, None, None, o))
        rows.append(o)
    whole = nan((n + more, D), torch.float32)
    gdn.check(gdn.gdn_conv_fwd(gdn.make_conv(1, n + more, D, W, "f32"), dev(x), dev(w), dev(b), None, None, whole, None))
    assert torch.equal(torch.cat(rows), whole)
