"""gdn_norm_fwd and gdn_norm_bwd against 64 bits: types, widths, 8-bit groups, strides, aliases, NaN rows."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import EPS, close, gen, nan, normal, tdtype

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def inputs(N, D, io, res, pad=0):
    g = gen(N + D)
    x, r = normal(g, (N, D + pad), io)[:, :D], normal(g, (N, D + pad), res, 3.0)[:, :D]
    return g, x, r, 1.0 + 0.2 * torch.randn(D, generator=g)


def kept(x, r, res):
    return (x.float() + r.float()).to(tdtype(res)) if r is not None else x.to(tdtype(res))


def norm_ref(s, w):
    return s / (s.square().mean(-1, keepdim=True) + EPS).sqrt() * w


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("N,D,pad", [(1, 8, 0), (24, 2048, 0), (37, 264, 8), (9, 520, 0), (5, 2056, 8), (3, 4096, 0), (4, 8192, 0),
                                     (2, 16384, 16), (1300, 64, 0)])
def test_forward_and_gradients(io, res, N, D, pad):
    g, x, r, w = inputs(N, D, io, res, pad)
    s = gdn.make_norm(N, D, io, res)
    y, total = nan((N, D + pad), tdtype(io))[:, :D], nan((N, D), tdtype(res))
    dev = [t.cuda() for t in (x, r, w)]
    gdn.check(gdn.gdn_norm_fwd(s, *dev, y, None, total))
    want = kept(x, r, res)
    assert torch.equal(total.cpu(), want)
    leaf, wl = want.double().requires_grad_(), w.double().requires_grad_()
    ref = norm_ref(leaf, wl)
    close(y, ref, "sum", "y")
    dy, ds = normal(g, (N, D + pad), io)[:, :D], normal(g, (N, D), res)
    loss = (ref * dy.double()).sum()
    d, dw = torch.autograd.grad(loss, [leaf, wl])
    ws = torch.full((gdn.gdn_norm_workspace_bytes(s),), 255, dtype=torch.uint8, device="cuda")
    for grad in (ds, None):
        dx, dres, gw = nan((N, D), tdtype(io)), nan((N, D), tdtype(res)), nan((D,), torch.float32)
        gdn.check(gdn.gdn_norm_bwd(s, total, dev[2], dy.cuda(), None if grad is None else grad.cuda(), dx, dres, gw, ws))
        both = d if grad is None else d + grad.double()
        close(dx, both, "sum", "dx")
        close(dres, both, "sum", "dres")
        close(gw, dw, "sum", "dw")
    again, only = nan((D,), torch.float32), nan((N, D), tdtype(io))
    gdn.check(gdn.gdn_norm_bwd(s, total, dev[2], dy.cuda(), None, only, None, again, ws))
    assert torch.equal(only, dx) and torch.equal(again, gw)


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("N,D,group", [(1, 32, 32), (24, 2048, 0), (7, 8, 0), (5, 264, 0), (6, 4096, 128), (3, 192, 64), (33, 16384, 128),
                                       (2, 16384, 0), (9, 96, 32), (4, 640, 128)])
def test_eight_bits(io, res, N, D, group):
    """A value is y / scale rounded to e4m3, so it is within half a step (2^-4 of it) or half the smallest one (2^-10)."""
    _, x, r, w = inputs(N, D, io, res)
    s = gdn.make_norm(N, D, io, res, "e4m3", group)
    y = torch.full((N, D), 1.0, device="cuda").to(torch.float8_e4m3fn)
    parts = D // group if group else 1
    scale, total = nan((N, parts), torch.float32), nan((N, D), tdtype(res))
    gdn.check(gdn.gdn_norm_fwd(s, x.cuda(), r.cuda(), w.cuda(), y, scale, total))
    want = kept(x, r, res)
    assert torch.equal(total.cpu(), want)
    ref = norm_ref(want.double(), w.double()).view(N, parts, -1)
    close(scale, ref.abs().amax(-1) / 448, "sum", "scale")
    value = ref / scale.cpu().double()[..., None]
    off = (y.cpu().double().view(N, parts, -1) - value).abs()
    assert (off <= value.abs().clamp(min=2.0 ** -6) * (2.0 ** -4 + 1e-5)).all()
    assert (y.cpu().float().view(N, parts, -1).abs().amax(-1) == 448).all()


def test_rows_of_zeros_and_nan():
    """A row of zeros gives zeros and the least scale; a NaN or an infinity stays in its row and shows in its scales."""
    N, D = 6, 256
    _, x, r, w = inputs(N, D, "bf16", "bf16")
    x[1], r[1] = 0, 0
    x[3, 7], x[4, 200] = math.nan, math.inf
    for group in (0, 64):
        s = gdn.make_norm(N, D, "bf16", None, "e4m3", group)
        y, scale = torch.empty((N, D), device="cuda", dtype=torch.float8_e4m3fn), nan((N, D // group if group else 1), torch.float32)
        gdn.check(gdn.gdn_norm_fwd(s, x.cuda(), r.cuda(), w.cuda(), y, scale, None))
        v, sc = y.float().cpu(), scale.cpu()
        assert (v[1] == 0).all() and torch.allclose(sc[1], torch.tensor(1e-30 / 448))
        assert v[3].isnan().all() and sc[3].isnan().all()
        assert v[4, 200].isnan() and sc[4].isnan().any()
        fine = [0, 2, 5]
        assert torch.isfinite(v[fine]).all() and torch.isfinite(sc[fine]).all()
    s = gdn.make_norm(N, D)
    y = nan((N, D), torch.bfloat16)
    gdn.check(gdn.gdn_norm_fwd(s, x.cuda(), r.cuda(), w.cuda(), y, None, None))
    assert (y[1] == 0).all() and y[3].isnan().all() and torch.isfinite(y[[0, 2, 5]].float()).all()


@pytest.mark.parametrize("io,res", TYPES)
def test_aliases_and_no_residual(io, res):
    N, D = 19, 512
    g, x, r, w = inputs(N, D, io, res)
    s = gdn.make_norm(N, D, io, res)
    y, stream_ = nan((N, D), tdtype(io)), r.cuda()
    gdn.check(gdn.gdn_norm_fwd(s, x.cuda(), stream_, w.cuda(), y, None, stream_))      # the residual stream in place
    want = kept(x, r, res)
    assert torch.equal(stream_.cpu(), want)
    close(y, norm_ref(want.double(), w.double()), "sum", "y")
    gdn.check(gdn.gdn_norm_fwd(s, x.cuda(), None, w.cuda(), y, None, None))            # a first layer: nothing to add
    close(y, norm_ref(kept(x, None, res).double(), w.double()), "sum", "y alone")
    dy, ds = normal(g, (N, D), io), normal(g, (N, D), res)
    ws = torch.empty(gdn.gdn_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    apart, inplace, dw = nan((N, D), tdtype(res)), ds.cuda(), nan((D,), torch.float32)
    gdn.check(gdn.gdn_norm_bwd(s, stream_, w.cuda(), dy.cuda(), ds.cuda(), None, apart, dw, ws))
    gdn.check(gdn.gdn_norm_bwd(s, stream_, w.cuda(), dy.cuda(), inplace, None, inplace, dw, ws))
    assert torch.equal(apart, inplace)


def test_no_rows():
    s = gdn.make_norm(0, 64)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w, dw = torch.ones(64, device="cuda"), nan((64,), torch.float32)
    assert gdn.gdn_norm_fwd(s, empty, empty, w, empty, None, empty) == gdn.GDN_OK
    ws = torch.empty(gdn.gdn_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    gdn.check(gdn.gdn_norm_bwd(s, empty, w, empty, None, empty, None, dw, ws))
    assert (dw == 0).all()


def test_rows_beyond_32_bits():
    """Rows so far apart that their offsets pass 2^31 elements."""
    N, D, far = 3, 64, 1 << 30
    _, x, r, w = inputs(N, D, "bf16", "bf16")
    wide = torch.empty(2 * far + D, dtype=torch.bfloat16, device="cuda").as_strided((N, D), (far, 1))
    wide.copy_(x)
    s = gdn.make_norm(N, D)
    y = nan((N, D), torch.bfloat16)
    gdn.check(gdn.gdn_norm_fwd(s, wide, r.cuda(), w.cuda(), y, None, None))
    close(y, norm_ref(kept(x, r, "bf16").double(), w.double()), "sum", "y")
