"""The state-space entry points refuse bad arguments before any device work, and size their workspaces; the 64-bit
definitions that the GPU tests compare against, checked against closed forms and differences (no GPU)."""
import ctypes
import math
import os
import re

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import conv_all, scan_all, scan_grads, scan_inputs

FAKE = 1 << 20        # a 256-byte aligned address; never dereferenced
BIG = 1 << 40
OK, NULL, SHAPE, ALIGN, MODE, WS = 0, 1, 2, 3, 4, 5
ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from linear_attention_recurrence_delta_gb300 import _build
        _build.build()
    return gdn.load()


def view(p=FAKE, tok=1024, head=128):
    return gdn.gdn_mla_view_t(p, tok, head)


def refused(status, want):
    assert int(status) == want, f"{gdn.gdn_status_string(int(status))}, not {gdn.STATUS_NAMES[want]}"


def test_every_declared_function_is_exported(lib):
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn_ssm.h")
    names = set(re.findall(r"\b(gdn_(?:norm|conv|scan)_\w+)\(", open(header).read()))
    assert len(names) == 12
    for n in names:
        assert hasattr(lib, n) and hasattr(gdn, n), n


# ---------------------------------------------------------------- norm

NORM = dict(N=8, D=256, io="bf16", res=None, out=None, group=0)


def norm(**kw):
    return gdn.make_norm(**{**NORM, **kw})


def norm_fwd(s, **kw):
    a = dict(x=(FAKE, 256), res=(FAKE, 256), w=FAKE, y=(FAKE, 256), scale=None, sum=(FAKE, 256))
    a.update(kw)
    return gdn.load().gdn_norm_fwd(ref(s), *a["x"], *a["res"], a["w"], *a["y"], a["scale"], *a["sum"], 0)


def norm_bwd(s, **kw):
    a = dict(sum=(FAKE, 256), w=FAKE, dy=(FAKE, 256), dsum=(FAKE, 256), dx=(FAKE, 256), dres=(FAKE, 256), dw=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    return gdn.load().gdn_norm_bwd(ref(s), *a["sum"], a["w"], *a["dy"], *a["dsum"], *a["dx"], *a["dres"], a["dw"], a["ws"], a["n"], 0)


def test_norm_refusals():
    refused(norm_fwd(None), NULL)
    for bad, want in ((dict(N=-1), SHAPE), (dict(N=(1 << 30) + 1), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE), (dict(D=16392), SHAPE), (dict(eps=-1.0), SHAPE),
                      (dict(eps=math.nan), SHAPE), (dict(io=7), MODE), (dict(res=7), MODE), (dict(out=7), MODE), (dict(out="f32"), MODE),
                      (dict(io="f32", res="bf16"), MODE), (dict(out="e4m3", group=16), SHAPE), (dict(out="e4m3", D=264, group=128), SHAPE),
                      (dict(group=128), SHAPE), (dict(out="e4m3", group=-32), SHAPE)):
        refused(norm_fwd(norm(**bad)), want)
        refused(norm_bwd(norm(**bad)), want)
        assert gdn.gdn_norm_workspace_bytes(norm(**bad)) == 0
    s, q = norm(), norm(out="e4m3", group=32)
    refused(norm_fwd(s, x=(None, 256)), NULL)
    refused(norm_fwd(s, y=(None, 256)), NULL)
    refused(norm_fwd(s, w=None), NULL)
    refused(norm_fwd(q), NULL)                              # no place for the scales
    refused(norm_fwd(s, scale=FAKE), MODE)                  # scales without 8-bit values
    for k in ("x", "res", "y", "sum"):
        refused(norm_fwd(s, **{k: (FAKE, 248)}), SHAPE)
        refused(norm_fwd(s, **{k: (FAKE, 260)}), ALIGN)
        refused(norm_fwd(s, **{k: (FAKE + 8, 256)}), ALIGN)
    refused(norm_fwd(s, w=FAKE + 4), ALIGN)
    refused(norm_fwd(q, scale=FAKE + 2), ALIGN)
    refused(norm_fwd(norm(io="f32", out="e4m3"), scale=FAKE, y=(FAKE, 260)), ALIGN)      # 8-bit rows want whole pieces of 8
    refused(norm_fwd(norm(N=0), x=(None, 0), w=None), OK)
    need = gdn.gdn_norm_workspace_bytes(s)
    assert need >= 256 and need % 256 == 0
    for k in ("sum", "dy"):
        refused(norm_bwd(s, **{k: (None, 256)}), NULL)
    for k in ("sum", "dy", "dsum", "dx", "dres"):
        refused(norm_bwd(s, **{k: (FAKE, 8)}), SHAPE)
        refused(norm_bwd(s, **{k: (FAKE + 4, 256)}), ALIGN)
    refused(norm_bwd(s, w=None), NULL)
    refused(norm_bwd(s, dw=None), NULL)
    refused(norm_bwd(s, ws=None), WS)
    refused(norm_bwd(s, n=need - 1), WS)
    refused(norm_bwd(s, ws=FAKE + 128), ALIGN)


# ---------------------------------------------------------------- convolution

CONV = dict(B=2, T=33, D=64, W=4)


def conv(backward, s, **kw):
    a = dict(x=view(), w=FAKE, bias=FAKE, cu=None, s0=FAKE, y=view(), sT=FAKE, dy=view(), dsT=FAKE, dx=view(), dw=FAKE, dbias=FAKE,
             ds0=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    ins = [ref(s), ref(a["x"]), a["w"], a["bias"], a["cu"], a["s0"]]
    if not backward:
        return gdn.load().gdn_conv_fwd(*ins, ref(a["y"]), a["sT"], 0)
    return gdn.load().gdn_conv_bwd(*ins, ref(a["dy"]), a["dsT"], ref(a["dx"]), a["dw"], a["dbias"], a["ds0"], a["ws"], a["n"], 0)


@pytest.mark.parametrize("backward", [0, 1])
def test_conv_refusals(backward):
    refused(conv(backward, None), NULL)
    for bad, want in ((dict(B=0), SHAPE), (dict(B=65536, rows=66), SHAPE), (dict(D=4), SHAPE), (dict(D=0), SHAPE), (dict(W=1), SHAPE),
                      (dict(W=5), SHAPE), (dict(T=-1), SHAPE), (dict(T=0, rows=5), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=65), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE), (dict(D=(1 << 24) + 8), SHAPE),
                      (dict(io=3), MODE)):
        refused(conv(backward, gdn.make_conv(**{**CONV, **bad})), want)
        if bad != dict(rows=65):                            # with offsets any number of rows will do
            assert gdn.gdn_conv_workspace_bytes(gdn.make_conv(**{**CONV, **bad})) == 0
    s = gdn.make_conv(**CONV)
    for k in ("dy", "dx") if backward else ("y",):
        refused(conv(backward, s, **{k: None}), NULL)
        refused(conv(backward, s, **{k: view(FAKE + 2)}), ALIGN)
    refused(conv(backward, s, x=view(tok=1028)), ALIGN)
    refused(conv(backward, s, x=view(tok=0)), SHAPE)
    refused(conv(backward, s, x=None), NULL)
    refused(conv(backward, s, w=None), NULL)
    for k in ("w", "bias", "s0", "dsT" if backward else "sT"):
        refused(conv(backward, s, **{k: FAKE + 8}), ALIGN)
    refused(conv(backward, s, cu=FAKE + 2), ALIGN)
    if backward:
        need = gdn.gdn_conv_workspace_bytes(s)
        assert need >= 256 and need % 256 == 0
        refused(conv(1, s, dw=None), NULL)
        refused(conv(1, s, dbias=None), NULL)
        refused(conv(1, s, bias=None), NULL)
        refused(conv(1, s, ws=None), WS)
        refused(conv(1, s, n=need - 1), WS)
        refused(conv(1, s, ws=FAKE + 64), ALIGN)
    else:
        refused(conv(0, gdn.make_conv(1, 0, 8, 4), x=None, y=None, sT=None), OK)


STEP = dict(B=4, T=1, D=64, slots=4)


def conv_step(s, **kw):
    a = dict(x=view(), w=FAKE, bias=FAKE, state=FAKE, src=FAKE, dst=None, y=view())
    a.update(kw)
    return gdn.load().gdn_conv_step(ref(s), ref(a["x"]), a["w"], a["bias"], a["state"], a["src"], a["dst"], ref(a["y"]), 0)


def test_conv_step_refusals():
    refused(conv_step(None), NULL)
    for bad, want in ((dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(T=9), SHAPE), (dict(D=12), SHAPE), (dict(W=5), SHAPE),
                      (dict(slots=0), SHAPE), (dict(io=2), MODE)):
        refused(conv_step(gdn.make_conv_step(**{**STEP, "W": 4, **bad})), want)
    s = gdn.make_conv_step(**STEP, W=4)
    refused(conv_step(gdn.make_conv_step(**{**STEP, "slots": 3}, W=4), src=None), SHAPE)      # sequence b is slot b
    for k in ("x", "w", "state", "y"):
        refused(conv_step(s, **{k: None}), NULL)
    for k in ("w", "bias", "state"):
        refused(conv_step(s, **{k: FAKE + 8}), ALIGN)
    for k in ("src", "dst"):
        refused(conv_step(s, **{k: FAKE + 1}), ALIGN)


# ---------------------------------------------------------------- scan

SCAN = dict(B=2, T=33, D=64, N=16, G=2)
VIEWS = ("x", "dt", "z", "Bm", "Cm")


def scan(backward, s, **kw):
    a = {k: view() for k in VIEWS + tuple("d" + v for v in VIEWS)}
    a.update(A=FAKE, skip=FAKE, bias=FAKE, cu=None, h0=FAKE, y=view(), hT=FAKE, saved=FAKE, sn=BIG, dy=view(), dhT=FAKE, dA=FAKE,
             dskip=FAKE, dbias=FAKE, dh0=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    ins = [ref(s)] + [ref(a[k]) for k in VIEWS] + [a["A"], a["skip"], a["bias"], a["cu"]]
    if not backward:
        return gdn.load().gdn_scan_fwd(*ins, a["h0"], ref(a["y"]), a["hT"], a["saved"], a["sn"], a["ws"], a["n"], 0)
    return gdn.load().gdn_scan_bwd(*ins, a["saved"], a["sn"], ref(a["dy"]), a["dhT"], *[ref(a["d" + k]) for k in VIEWS], a["dA"],
                                   a["dskip"], a["dbias"], a["dh0"], a["ws"], a["n"], 0)


@pytest.mark.parametrize("backward", [0, 1])
def test_scan_refusals(backward):
    refused(scan(backward, None), NULL)
    for bad, want in ((dict(B=0), SHAPE), (dict(B=65536, rows=66), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE), (dict(N=72), SHAPE),
                      (dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(D=72), SHAPE), (dict(D=0), SHAPE), (dict(T=-1), SHAPE),
                      (dict(T=0, rows=3), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=67), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE), (dict(D=1 << 26), SHAPE),
                      (dict(io=9), MODE)):
        refused(scan(backward, gdn.make_scan(**{**SCAN, **bad})), want)
        if bad != dict(rows=67):
            assert gdn.gdn_scan_workspace_bytes(gdn.make_scan(**{**SCAN, **bad}), backward) == 0
            assert gdn.gdn_scan_saved_bytes(gdn.make_scan(**{**SCAN, **bad})) == 0
    s = gdn.make_scan(**SCAN)
    for k in ("x", "dt", "Bm", "Cm") + (("dy", "dx", "ddt", "dz", "dBm", "dCm") if backward else ("y",)):
        refused(scan(backward, s, **{k: None}), NULL)
        refused(scan(backward, s, **{k: view(FAKE + 4)}), ALIGN)
        refused(scan(backward, s, **{k: view(tok=1020)}), ALIGN)
        refused(scan(backward, s, **{k: view(tok=-8)}), SHAPE)
    refused(scan(backward, s, Bm=view(head=-8)), SHAPE)
    refused(scan(backward, s, A=None), NULL)
    for k in ("A", "skip", "bias") + (("dhT", "dh0") if backward else ("h0", "hT")):
        refused(scan(backward, s, **{k: FAKE + 8}), ALIGN)
    refused(scan(backward, s, cu=FAKE + 2), ALIGN)
    need, kept = gdn.gdn_scan_workspace_bytes(s, backward), gdn.gdn_scan_saved_bytes(s)
    assert need >= 256 and need % 256 == 0 and kept >= 256 and kept % 256 == 0
    refused(scan(backward, s, ws=None), WS)
    refused(scan(backward, s, n=need - 1), WS)
    refused(scan(backward, s, ws=FAKE + 64), ALIGN)
    refused(scan(backward, s, sn=kept - 1), WS)
    refused(scan(backward, s, saved=FAKE + 16), ALIGN)
    if backward:
        refused(scan(1, s, saved=None), WS)
        for k in ("dA", "dskip", "dbias", "skip", "bias", "z"):
            refused(scan(1, s, **{k: None}), NULL)
    else:
        refused(scan(0, gdn.make_scan(1, 0, 8, 8), hT=None, **{k: None for k in VIEWS}, y=None), OK)


def scan_step(s, **kw):
    a = {k: view() for k in VIEWS}
    a.update(A=FAKE, skip=FAKE, bias=FAKE, state=FAKE, src=FAKE, dst=None, y=view())
    a.update(kw)
    return gdn.load().gdn_scan_step(ref(s), *[ref(a[k]) for k in VIEWS], a["A"], a["skip"], a["bias"], a["state"], a["src"], a["dst"],
                                    ref(a["y"]), 0)


def test_scan_step_refusals():
    refused(scan_step(None), NULL)
    for bad, want in ((dict(B=0), SHAPE), (dict(T=0), SHAPE), (dict(T=9), SHAPE), (dict(D=20), SHAPE), (dict(N=4), SHAPE), (dict(G=3), SHAPE),
                      (dict(slots=0), SHAPE), (dict(io=2), MODE)):
        refused(scan_step(gdn.make_scan_step(**{**STEP, "N": 16, **bad})), want)
    s = gdn.make_scan_step(**STEP, N=16)
    refused(scan_step(gdn.make_scan_step(**{**STEP, "slots": 3}, N=16), src=None), SHAPE)
    for k in ("x", "dt", "Bm", "Cm", "A", "state", "y"):
        refused(scan_step(s, **{k: None}), NULL)
    for k in ("A", "skip", "bias", "state"):
        refused(scan_step(s, **{k: FAKE + 8}), ALIGN)
    for k in ("src", "dst"):
        refused(scan_step(s, **{k: FAKE + 1}), ALIGN)


def test_workspaces_follow_the_rows():
    """Every valid shape has a workspace; sequences that T allows and the rows do not hold take next to none of it."""
    for back in (0, 1):
        for D in (64, 512, 2048):
            sizes = [gdn.gdn_scan_workspace_bytes(gdn.make_scan(1, T, D, 16, rows=20000), back) for T in (1, 100, 20000)]
            assert all(n >= 256 for n in sizes)
        one, many = (gdn.gdn_scan_workspace_bytes(gdn.make_scan(B, 16384, 2048, 16, rows=16384), back) for B in (1, 512))
        assert many <= one + 2 * 512 * 2048 * 18 * 4
    for B, T, D, N in ((8, 384, 2048, 8), (1, 384, 12992, 8), (3, 700, 40, 16), (12, 5000, 512, 64)):      # one area for both directions
        fwd, bwd = (gdn.gdn_scan_workspace_bytes(gdn.make_scan(B, T, D, N), back) for back in (0, 1))
        assert bwd >= fwd
    assert gdn.gdn_scan_saved_bytes(gdn.make_scan(4, 1000, 64, 16)) >= (4000 // 16 + 4) * 64 * 16 * 4


def test_binding_takes_views_and_refuses_other_tensors():
    x = torch.zeros(10, 64, dtype=torch.bfloat16)
    s = gdn.make_conv(1, 10, 32, 4)
    w, y = torch.zeros(32, 4), torch.zeros(10, 32, dtype=torch.bfloat16)
    for args in ((x.float()[:, :32], w, y), (x[:, :32], w.double(), y), (x[:, :32], w.half(), y), (x[:, :32], w, y.float()),
                 (x[:, :32], w.T, y), (x[:, ::2], w, y)):
        with pytest.raises(ValueError):
            gdn.gdn_conv_fwd(s, args[0], args[1], None, None, None, args[2], None)
    with pytest.raises(ValueError):
        gdn.gdn_conv_fwd(s, x[:, :32], w, None, torch.zeros(2, dtype=torch.int64), None, y, None)


# ---------------------------------------------------------------- the definitions

def test_scan_definition():
    """One state that never decays sums what is written; a constant decay gives a geometric sum; gradients are differences."""
    one = lambda *s: torch.ones(s, dtype=torch.float64)  # noqa: E731
    i = {"x": one(4, 8), "dt": 0.5 * one(4, 8), "z": None, "Bm": one(4, 1, 8), "Cm": one(4, 1, 8) / 8, "A_log": -100 * one(8, 8),
         "skip": None, "bias": None, "h0": torch.zeros(1, 8, 8, dtype=torch.float64)}
    y, h = scan_all(i, [4], softplus=False)
    assert torch.allclose(y[:, 0], torch.tensor([0.5, 1.0, 1.5, 2.0], dtype=torch.float64)) and torch.allclose(h, 2 * one(1, 8, 8))
    i["A_log"] = math.log(2 * math.log(2.0)) * one(8, 8)        # exp(-0.5 * 2 log 2) = 1/2
    y, _ = scan_all(i, [4], softplus=False)
    assert torch.allclose(y[:, 3], torch.tensor([0.5, 0.75, 0.875, 0.9375], dtype=torch.float64))
    i["dt"] = math.log(math.expm1(0.5)) * one(4, 8)
    assert torch.allclose(scan_all(i, [4])[0], y)
    lens = [4, 3]
    i = scan_inputs(1, lens, 16, 8, 2, "f32")
    _, _, grads = scan_grads(i, lens)
    x = {k: t.double() for k, t in i.items()}

    def loss(v):
        y, h = scan_all(v, lens)
        return ((y * x["dy"]).sum() + (h * x["dhT"]).sum()).item()

    for k, g in grads.items():
        v = torch.randn(g.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
        d = (loss({**x, k: x[k] + 1e-6 * v}) - loss({**x, k: x[k] - 1e-6 * v})) / 2e-6
        assert abs(d - (g * v).sum().item()) <= 1e-7 * max(1.0, abs(d)), k


def test_conv_definition():
    """A single tap of one at lag k delays by k; states join the sequences' ends."""
    x = torch.arange(1.0, 7.0, dtype=torch.float64)[:, None].expand(6, 8)
    s0 = -torch.arange(3.0, 0.0, -1.0, dtype=torch.float64)[None, :, None].expand(2, 3, 8)
    for k in range(4):
        w = torch.zeros(8, 4, dtype=torch.float64)
        w[:, 3 - k] = 1
        y, s = conv_all(x, w, None, s0, [4, 2], False)
        first = ([-1.0, -2.0, -3.0][:k][::-1] + [1.0, 2.0, 3.0, 4.0])[:4]
        second = ([-1.0, -2.0, -3.0][:k][::-1] + [5.0, 6.0])[:2]
        assert y[:, 0].tolist() == first + second
        assert s[0, :, 0].tolist() == [2.0, 3.0, 4.0] and s[1, :, 0].tolist() == [-1.0, 5.0, 6.0]
