"""Every tensor that the state-space kernels address by rows, with rows so far apart that their offsets pass 2^31 elements: the
same bits as from rows side by side.  Tensors are spread four at a time (5 GB each)."""
import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import ORDER, cuda, gen, nan, normal, scan_inputs

pytestmark = pytest.mark.gpu

ROWS, D, N, FAR = 36, 16, 16, 1 << 26
BF16, F32 = torch.bfloat16, torch.float32


def spread(t):
    wide = torch.empty(ROWS * FAR, dtype=t.dtype, device="cuda").as_strided(t.shape, (FAR,) + t.contiguous().stride()[1:])
    return wide.copy_(t)


def check(call, ins, outs, others):
    """call(tensors) with the names of `ins` and `outs` (rows) and `others` (no rows) filled in."""
    def run(names):
        t = {k: (spread(v) if k in names else v.clone()) for k, v in {**ins, **outs, **others}.items()}
        call(t)
        return {k: t[k].contiguous().view(torch.uint8) for k in (*outs, *others)}
    want, names = run(()), [*ins, *outs]
    for at in range(0, len(names), 4):
        got = run(names[at: at + 4])
        for k in want:
            assert torch.equal(got[k], want[k]), (k, names[at: at + 4])


def test_norm():
    g = gen(1)
    ins = {k: normal(g, (ROWS, D), "bf16").cuda() for k in ("x", "res", "dy", "dsum")}
    outs = {k: nan((ROWS, D), BF16) for k in ("y", "sum", "dx", "dres")}
    w, s = torch.rand(D, generator=g).cuda() + 0.5, gdn.make_norm(ROWS, D)
    ws = torch.empty(gdn.gdn_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")

    def call(t):
        gdn.check(gdn.gdn_norm_fwd(s, t["x"], t["res"], w, t["y"], None, t["sum"]))
        gdn.check(gdn.gdn_norm_bwd(s, t["sum"], w, t["dy"], t["dsum"], t["dx"], t["dres"], t["dw"], ws))
    check(call, ins, outs, {"dw": nan((D,), F32)})


def test_convolution():
    g = gen(2)
    ins = {k: normal(g, (ROWS, D), "bf16").cuda() for k in ("x", "dy")}
    outs = {k: nan((ROWS, D), BF16) for k in ("y", "dx", "ystep")}
    taps, s, one = torch.randn((D, 4), generator=g).cuda(), gdn.make_conv(1, ROWS, D, 4), gdn.make_conv_step(ROWS, 1, D, 4, ROWS)
    ws = torch.empty(gdn.gdn_conv_workspace_bytes(s), dtype=torch.uint8, device="cuda")

    def call(t):
        gdn.check(gdn.gdn_conv_fwd(s, t["x"], taps, None, None, None, t["y"], None))
        gdn.check(gdn.gdn_conv_bwd(s, t["x"], taps, None, None, None, t["dy"], None, t["dx"], t["dw"], None, None, ws))
        gdn.check(gdn.gdn_conv_step(one, t["x"], taps, None, t["state"], None, None, t["ystep"]))
    check(call, ins, outs, {"dw": nan((D, 4), F32), "state": normal(g, (ROWS, 3, D), "bf16").cuda()})


@pytest.mark.parametrize("gate", [True, False])
def test_scan(gate):
    i = cuda(scan_inputs(3, [ROWS], D, N, 1, "bf16", gate=gate))
    ins = {k: i[k] for k in ("x", "dt", "z", "Bm", "Cm", "dy") if i[k] is not None}
    outs = {"d" + k: torch.full_like(i[k], float("nan")) for k in ORDER[:5] if i[k] is not None}
    outs.update(y=nan((ROWS, D), BF16), ystep=nan((ROWS, D), BF16))
    others = {"d" + k: nan(i[k].shape, F32) for k in ("A_log", "skip", "bias")}
    others["state"] = torch.randn((ROWS, D, N), generator=gen(4)).cuda()
    s, one = gdn.make_scan(1, ROWS, D, N), gdn.make_scan_step(ROWS, 1, D, N, ROWS)
    ws, saved = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (gdn.gdn_scan_workspace_bytes(s, 1), gdn.gdn_scan_saved_bytes(s)))

    def call(t):
        args = [t.get(k) for k in ORDER[:5]] + [i["A_log"], i["skip"], i["bias"]]
        gdn.check(gdn.gdn_scan_fwd(s, *args, None, i["h0"], t["y"], None, saved, ws))
        gdn.check(gdn.gdn_scan_bwd(s, *args, None, saved, t["dy"], None, *[t.get("d" + k) for k in ORDER], None, ws))
        gdn.check(gdn.gdn_scan_step(one, *args, t["state"], None, None, t["ystep"]))
    check(call, ins, outs, others)
