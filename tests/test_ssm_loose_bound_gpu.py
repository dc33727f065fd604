"""T is only a bound: one that nobody knows (the largest int) gives the bits of T = rows."""
import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import cuda, gen, nan, normal, offsets, scan_inputs, scan_run, tdtype

pytestmark = pytest.mark.gpu

LENS, MOST = [70, 0, 300, 1, 131], 2**31 - 1


def same(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_convolution(io):
    D, W, rows, B, g = 72, 4, sum(LENS), len(LENS), gen(1)
    x, dy, s0, dsT = (normal(g, s, io).cuda() for s in ((rows, D), (rows, D), (B, W - 1, D), (B, W - 1, D)))
    w, bias, cu = torch.randn((D, W), generator=g).cuda(), torch.randn(D, generator=g).cuda(), offsets(LENS).cuda()

    def run(T):
        s, dt = gdn.make_conv(B, T, D, W, io, rows=rows), tdtype(io)
        ws = torch.empty(gdn.gdn_conv_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        out = {"y": nan((rows, D), dt), "sT": nan(s0.shape, dt), "dx": nan((rows, D), dt), "dw": nan((D, W), torch.float32),
               "dbias": nan((D,), torch.float32), "ds0": nan(s0.shape, dt)}
        gdn.check(gdn.gdn_conv_fwd(s, x, w, bias, cu, s0, out["y"], out["sT"]))
        gdn.check(gdn.gdn_conv_bwd(s, x, w, bias, cu, s0, dy, dsT, out["dx"], out["dw"], out["dbias"], out["ds0"], ws))
        return out
    same(run(rows), run(MOST))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_scan(io):
    i, cu = cuda(scan_inputs(2, LENS, 40, 16, 1, io)), offsets(LENS).cuda()
    same(*(scan_run(i, LENS, io, cu=cu, T=T, train=True) for T in (sum(LENS), MOST)))
