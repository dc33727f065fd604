"""gdn_mla_bwd where a few keys take a query's weight: every gradient against 64 bits, on both sides of the lengths at
which the gradient of the queries changes its form."""
import math

import pytest
import torch

from tests.mla_testlib import TOL_MAX, TOL_NORM, attn_inputs, attn_ref, attn_run

pytestmark = pytest.mark.gpu


def slack(x, n, scale, dO, eta):
    """What a relative error of eta in every weight can do to each result, in size.

    The weights are exp(s - lse) with s and lse in 32 bits: their rounding is an absolute error of the exponent, so it
    grows with the scores, whatever the kernel.  A row's weights then add up to 1 + eta, and dP - delta is off by
    eta |delta| where it should cancel.  One sequence, causal, one key head."""
    q = torch.cat([x["qn"], x["qr"]], -1).double() if x["qr"] is not None else x["qn"].double()
    k = torch.cat([x["kn"][:, 0], x["kr"]], -1).double() if x["kr"] is not None else x["kn"][:, 0].double()
    v, dO = x["v"][:, 0].double(), dO.double()
    dn = x["qn"].shape[-1]
    out = {"qn": [], "qr": [], "kn": 0.0, "kr": 0.0, "v": 0.0, "o": []}
    for h in range(q.shape[1]):
        w = (q[:, h] @ k.T * scale).masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -math.inf).softmax(-1)
        delta = ((w @ v) * dO[:, h]).sum(-1).abs()
        dq, dk = scale * eta * delta[:, None] * (w @ k.abs()), scale * eta * (w.T @ (delta[:, None] * q[:, h].abs()))
        out["qn"].append(dq[:, :dn])
        out["qr"].append(dq[:, dn:])
        out["kn"], out["kr"] = out["kn"] + dk[:, :dn], out["kr"] + dk[:, dn:]
        out["v"] = out["v"] + eta * (w.T @ dO[:, h].abs())
        out["o"].append(eta * (w @ v.abs()))
    return {k: (torch.stack(t, 1) if isinstance(t, list) else t) for k, t in out.items()}


def near(got, ref, more, io, way, name):
    got = got.detach().double().cpu()
    d, more = (got - ref.detach()).abs(), more.reshape(ref.shape)
    assert torch.isfinite(got).all(), name
    top, norm = ref.abs().max().item(), ref.norm().item()
    assert d.norm().item() <= TOL_NORM[io, way] * norm + more.norm().item(), \
        f"{name}: norm {d.norm().item() / norm:.2e} > {TOL_NORM[io, way]:.1e} + {more.norm().item() / norm:.1e}"
    assert d.max().item() <= TOL_MAX[io, way] * top + more.max().item(), \
        f"{name}: max {d.max().item() / top:.2e} > {TOL_MAX[io, way]:.1e} + {more.max().item() / top:.1e}"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.3, 1.0, 3.0, 6.0])
@pytest.mark.parametrize("n", [40, 256, 257, 384, 640, 1100])
@pytest.mark.parametrize("dn,dr,dv", [(64, 0, 64), (64, 64, 128), (128, 64, 128)])
def test_gradients_of_sharp_scores(n, dn, dr, dv, scale, io):
    """Scores with a spread of 4 to 125.  Errors of the exponent: the scores' sum of up to 12 steps of 16 products, lse by
    four roundings and its way back by two more, each 2^-24 of the largest score: 2^-20 of it with all of them one way."""
    x, dO = attn_inputs(n + dn + dv, [n], [n], 2, 1, dn, dr, dv, io)
    ro, rl, rd = attn_ref(x, [n], [n], scale, True, dO)
    o, lse, d = attn_run(x, [n], [n], scale, True, io, dO)
    q = x["qn"].double().norm(dim=-1).max() if dr == 0 else torch.cat([x["qn"], x["qr"]], -1).double().norm(dim=-1).max()
    k = torch.cat([x["kn"][:, 0]] + ([x["kr"]] if dr else []), -1).double().norm(dim=-1).max()
    largest = min(scale * (q * k).item(), 2.0 * max(rl.abs().max().item(), 1.0))
    more = slack(x, n, scale, dO, 2.0 ** -20 * largest)
    near(o, ro, more["o"], io, "fwd", "o")
    for name in rd:
        near(d[name], rd[name], more[name], io, "bwd", f"d{name}")
