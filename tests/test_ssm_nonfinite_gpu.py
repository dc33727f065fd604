"""NaN, infinities and sums past fp32 in the scan: they reach what the definition makes of them, and nothing beside it."""
import math

import pytest
import torch

from tests.ssm_testlib import WORK, cuda, nan, offsets, scan_grads, scan_inputs, scan_run

pytestmark = pytest.mark.gpu


def same(got, ref, what, name):
    """Finite exactly where the definition in 64 bits is, and there within the bounds of `close`."""
    step = torch.finfo(got.dtype).eps / 2
    got, ref = got.detach().double().cpu(), ref.detach().double()
    ok = ref.isfinite()
    assert torch.equal(got.isfinite(), ok), f"{name}: {(got.isfinite() != ok).sum().item()} of {ok.numel()} values differ in being finite"
    if ok.any():
        got, ref = got[ok], ref[ok]
        assert (got - ref).abs().sub(step * ref.abs()).max() <= WORK[what] * ref.abs().max(), name


def check(i, lens, io):
    y, hT, grads = scan_grads(i, lens)
    got = scan_run(cuda(i), lens, io, cu=offsets(lens).cuda(), train=True)
    same(got["y"], y, "scan", "y")
    same(got["hT"], hT, "scan", "hT")
    for k, d in grads.items():
        same(got["d" + k], d, "scan_bwd", "d" + k)


POISON = [("x", math.nan), ("x", math.inf), ("dt", math.nan), ("z", math.nan), ("Bm", math.nan), ("Cm", math.nan), ("dy", math.nan),
          ("dy", -math.inf)]


@pytest.mark.parametrize("key,value", POISON)
@pytest.mark.parametrize("io,D,N,G", [("f32", 24, 16, 1), ("bf16", 96, 16, 2), ("f32", 40, 8, 1), ("bf16", 24, 24, 1), ("f32", 16, 64, 1)])
def test_one_token(io, D, N, G, key, value):
    """One value at one token in the middle of a sequence: of dBm and dCm too only the tokens that depend on it."""
    lens = [13, 40, 9]
    i = scan_inputs(D + N, lens, D, N, G, io)
    i[key].select(0, 13 + 21)[(0, 5) if i[key].ndim == 3 else 5] = value
    check(i, lens, io)


@pytest.mark.parametrize("key", ["x", "dy"])
def test_one_token_of_split_calls(key):
    """The same where segments of time run side by side."""
    lens = [600, 433]
    i = scan_inputs(2, lens, 16, 16, 1, "f32")
    i[key][333, 5] = math.nan
    check(i, lens, "f32")


def test_products_past_fp32():
    """A state times a gradient that passes fp32 at one token: an infinite row of dCm there, the others as they are."""
    n, at = 30, 19
    i = scan_inputs(6, [n], 24, 16, 1, "f32", gate=False)
    i["x"][at, 3], i["dy"][at, 3] = 1e30, 1e20
    _, _, grads = scan_grads(i, [n])
    assert (grads["Cm"][at].abs().max() > 3.5e38) and grads["Cm"][at - 1].abs().max() < 1e8
    got = scan_run(cuda(i), [n], "f32", cu=offsets([n]).cuda(), train=True)["dCm"].double().cpu()
    for t in range(n):
        ref = grads["Cm"][t]
        if t == at:
            big = ref.abs() > 3.5e38
            assert got[t][big].isinf().all() and (got[t][big].sign() == ref[big].sign()).all()
        else:
            assert (got[t] - ref).abs().max() <= WORK["scan_bwd"] * ref.abs().max(), t


@pytest.mark.parametrize("which", ["skip", "bias"])
def test_sums_over_tokens_past_fp32(which):
    """dD or d dt_bias past fp32 after some of its tokens is infinite, not a NaN.  Every term has one sign: rates of 2e-9 over 200
    tokens change a state by less than 1e-6 of it, so d delta[t] = 8 (200 - t) g (C B) x to that."""
    n, D, N = 200, 16, 8
    i = scan_inputs(1, [n], D, N, 1, "f32", gate=False, softplus=False, h0=False)
    i["x"], i["dt"], i["bias"], i["A_log"] = torch.ones(n, D), torch.full((n, D), 0.01), torch.zeros(D), torch.full((D, N), -20.0)
    i["dhT"] = torch.zeros(1, D, N)
    i["Bm"], i["Cm"] = torch.ones(n, 1, N), torch.full((n, 1, N), 1e-10 if which == "skip" else 1.0)
    i["dy"] = torch.full((n, D), 3e37 if which == "skip" else 1e34)      # sums 6e39; 8 x 1e34 x 20100 = 1.6e39
    got = scan_run(cuda(i), [n], "f32", softplus=False, cu=offsets([n]).cuda(), train=True)
    assert got["d" + which].isposinf().all()
    for k in ("x", "dt", "Bm", "skip" if which == "bias" else "bias"):
        assert got["d" + k].isfinite().all(), k


@pytest.mark.parametrize("io,N", [("f32", 16), ("bf16", 8), ("f32", 40), ("bf16", 64)])
@pytest.mark.parametrize("lens", [[13, 1, 40], [333]])
def test_rates_past_fp32(io, N, lens):
    """exp(A_log) past fp32 forgets at once, as in 64 bits, whatever a length leaves of the last tile: no NaN."""
    i = scan_inputs(N, lens, 24, N, 1, io)
    i["A_log"][::2] = 95.0
    i["A_log"][1, ::3] = 88.9
    check(i, lens, io)


def test_rates_past_fp32_of_new_tokens():
    import linear_attention_recurrence_delta_gb300 as gdn
    from tests.ssm_testlib import ORDER, scan_all
    B, T, D, N = 3, 2, 24, 16
    i = scan_inputs(4, [T] * B, D, N, 1, "f32", softplus=False)
    i["A_log"][::2] = 95.0
    i["dt"][0], i["bias"] = 0.0, torch.zeros(D)      # a step of size zero changes nothing, whatever the rate
    dev, y = cuda(i), nan((B * T, D), torch.float32)
    state = dev["h0"].clone()
    gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(B, T, D, N, B, 1, "f32", softplus=False), *[dev[k] for k in ORDER], state, None, None, y))
    ref, h = scan_all({k: t.double() for k, t in i.items()}, [T] * B, softplus=False)
    same(y, ref, "scan", "y")
    same(state, h, "scan", "state")
