"""The state-space calls that a user's program may make and the other tests do not: captured and replayed, on two streams at
once, from many sequences, from shared slots, over offsets that pass 32 bits, with offsets out of order, with tensors elsewhere."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import (ORDER, close, conv_all, cuda, gen, nan, normal, offsets, scan_all, scan_inputs, scan_one, scan_run,
                               tdtype)

pytestmark = pytest.mark.gpu


def layer_calls(seed, lens, D, N, slots):
    """One of every call on fixed buffers: a function that makes them, the inputs and the outputs."""
    rows, B, dim = sum(lens), len(lens), 512
    g = gen(seed)
    i = cuda(scan_inputs(seed, lens, D, N, 1, "bf16"))
    n = {"x": normal(g, (rows, dim), "bf16").cuda(), "res": normal(g, (rows, dim), "bf16").cuda(), "dy": normal(g, (rows, dim), "bf16").cuda()}
    w, taps = torch.rand(dim, generator=g).cuda() + 0.5, torch.randn((D, 4), generator=g).cuda()
    cu = offsets(lens).cuda()
    slot = torch.randperm(slots, generator=g)[:B].int().cuda()
    conv_pool, scan_pool = normal(g, (slots, 3, D), "bf16").cuda(), torch.randn((slots, D, N), generator=g).cuda()
    s = (gdn.make_norm(rows, dim), gdn.make_norm(rows, dim, out="e4m3", group=128), gdn.make_conv(B, max(lens), D, 4, rows=rows),
         gdn.make_conv_step(B, 1, D, 4, slots), gdn.make_scan_step(B, 1, D, N, slots))
    ws = [torch.empty(k, dtype=torch.uint8, device="cuda") for k in (gdn.gdn_norm_workspace_bytes(s[0]), gdn.gdn_conv_workspace_bytes(s[2]))]
    b16 = lambda *q: nan(q, torch.bfloat16)  # noqa: E731
    out = {"y": b16(rows, dim), "sum": b16(rows, dim), "scale": nan((rows, dim // 128), torch.float32), "dx": b16(rows, dim),
           "dw": nan((dim,), torch.float32), "u": b16(rows, D), "sT": b16(B, 3, D), "du": b16(rows, D), "dtaps": nan((D, 4), torch.float32),
           "q": torch.empty((rows, dim), dtype=torch.float8_e4m3fn, device="cuda"), "cy": b16(B, D), "sy": b16(B, D),
           "conv_pool": conv_pool, "scan_pool": scan_pool}

    def call():
        gdn.check(gdn.gdn_norm_fwd(s[0], n["x"], n["res"], w, out["y"], None, out["sum"]))
        gdn.check(gdn.gdn_norm_fwd(s[1], n["x"], n["res"], w, out["q"], out["scale"], None))
        gdn.check(gdn.gdn_norm_bwd(s[0], out["sum"], w, n["dy"], None, out["dx"], None, out["dw"], ws[0]))
        gdn.check(gdn.gdn_conv_fwd(s[2], i["x"], taps, None, cu, None, out["u"], out["sT"]))
        gdn.check(gdn.gdn_conv_bwd(s[2], i["x"], taps, None, cu, None, i["dy"], None, out["du"], out["dtaps"], None, None, ws[1]))
        gdn.check(gdn.gdn_conv_step(s[3], i["x"][:B], taps, None, conv_pool, slot, None, out["cy"]))
        gdn.check(gdn.gdn_scan_step(s[4], *[i[k][:B] if k in ORDER[:5] else i[k] for k in ORDER], scan_pool, slot, None, out["sy"]))
        out.update({"scan " + k: t for k, t in scan_run(i, lens, "bf16", cu=cu, train=True).items()})
    return call, {"res": n["res"], "nx": n["x"], "ndy": n["dy"], "x": i["x"], "dt": i["dt"], "dy": i["dy"], "conv_pool": conv_pool,
                  "scan_pool": scan_pool}, out


def bits(t):
    return t.contiguous().view(torch.uint8).clone()


def test_captured_and_replayed():
    """A captured pass through all calls gives, for new inputs in the same buffers, the bits of the eager pass."""
    call, ins, out = layer_calls(1, [90, 1, 200], 96, 16, 7)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    held = dict(out)
    for seed in (5, 6):
        g = gen(seed)
        fresh = {k: (0.5 * torch.randn(t.shape, generator=g)).to(t.dtype) for k, t in ins.items()}

        def fill():
            for k, t in ins.items():
                t.copy_(fresh[k])
        fill()
        graph.replay()
        got = {k: bits(t) for k, t in held.items()}
        fill()
        call()
        for k, t in out.items():
            assert torch.equal(got[k], bits(t)), k


def test_two_streams_at_once():
    """Passes over two sets of buffers, enqueued on two streams without a wait between, give the bits of passes alone."""
    sets = [layer_calls(s, [400, 33, 250], 96, 16, 7) for s in (1, 2)]
    alone = []
    for call, ins, out in sets:
        first = {k: t.clone() for k, t in ins.items()}
        call()
        alone.append({k: bits(t) for k, t in out.items()})
        for k, t in ins.items():
            t.copy_(first[k])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for (call, ins, out), st in zip(sets, streams):
            with torch.cuda.stream(st):
                pools = {k: ins[k].clone() for k in ("conv_pool", "scan_pool")}
                call()
                for k, t in pools.items():
                    out[k + " after"] = out[k].clone()
                    ins[k].copy_(t)
    torch.cuda.synchronize()
    for (call, ins, out), want in zip(sets, alone):
        for k, v in want.items():
            assert torch.equal(v, bits(out.get(k + " after", out[k]))), k


def test_many_short_sequences():
    """As many sequences as a call takes, most of one row, some empty."""
    B, D, N = 65535, 8, 8
    g = gen(3)
    lens = torch.randint(0, 3, (B,), generator=g).tolist()
    i = scan_inputs(2, [2], D, N, 1, "f32")
    rows = sum(lens)
    for k in ("x", "dt", "z", "dy"):
        i[k] = normal(g, (rows, D), "f32", 0.5)
    for k in ("Bm", "Cm"):
        i[k] = normal(g, (rows, 1, N), "f32")
    i["h0"], i["dhT"] = torch.randn((B, D, N), generator=g), torch.randn((B, D, N), generator=g)
    cu = offsets(lens) if B < 100 else torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(lens).cumsum(0)]).int()
    got = scan_run(cuda(i), lens, "f32", cu=cu.cuda(), T=2, train=True)
    taps = torch.randn((D, 4), generator=g)
    s0 = normal(g, (B, 3, D), "f32")
    u, sT = nan((rows, D), torch.float32), nan(s0.shape, torch.float32)
    gdn.check(gdn.gdn_conv_fwd(gdn.make_conv(B, 2, D, 4, "f32", rows=rows), i["x"].cuda(), taps.cuda(), None, cu.cuda(), s0.cuda(), u, sT))
    assert torch.isfinite(u).all()
    for b in list(range(5)) + [30000, B - 2, B - 1]:
        at, n = int(cu[b]), lens[b]
        part = [i[k][at: at + n].double() for k in ORDER[:5]]
        y, h = scan_one(*part, i["A_log"].double(), i["skip"].double(), i["bias"].double(), i["h0"][b].double(), True)
        close(got["hT"][b], h, "scan", f"hT {b}")
        v, state = conv_all(i["x"][at: at + n].double(), taps.double(), None, s0[b: b + 1].double(), [n], True)
        close(sT[b], state[0], "sum", f"sT {b}")
        if n:
            close(got["y"][at: at + n], y, "scan", f"y {b}")
            close(u[at: at + n], v, "sum", f"u {b}")
    assert all(torch.isfinite(t).all() for t in got.values() if t is not None)


def test_one_state_for_several_sequences():
    """Sequences that go on from one common prompt read one slot and write their own."""
    D, N, B, slots = 32, 16, 4, 9
    i = scan_inputs(4, [1] * B, D, N, 1, "f32")
    dev, g = cuda(i), gen(8)
    pool, conv = torch.randn((slots, D, N), generator=g), normal(g, (slots, 3, D), "f32")
    src, dst = torch.full((B,), 5, dtype=torch.int32), torch.tensor([0, 8, 2, 3], dtype=torch.int32)
    y, state = nan((B, D), torch.float32), pool.cuda()
    gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(B, 1, D, N, slots, 1, "f32"), *[dev[k] for k in ORDER], state, src.cuda(), dst.cuda(), y))
    ref, h = scan_all({**{k: t.double() for k, t in i.items()}, "h0": pool[5].double().expand(B, D, N)}, [1] * B)
    close(y, ref, "scan", "y")
    close(state[dst.long().cuda()], h, "scan", "state")
    assert torch.equal(state.cpu()[[1, 4, 5, 6, 7]], pool[[1, 4, 5, 6, 7]])
    taps, u, cs = torch.randn((D, 4), generator=g), nan((B, D), torch.float32), conv.cuda()
    gdn.check(gdn.gdn_conv_step(gdn.make_conv_step(B, 1, D, 4, slots, "f32"), dev["x"], taps.cuda(), None, cs, src.cuda(), dst.cuda(), u))
    ref, after = conv_all(i["x"].double(), taps.double(), None, conv[5].double().expand(B, 3, D), [1] * B, True)
    close(u, ref, "sum", "u")
    assert torch.equal(cs.cpu()[dst.long()].double(), after)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_drafted_tokens_are_single_tokens(io):
    """Eight tokens in one call give the bits of eight calls."""
    D, N, B = 40, 24, 3
    i = cuda(scan_inputs(5, [8] * B, D, N, 1, io))
    pool, dt = torch.randn((B, D, N), generator=gen(1)).cuda(), tdtype(io)
    y, state = nan((B * 8, D), dt), pool.clone()
    gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(B, 8, D, N, B, 1, io), *[i[k] for k in ORDER], state, None, None, y))
    one, rows = pool.clone(), torch.arange(B, device="cuda") * 8
    for t in range(8):
        o = nan((B, D), dt)
        part = [i[k][rows + t] if k in ORDER[:5] else i[k] for k in ORDER]
        gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(B, 1, D, N, B, 1, io), *part, one, None, None, o))
        assert torch.equal(o, y[rows + t])
    assert torch.equal(one, state)


def test_a_step_of_size_zero_changes_nothing():
    """Without softplus a step size may be zero: the state keeps its bits, whatever the rates."""
    D, N, T = 16, 16, 40
    i = scan_inputs(7, [T], D, N, 1, "f32", bias=False)
    i["dt"] = torch.zeros(T, D)
    got = scan_run(cuda(i), [T], "f32", softplus=False)
    assert torch.equal(got["hT"].cpu(), i["h0"])


def test_cut_and_bad_offsets():
    """Sequences over T rows are cut there; offsets outside the tensor count as its bounds, descending ones as nothing."""
    D, N, rows = 24, 16, 60
    i = scan_inputs(9, [rows], D, N, 1, "f32")
    i["h0"], i["dhT"] = (torch.randn((4, D, N), generator=gen(k)) for k in (1, 2))
    cu = torch.tensor([-5, 18, 50, 40, 99], dtype=torch.int32)
    got = scan_run(cuda(i), [0] * 4, "f32", cu=cu.cuda(), T=17, train=True)
    seen = torch.zeros(rows, dtype=torch.bool)
    for b, (at, n) in enumerate(((0, 17), (18, 17), (50, 0), (40, 17))):
        part = [i[k][at: at + n].double() for k in ORDER[:5]]
        y, h = scan_one(*part, i["A_log"].double(), i["skip"].double(), i["bias"].double(), i["h0"][b].double(), True)
        close(got["y"].cpu()[at: at + n], y, "scan", f"y {b}")
        close(got["hT"][b], h, "scan", f"hT {b}")
        seen[at: at + n] = True
    for k in ("y", "dx", "ddt", "dz", "dBm", "dCm"):
        assert got[k].cpu()[~seen].isnan().all() and torch.isfinite(got[k].cpu()[seen]).all(), k
    assert all(torch.isfinite(got[k]).all() for k in ("dA_log", "dskip", "dbias", "dh0"))


def test_rows_beyond_32_bits():
    """Rows so far apart that their offsets pass 2^31 elements, for every tensor that the kernels address by rows."""
    n, D, N, far = 36, 16, 16, 1 << 26
    i = scan_inputs(3, [n], D, N, 1, "bf16")
    dev = cuda(i)
    for k in ("x", "dt", "Bm"):
        t = i[k]
        wide = torch.empty(n * far, dtype=t.dtype, device="cuda").as_strided(t.shape, (far,) + t.contiguous().stride()[1:])
        dev[k] = wide.copy_(t)
    got, want = scan_run(dev, [n], "bf16", train=True), scan_run(cuda(i), [n], "bf16", train=True)
    for k in want:
        assert torch.equal(bits(got[k]), bits(want[k])), k
    taps = torch.randn((D, 4), generator=gen(1)).cuda()
    u, v = nan((n, D), torch.bfloat16), nan((n, D), torch.bfloat16)
    c = gdn.make_conv(1, n, D, 4)
    gdn.check(gdn.gdn_conv_fwd(c, dev["x"], taps, None, None, None, u, None))
    gdn.check(gdn.gdn_conv_fwd(c, i["x"].cuda(), taps, None, None, None, v, None))
    assert torch.equal(u, v)


def test_tensors_elsewhere_are_refused():
    """A tensor in host memory raises before anything is enqueued."""
    n, x = gdn.make_norm(4, 64), torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w, y = torch.ones(64, device="cuda"), torch.full((4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_norm_fwd(n, x.cpu(), None, w, y, None, None)
    with pytest.raises(ValueError):
        gdn.gdn_norm_fwd(n, x, None, w.cpu(), y, None, None)
    with pytest.raises(ValueError):
        gdn.gdn_conv_fwd(gdn.make_conv(1, 4, 64, 2), x, torch.ones(64, 2), None, None, None, y, None)
    torch.cuda.synchronize()
    assert (y == 3).all()


def test_a_nan_reaches_its_own_channel_only():
    """In one sequence a NaN in x at token t leaves earlier tokens and, for outputs and their gradients, other channels alone."""
    n, D, N = 40, 24, 16
    i = scan_inputs(12, [n], D, N, 1, "f32", h0=False)
    i["x"][20, 5] = math.nan
    got = scan_run(cuda(i), [n], "f32")
    y, other = got["y"].cpu(), [c for c in range(D) if c != 5]
    assert torch.isfinite(y[:, other]).all() and torch.isfinite(y[:20]).all() and y[20:, 5].isnan().all()
    assert torch.isfinite(got["hT"].cpu()[:, other]).all() and got["hT"].cpu()[:, 5].isnan().all()
