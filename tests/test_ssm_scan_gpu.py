"""gdn_scan_fwd, gdn_scan_bwd and gdn_scan_step against 64 bits: states, groups, lengths from zero on, splits, slots."""
import math

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn
from tests.ssm_testlib import ORDER, close, cuda, gen, nan, normal, offsets, scan_all, scan_grads, scan_inputs, scan_one, scan_run, tdtype

pytestmark = pytest.mark.gpu


def compare(i, lens, io, gap=0, pad=0, softplus=True, dhT=True, cu=True, T=None):
    y, hT, grads = scan_grads(i, lens, softplus, gap, dhT)
    own = torch.zeros(i["x"].shape[0], dtype=torch.bool)
    own[gap: gap + sum(lens)] = True
    dev = cuda(i)
    got = scan_run(dev, lens, io, softplus, offsets(lens, gap).cuda() if cu else None, T, True, dhT)
    close(got["y"], y, "scan", "y", own)
    close(got["hT"], hT, "scan", "hT")
    assert got["y"].cpu()[~own].isnan().all()
    for k in ("x", "dt", "z", "Bm", "Cm"):
        if i[k] is not None:
            close(got["d" + k], grads[k], "scan_bwd", "d" + k, own)
            assert got["d" + k].cpu()[~own].isnan().all()
    for k in ("A_log", "skip", "bias", "h0"):
        if i[k] is not None:
            close(got["d" + k], grads[k], "scan_bwd", "d" + k)
    return dev, got


SMALL = [([1], 8, 8, 1), ([2, 0, 17], 24, 16, 1), ([16, 15, 33], 40, 24, 1), ([5, 31], 64, 32, 2), ([40, 1], 24, 64, 3),
         ([32, 64, 50], 136, 16, 1), ([0, 0], 8, 8, 1), ([19], 80, 8, 1), ([48], 32, 56, 2)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D,N,G", SMALL)
def test_sequences_and_gradients(io, lens, D, N, G):
    i = scan_inputs(D + N, lens, D, N, G, io, gap=3, pad=2)
    compare(i, lens, io, 3, 2, T=max(max(lens), 1))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,D,N,G", [([1000], 16, 16, 1), ([700, 3, 0, 431], 24, 8, 1), ([513], 16, 40, 2)])
def test_split_in_time(io, lens, D, N, G):
    """Few channels over many tokens: segments run side by side, with and without states at the ends."""
    rows = sum(lens)
    s = gdn.make_scan(len(lens), max(lens), D, N, G, io, rows=rows)
    assert gdn.gdn_scan_workspace_bytes(s, 0) > 256          # the segments' states: the call is split
    compare(scan_inputs(rows, lens, D, N, G, io), lens, io)
    compare(scan_inputs(rows + 1, lens, D, N, G, io, h0=False), lens, io, dhT=False)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate,skip,bias,softplus,h0,dhT", [(False, True, True, True, True, True), (True, False, True, True, False, True),
                                                            (True, True, False, True, True, False), (True, True, True, False, True, True),
                                                            (False, False, False, False, False, False)])
def test_parts_left_out(io, gate, skip, bias, softplus, h0, dhT):
    lens = [37, 20]
    compare(scan_inputs(3, lens, 48, 16, 2, io, gate, skip, bias, softplus, h0), lens, io, softplus=softplus, dhT=dhT)


def test_equal_sequences_without_offsets():
    lens = [45, 45, 45]
    compare(scan_inputs(9, lens, 56, 16, 1, "bf16"), lens, "bf16", cu=False)


def test_gradients_against_differences():
    """The gradients along random directions against central differences of the definition in 64 bits: with steps of 1e-5
    the differences are good to about 1e-9, the gradients to the f32 bound above."""
    lens = [30, 13]
    i = scan_inputs(11, lens, 24, 16, 1, "f32")
    got = scan_run(cuda(i), lens, "f32", cu=offsets(lens).cuda(), train=True)
    x = {k: t.double() for k, t in i.items()}

    def loss(v):
        y, hT = scan_all(v, lens)
        return ((y * x["dy"]).sum() + (hT * x["dhT"]).sum()).item()

    g = gen(5)
    for k in ORDER + ("h0",):
        v = torch.randn(x[k].shape, generator=g, dtype=torch.float64)
        d = (loss({**x, k: x[k] + 1e-5 * v}) - loss({**x, k: x[k] - 1e-5 * v})) / 2e-5
        mine = got["d" + k].double().cpu()
        assert abs((mine * v).sum().item() - d) <= 9e-5 * mine.abs().max().item() * v.abs().sum().item() ** 0.5 * 10 + 1e-6, k


def test_same_bits_and_graphs():
    """Calls repeat bit for bit, on another stream and from a captured graph whose inputs change between replays."""
    lens = [300, 77, 512]
    i = cuda(scan_inputs(2, lens, 72, 16, 1, "bf16"))
    cu = offsets(lens).cuda()
    first = scan_run(i, lens, "bf16", cu=cu, train=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = scan_run(i, lens, "bf16", cu=cu, train=True)
    torch.cuda.current_stream().wait_stream(side)
    for k in first:
        assert torch.equal(first[k].view(torch.uint8), second[k].view(torch.uint8)), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = scan_run(i, lens, "bf16", cu=cu, train=True)
    other = cuda(scan_inputs(4, lens, 72, 16, 1, "bf16"))
    for src in (i, other):
        fresh = {k: t.clone() for k, t in src.items()}
        for k, t in i.items():
            t.copy_(fresh[k])
        graph.replay()
        want = scan_run(i, lens, "bf16", cu=cu, train=True)
        for k in held:
            assert torch.equal(held[k].view(torch.uint8), want[k].view(torch.uint8)), k


def test_nothing_crosses_sequences():
    lens = [50, 20, 33]
    i = scan_inputs(6, lens, 32, 16, 1, "bf16")
    for k in ("x", "dt", "z", "Bm", "Cm", "dy"):
        i[k][50:70] = math.nan
    i["h0"][1] = math.inf
    got = scan_run(cuda(i), lens, "bf16", cu=offsets(lens).cuda(), train=True)
    keep = torch.ones(103, dtype=torch.bool)
    keep[50:70] = False
    for k in ("y", "dx", "ddt", "dz", "dBm", "dCm"):
        assert torch.isfinite(got[k].cpu()[keep]).all(), k
    for k in ("hT", "dh0"):
        assert torch.isfinite(got[k][[0, 2]]).all(), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_extreme_step_sizes(io):
    """Steps so large that nothing is left of a state, and so small that nothing of a token gets in."""
    lens = [70]
    i = scan_inputs(8, lens, 16, 16, 1, io)
    i["dt"][10:20], i["dt"][40:50] = 60.0, -80.0
    i["bias"].zero_()
    compare(i, lens, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,N,G,parts", [(1, 1, 8, 8, 1, True), (24, 1, 2048, 16, 1, True), (5, 8, 48, 24, 2, True), (3, 2, 40, 64, 1, False),
                                             (9, 3, 96, 40, 3, True)])
def test_new_tokens(io, B, T, D, N, G, parts):
    """States by slot: in place, from one slot to another, from none (zeros), to none (a place without a request)."""
    i = scan_inputs(B + D, [T] * B, D, N, G, io, gate=parts, skip=parts, bias=parts)
    g, slots = gen(B), 2 * B + 3
    pool, order = 0.5 * torch.randn((slots, D, N), generator=g), torch.randperm(slots, generator=g).int()
    src, dst = order[:B].clone(), order[B: 2 * B].clone()
    s = gdn.make_scan_step(B, T, D, N, slots, G, io)
    dev, x = cuda(i), {k: None if t is None else t.double() for k, t in i.items()}

    def check(src, dst):
        y, state = nan((B * T, D), tdtype(io)), pool.cuda()
        gdn.check(gdn.gdn_scan_step(s, *[dev[k] for k in ORDER], state, None if src is None else src.cuda(),
                                    None if dst is None else dst.cuda(), y))
        a = list(range(B)) if src is None else src.tolist()
        to = a if dst is None else dst.tolist()
        want, kept = pool.double(), torch.ones(slots, dtype=torch.bool)
        for q in range(B):
            before = pool[a[q]].double() if 0 <= a[q] < slots else torch.zeros(D, N, dtype=torch.float64)
            part = [None if x[k] is None else x[k][q * T: (q + 1) * T] for k in ORDER[:5]]
            ref, after = scan_one(*part, x["A_log"], x["skip"], x["bias"], before, True)
            close(y[q * T: (q + 1) * T], ref, "scan", f"y of {q}")
            if 0 <= to[q] < slots:
                want[to[q]], kept[to[q]] = after, False
        close(state, want, "scan", "state")
        assert torch.equal(state.cpu()[kept], pool[kept])

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
    D, N, n, more = 64, 16, 300, 9
    i = scan_inputs(1, [n + more], D, N, 1, "f32", h0=False)
    dev = cuda(i)
    whole = scan_run(dev, [n + more], "f32")
    front = {k: t if t is None or k in ("A_log", "skip", "bias") else t[:n] for k, t in dev.items()}
    got = scan_run(front, [n], "f32")
    rows, state = [got["y"]], got["hT"]
    for t, T in ((n, 1), (n + 1, 3), (n + 4, 5)):
        part = [dev[k][t: t + T] if k in ORDER[:5] else dev[k] for k in ORDER]
        y = nan((T, D), torch.float32)
        gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(1, T, D, N, 1, 1, "f32"), *part, state, None, None, y))
        rows.append(y)
    close(torch.cat(rows), whole["y"].cpu(), "scan", "y")
    close(state, whole["hT"].cpu(), "scan", "hT")


def test_slots_beyond_32_bits():
    """A pool whose slots' offsets pass 2^31 values."""
    D, N, slots = 2048, 16, 70000
    i = scan_inputs(1, [1, 1], D, N, 1, "bf16")
    state = torch.empty((slots, D, N), device="cuda")
    slot = torch.tensor([69999, 5], dtype=torch.int32)
    for q in range(2):
        state[int(slot[q])] = i["h0"][q].cuda()
    y, dev = nan((2, D), torch.bfloat16), cuda(i)
    gdn.check(gdn.gdn_scan_step(gdn.make_scan_step(2, 1, D, N, slots), *[dev[k] for k in ORDER], state, slot.cuda(), None, y))
    ref, hT = scan_all({k: t.double() for k, t in i.items()}, [1, 1])
    close(y, ref, "scan", "y")
    close(state[slot.long().cuda()], hT, "scan", "state")
