"""The bounded waits of the tensor-core latent-attention kernels, run out without faulting the GPU.

The library's test hook GDN_TEST_STARVE_CHUNK=k (read once per process, so each case is a child process) announces a
kernel's k-th tile to its barrier but never loads it.  The wait for it expires, every role of the CTA runs through, the
call's status reads GDN_ERR_TIMEOUT, and the same context then runs a call that has no k-th tile to parity.
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

GDN_ERR_TIMEOUT = 7

_CHILD = r"""
import json, math, sys, time
import torch
import linear_attention_recurrence_delta_gb300 as gdn
from tests.mla_testlib import attn_inputs, attn_ref, attn_run, close, decode_ref
from tests.test_mla_decode_gpu import call, setup
what = sys.argv[1]
t0 = time.perf_counter()
try:
    if what == "decode":
        n, T, H = [3000] * 8, 1, 16
    elif what == "decode pairs":
        n, T, H = [3000] * 8, 2, 40
    elif what == "decode two groups":
        n, T, H = [3000] * 8, 4, 40
    if what.startswith("decode"):
        a = (T, H, 64, 32, 64, "bf16")
        table, pages, cache, rows, qc, qr = setup(1, n, *a)
        call(n, *a, table, pages, cache, qc, qr, 0.1)
    else:
        dims = (64, 64, 128) if what.endswith("2") else (128, 64, 128)
        x, dO = attn_inputs(1, [700], [700], 2, 1, *dims, "bf16")
        if what.startswith("forward"):
            attn_run(x, [700], [700], 0.1, True, "bf16")
        else:      # the forward starves too, and raises; the gradients are called without it
            N, H = 700, 2
            s = gdn.make_mla_attn(1, H, 1, N, N, *dims, "bf16", 0.1)
            dev = {k: t.cuda() for k, t in x.items()}
            ws = torch.empty(gdn.gdn_mla_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
            o, lse = torch.zeros(N, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, N, device="cuda")
            d = [torch.empty_like(t) for t in dev.values()]
            gdn.check(gdn.gdn_mla_bwd(s, *dev.values(), None, None, o, lse, dO.cuda(), *d, ws))
            gdn.check(gdn.gdn_last_device_status(ws))
    status = 0
except gdn.GdnError as e:
    status = e.status
secs = time.perf_counter() - t0
# calls with a first tile only
n = [60, 1]
a = (1, 16, 64, 32, 64, "bf16")
table, pages, cache, rows, qc, qr = setup(2, n, *a)
o, _ = call(n, *a, table, pages, cache, qc, qr, 0.1)
for b in range(2):
    close(o[b].cpu(), decode_ref(qc[b], qr[b], rows[b], 0.1)[0], "bf16", "fwd", "o")
x, dO = attn_inputs(3, [100], [100], 2, 2, 64, 32, 64, "bf16")
ro, _, _ = attn_ref(x, [100], [100], 0.1, True)
close(attn_run(x, [100], [100], 0.1, True, "bf16")[0], ro, "bf16", "fwd", "o")
print(json.dumps({"status": status, "secs": secs}))
"""


@pytest.mark.parametrize("what", ["forward 2", "forward 3", "gradients 2", "gradients 3", "decode", "decode pairs", "decode two groups"])
def test_starved_load_times_out_and_context_survives(what):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, GDN_TEST_STARVE_CHUNK="1", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", _CHILD, what], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["status"] == GDN_ERR_TIMEOUT
    assert res["secs"] < 60.0


_SECOND_WALK = r"""
import json
import torch
import linear_attention_recurrence_delta_gb300 as gdn
from tests.mla_testlib import attn_inputs, attn_ref
# 480 tokens of one head: a tile of queries walks at most four tiles of 128 keys, so step 5 of the queries' gradient belongs
# to the second walk that sharp scores ask for, and the pass over the keys has five steps of 96 queries, 0 to 4
N, H, dims = 480, 1, (128, 64, 128)
x, dO = attn_inputs(1, [N], [N], H, H, *dims, "bf16")
def grads(scale):
    s = gdn.make_mla_attn(1, H, H, N, N, *dims, "bf16", scale)
    dev = {k: t.cuda() for k, t in x.items()}
    ws = torch.empty(gdn.gdn_mla_workspace_bytes(s, 1), dtype=torch.uint8, device="cuda")
    ro, rl, _ = attn_ref(x, [N], [N], scale, True)
    d = [torch.empty_like(t) for t in dev.values()]
    gdn.check(gdn.gdn_mla_bwd(s, *dev.values(), None, None, ro.cuda().bfloat16(), rl.cuda().float().contiguous(), dO.cuda(), *d, ws))
    return gdn.gdn_last_device_status(ws)
sharp, flat = grads(1.0), grads(0.05)
print(json.dumps({"sharp": sharp, "flat": flat}))
"""


def test_starved_second_walk_times_out_and_context_survives():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, GDN_TEST_STARVE_CHUNK="5", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", _SECOND_WALK], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    assert json.loads(r.stdout.strip().splitlines()[-1]) == {"sharp": GDN_ERR_TIMEOUT, "flat": 0}
