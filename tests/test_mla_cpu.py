"""The latent-attention entry points refuse bad arguments before any device work, and size their workspaces (no GPU)."""
import ctypes
import os

import pytest
import torch

import linear_attention_recurrence_delta_gb300 as gdn

FAKE = 1 << 20        # a 256-byte aligned address; never dereferenced
BIG = 1 << 40
OK, NULL, SHAPE, ALIGN, MODE, WS = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        from linear_attention_recurrence_delta_gb300 import _build
        _build.build()
    return gdn.load()


def view(p=FAKE, tok=1024, head=128):
    return gdn.gdn_mla_view_t(p, tok, head)


def refused(status, want):
    assert status == want, f"{gdn.gdn_status_string(status)}"


# ---------------------------------------------------------------- norm, rotation, cache write

def prep(shape, **kw):
    a = dict(kv=(FAKE, 320), w=FAKE, rot=FAKE, pos=FAKE, seq=None, table=None, qr=view(), lat=view(), kr=view(), qr_out=view())
    a.update(kw)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return int(gdn.load().gdn_mla_prep(ctypes.byref(shape) if shape else None, *a["kv"], a["w"], a["rot"], a["pos"], a["seq"],
                                       a["table"], ref(a["qr"]), ref(a["lat"]), ref(a["kr"]), ref(a["qr_out"]), 0))


def test_prep_refusals():
    s = gdn.make_mla_prep(8, 4, 256, 64, "bf16", 100)
    refused(prep(None), NULL)
    for bad in (dict(dc=0), dict(dc=4), dict(dc=1032), dict(dr=8), dict(dr=144), dict(N=-1), dict(H=-1), dict(npos=-1),
                dict(eps=-1.0), dict(eps=float("nan"))):
        a = dict(N=8, H=4, dc=256, dr=64, npos=100)
        a.update(bad)
        refused(prep(gdn.make_mla_prep(**a)), SHAPE)
        assert gdn.gdn_mla_prep_workspace_bytes(gdn.make_mla_prep(**a)) == 0
    refused(prep(gdn.make_mla_prep(8, 4, 256, 64, 7, 100)), MODE)
    for k in ("w", "rot", "pos", "qr", "lat", "kr", "qr_out"):
        refused(prep(s, **{k: None}), NULL)
    refused(prep(s, kv=(None, 320)), NULL)
    refused(prep(s, kv=(FAKE, 312)), SHAPE)
    refused(prep(s, kv=(FAKE, 324)), ALIGN)
    refused(prep(s, kv=(FAKE + 8, 320)), ALIGN)
    refused(prep(s, pos=FAKE + 2), ALIGN)
    refused(prep(s, qr=view(FAKE + 2)), ALIGN)
    refused(prep(s, qr=view(tok=1020)), ALIGN)
    refused(prep(s, qr_out=view(head=4)), ALIGN)
    refused(prep(s, lat=view(tok=0)), SHAPE)
    refused(prep(s, kr=view(tok=-64)), SHAPE)
    paged = dict(N=8, H=4, dc=256, dr=64, npos=100, B=2, page=64, npages=9, maxpages=4)
    p = gdn.make_mla_prep(**paged)
    refused(prep(p), NULL)
    refused(prep(p, seq=FAKE), NULL)
    refused(prep(p, seq=FAKE, table=FAKE, lat=view(FAKE + 8)), ALIGN)
    for k in ("B", "npages", "maxpages"):
        refused(prep(gdn.make_mla_prep(**{**paged, k: 0})), SHAPE)
    refused(prep(gdn.make_mla_prep(**{**paged, "npages": 1 << 30})), SHAPE)
    refused(prep(gdn.make_mla_prep(**{**paged, "page": -1})), SHAPE)
    assert gdn.gdn_mla_prep_workspace_bytes(p) == 0


def prep_bwd(shape, **kw):
    a = dict(kv=(FAKE, 320), w=FAKE, rot=FAKE, pos=FAKE, dlat=view(), dkr=view(), dqr=view(), dkv=(FAKE, 320), dw=FAKE,
             dqr_out=view(), ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return int(gdn.load().gdn_mla_prep_bwd(ctypes.byref(shape), *a["kv"], a["w"], a["rot"], a["pos"], ref(a["dlat"]),
                                           ref(a["dkr"]), ref(a["dqr"]), *a["dkv"], a["dw"], ref(a["dqr_out"]), a["ws"],
                                           a["ws_bytes"], 0))


def test_prep_bwd_refusals():
    s = gdn.make_mla_prep(8, 4, 256, 64, "bf16", 100)
    need = gdn.gdn_mla_prep_workspace_bytes(s)
    assert need >= 256 and need % 256 == 0
    for k in ("w", "rot", "pos", "dlat", "dkr", "dqr", "dw", "dqr_out"):
        refused(prep_bwd(s, **{k: None}), NULL)
    refused(prep_bwd(s, dkv=(None, 320)), NULL)
    refused(prep_bwd(s, dkv=(FAKE, 256)), SHAPE)
    refused(prep_bwd(s, dkv=(FAKE, 322)), ALIGN)
    refused(prep_bwd(s, ws=None), WS)
    refused(prep_bwd(s, ws_bytes=need - 1), WS)
    refused(prep_bwd(s, ws=FAKE + 128), ALIGN)
    refused(prep_bwd(gdn.make_mla_prep(8, 4, 256, 64, "bf16", 100, B=1, page=8, npages=1, maxpages=1)), MODE)


# ---------------------------------------------------------------- expanded attention

ATTN = dict(B=2, H=4, Hkv=2, Tq=33, Tk=65, dn=64, dr=64, dv=128)


def attn_shape(**kw):
    return gdn.make_mla_attn(**{**ATTN, **kw})


def attn(shape, backward, **kw):
    a = dict(qn=view(), qr=view(), kn=view(), kr=view(), v=view(), cu_q=None, cu_k=None, o=FAKE, lse=FAKE, dO=FAKE, dqn=view(),
             dqr=view(), dkn=view(), dkr=view(), dv=view(), ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    ins = [ref(a[k]) for k in ("qn", "qr", "kn", "kr", "v")] + [a["cu_q"], a["cu_k"], a["o"], a["lse"]]
    tail = [a["ws"], a["ws_bytes"], 0]
    sp = ctypes.byref(shape) if shape else None
    if not backward:
        return int(gdn.load().gdn_mla_fwd(sp, *ins, *tail))
    return int(gdn.load().gdn_mla_bwd(sp, *ins, a["dO"], *[ref(a[k]) for k in ("dqn", "dqr", "dkn", "dkr", "dv")], *tail))


@pytest.mark.parametrize("backward", [0, 1])
def test_attention_refusals(backward):
    s = attn_shape()
    refused(attn(None, backward), NULL)
    for bad in (dict(B=0), dict(B=65536), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(dn=0), dict(dn=12), dict(dn=136), dict(dr=4),
                dict(dr=72), dict(dv=0), dict(dv=136), dict(Tq=-1, Nq=0), dict(Tk=-1, Nk=0), dict(Nq=-1), dict(Nk=-1),
                dict(scale=float("nan")), dict(scale=-0.1)):
        refused(attn(attn_shape(**bad), backward), SHAPE)
        assert gdn.gdn_mla_workspace_bytes(attn_shape(**bad), backward) == 0
    refused(attn(attn_shape(io=5), backward), MODE)
    refused(attn(attn_shape(Nq=65), backward), SHAPE)          # no offsets: the rows have to be B * T
    refused(attn(attn_shape(Nk=131), backward), SHAPE)
    for k in ("qn", "qr", "kn", "kr", "v"):
        refused(attn(s, backward, **{k: None}), NULL)
        refused(attn(s, backward, **{k: view(FAKE + 4)}), ALIGN)
        refused(attn(s, backward, **{k: view(tok=1028)}), ALIGN)
        refused(attn(s, backward, **{k: view(tok=0)}), SHAPE)
        if k != "kr":
            refused(attn(s, backward, **{k: view(head=-8)}), SHAPE)
    refused(attn(s, backward, o=None), NULL)
    refused(attn(s, backward, o=FAKE + 8), ALIGN)
    refused(attn(s, backward, cu_q=FAKE + 2), ALIGN)
    need = gdn.gdn_mla_workspace_bytes(s, backward)
    assert need >= 256 and need % 256 == 0
    refused(attn(s, backward, ws=None), WS)
    refused(attn(s, backward, ws_bytes=need - 1), WS)
    refused(attn(s, backward, ws=FAKE + 16), ALIGN)
    if backward:
        for k in ("lse", "dO", "dqn", "dqr", "dkn", "dkr", "dv"):
            refused(attn(s, 1, **{k: None}), NULL)
        for k in ("dqn", "dqr", "dkn", "dkr", "dv"):
            refused(attn(s, 1, **{k: view(FAKE + 2)}), ALIGN)


# ---------------------------------------------------------------- the paged latent cache

CACHE = dict(B=3, T=1, H=16, dc=256, dr=64, page=64, npages=40, maxpages=10)


def decode(shape, **kw):
    a = dict(qc=view(), qr=view(), cache=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    ref = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return int(gdn.load().gdn_mla_decode(ctypes.byref(shape) if shape else None, ref(a["qc"]), ref(a["qr"]), a["cache"],
                                         a["table"], a["lens"], a["o"], a["lse"], a["ws"], a["ws_bytes"], 0))


def test_decode_refusals():
    s = gdn.make_mla_cache(**CACHE)
    refused(decode(None), NULL)
    for bad in (dict(B=0), dict(T=0), dict(T=9), dict(H=0), dict(T=8, H=129), dict(dc=0), dict(dc=20), dict(dc=520), dict(dr=4),
                dict(dr=72), dict(page=0), dict(page=12), dict(npages=0), dict(maxpages=0), dict(npages=1 << 26),
                dict(maxpages=1 << 26), dict(scale=float("nan")), dict(scale=-1.0),
                dict(B=65535, maxpages=1 << 20)):
        refused(decode(gdn.make_mla_cache(**{**CACHE, **bad})), SHAPE)
        assert gdn.gdn_mla_decode_workspace_bytes(gdn.make_mla_cache(**{**CACHE, **bad})) == 0
    refused(decode(gdn.make_mla_cache(**CACHE, io=3)), MODE)
    for k in ("qc", "qr", "cache", "table", "lens", "o"):
        refused(decode(s, **{k: None}), NULL)
    refused(decode(s, qc=view(FAKE + 8)), ALIGN)
    refused(decode(s, qr=view(head=4)), ALIGN)
    refused(decode(s, cache=FAKE + 8), ALIGN)
    refused(decode(s, table=FAKE + 2), ALIGN)
    refused(decode(s, lens=FAKE + 1), ALIGN)
    need = gdn.gdn_mla_decode_workspace_bytes(s)
    assert need >= 256 and need % 256 == 0
    refused(decode(s, ws_bytes=need - 1), WS)
    refused(decode(s, ws=None), WS)
    refused(decode(s, ws=FAKE + 64), ALIGN)


# ---------------------------------------------------------------- the binding's views

def test_views():
    from linear_attention_recurrence_delta_gb300.mla import _view
    t = torch.zeros(5, 4, 24)
    v = _view(t[..., 8:])
    assert (v.p, v.tok, v.head) == (t.data_ptr() + 32, 96, 24)
    v = _view(torch.zeros(2, 5, 4, 24))
    assert (v.tok, v.head) == (96, 24)
    v = _view(torch.zeros(2, 1, 4, 24))
    assert (v.tok, v.head) == (96, 24)
    v = _view(torch.zeros(1, 4, 24)[:, :, :20])
    assert v.head == 24 and v.tok % 8 == 0 and v.tok > 0
    v = _view(torch.zeros(7, 24)[:, :16], heads=False)
    assert v.tok == 24
    assert _view(None) is None
    for bad in (torch.zeros(5, 24), torch.zeros(2, 2, 5, 4, 24), torch.zeros(5, 24, 4).transpose(1, 2),
                torch.zeros(2, 7, 4, 24)[:, :5]):
        with pytest.raises(ValueError):
            _view(bad)


def test_names_are_exported():
    for n in ("gdn_mla_prep", "gdn_mla_prep_bwd", "gdn_mla_prep_workspace_bytes", "gdn_mla_fwd", "gdn_mla_bwd",
              "gdn_mla_workspace_bytes", "gdn_mla_decode", "gdn_mla_decode_workspace_bytes"):
        assert callable(getattr(gdn, n)) and hasattr(gdn.load(), n)


# ---------------------------------------------------------------- the sources

def test_each_cta_loads_its_own_tiles():
    """The library is loaded by every rank of a job on several GPUs: no load or commit of it goes to several CTAs at once."""
    from linear_attention_recurrence_delta_gb300 import _build
    for path in _build._inputs():
        if not path.endswith(".py"):
            with open(path) as f:
                assert "multicast" not in f.read().lower(), path


def test_prep_wants_positions():
    """With no rows of rot every token's position would be outside the table: a call that writes nothing is refused."""
    s = gdn.make_mla_prep(8, 4, 256, 64)
    assert s.npos == 0
    refused(prep(s), SHAPE)
    refused(prep_bwd(s), SHAPE)
    refused(prep(gdn.make_mla_prep(8, 4, 256, 0), rot=None), SHAPE)
    assert gdn.gdn_mla_prep_workspace_bytes(s) == 0
    assert prep(gdn.make_mla_prep(0, 4, 256, 64)) == OK


def _calls():
    """Each operator as a function of its tensors by name, with tensors of the types that it reads."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *shape, dt=bf: torch.zeros(shape, dtype=dt)  # noqa: E731
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    p = gdn.make_mla_prep(8, 4, 64, 32, "bf16", 10)
    pp = gdn.make_mla_prep(8, 4, 64, 32, "bf16", 10, B=2, page=8, npages=4, maxpages=2)
    a = gdn.make_mla_attn(1, 4, 2, 8, 8, 64, 32, 64)
    c = gdn.make_mla_cache(2, 1, 4, 64, 32, 8, 4, 2)
    rows = dict(kv=z(8, 96), w=z(64, dt=f32), rot=z(10, 32, dt=f32), pos=z(8, dt=i32))
    qkv = dict(qn=z(8, 4, 64), qr=z(8, 4, 32), kn=z(8, 2, 64), kr=z(8, 32), v=z(8, 2, 64), cu_q=z(2, dt=i32), cu_k=z(2, dt=i32),
               o=z(8, 4, 64), lse=z(4, 8, dt=f32))
    return {
        "prep": (lambda **t: gdn.gdn_mla_prep(p, **t, seq=None, table=None),
                 dict(rows, qr=z(8, 4, 32), lat=z(8, 64), kr=z(8, 32), qr_out=z(8, 4, 32))),
        "prep paged": (lambda **t: gdn.gdn_mla_prep(pp, **t, kr=None),
                       dict(rows, seq=z(8, dt=i32), table=z(2, 2, dt=i32), qr=z(8, 4, 32), lat=z(4, 8, 96), qr_out=z(8, 4, 32))),
        "prep_bwd": (lambda **t: gdn.gdn_mla_prep_bwd(p, **t, ws=ws),
                     dict(rows, dlat=z(8, 64), dkr=z(8, 32), dqr=z(8, 4, 32), dkv=z(8, 96), dw=z(64, dt=f32), dqr_out=z(8, 4, 32))),
        "fwd": (lambda **t: gdn.gdn_mla_fwd(a, **t, ws=ws), qkv),
        "bwd": (lambda **t: gdn.gdn_mla_bwd(a, **t, ws=ws),
                dict(qkv, dO=z(8, 4, 64), dqn=z(8, 4, 64), dqr=z(8, 4, 32), dkn=z(8, 2, 64), dkr=z(8, 32), dv=z(8, 2, 64))),
        "decode": (lambda **t: gdn.gdn_mla_decode(c, **t, ws=ws),
                   dict(qc=z(2, 1, 4, 64), qr=z(2, 1, 4, 32), cache=z(4, 8, 96), table=z(2, 2, dt=i32), lens=z(2, dt=i32),
                        o=z(2, 1, 4, 64), lse=z(2, 1, 4, dt=f32))),
    }


@pytest.mark.parametrize("what", list(_calls()))
def test_tensors_of_other_types(what, monkeypatch):
    """Positions, offsets, lengths and tables in torch's default int64, norm weights in bf16 and any other tensor of a type
    that the call would misread raise before the library sees an address."""
    call, tensors = _calls()[what]

    class Reached(Exception):
        pass

    class Lib:
        def __getattr__(self, name):
            def f(*args):
                raise Reached
            return f

    from linear_attention_recurrence_delta_gb300 import mla
    monkeypatch.setattr(mla, "load", Lib)
    monkeypatch.setattr(mla, "_stream", lambda s: 0)
    with pytest.raises(Reached):
        call(**tensors)
    for name, t in tensors.items():
        other = {torch.int32: torch.int64, torch.float32: torch.bfloat16, torch.bfloat16: torch.float32}[t.dtype]
        with pytest.raises(ValueError):
            call(**{**tensors, name: t.to(other)})


def test_alignment_of_rot():
    """Of the fp32 and int32 arrays rot alone is read 16 bytes at a time."""
    s = gdn.make_mla_prep(8, 4, 256, 64, "bf16", 100)
    refused(prep(s, rot=FAKE + 4), ALIGN)
    refused(prep_bwd(s, rot=FAKE + 8), ALIGN)
    refused(prep(s, w=FAKE + 2), ALIGN)
