"""Host-side checks of the 8-bit cache's entry points (no GPU needed, no kernel
launched): every refusal that include/attn.h documents, by its status."""

import pytest

from exact_io_aware_order_gb300 import _lib, build

P = 0x10000  # fake aligned address; validation fails before it is used


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


@pytest.fixture(scope="module")
def E():
    return {n[len("ATTN_ERR_"):]: v for n, v in _lib.status_codes().items() if "ERR" in n}


BASE = dict(kc=P, vc=P, ks=P, vs=P, bt=P, n_kv=2, d=128, bs=16, mb=8, nb=16, mx=128)


def rows(L, read, **kw):
    a = dict(BASE, k=P, v=P, kt=128, kh=1280, vt=128, vh=1280, cu=P, lens=P, B=3, T=10)
    a.update(kw)
    tail = (a["B"], a["T"], a["n_kv"], a["d"], a["bs"], a["mb"], a["nb"], a["mx"], None)
    st = (a["kt"], a["kh"], a["vt"], a["vh"])
    if read:
        return L.attn_cache_read_fp8(a["kc"], a["vc"], a["ks"], a["vs"], a["k"], a["v"], *st,
                                     a["bt"], a["cu"], a["lens"], *tail)
    return L.attn_cache_write_fp8(a["k"], a["v"], *st, a["kc"], a["vc"], a["ks"], a["vs"], a["bt"],
                                  a["cu"], a["lens"], *tail)


def splitkv(L, **kw):
    a = dict(BASE, q=P, lens=P, S=4, op=P, lp=P, B=2, n_q=8, scale=0.1, w=-1, cap=0.0, al=None)
    a.update(kw)
    return L.attn_decode_fp8_splitkv(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["lens"],
                                     a["S"], a["op"], a["lp"], a["B"], a["n_q"], a["n_kv"], a["d"],
                                     a["bs"], a["mb"], a["nb"], a["mx"], a["scale"], a["w"],
                                     a["cap"], a["al"], None)


def decode(L, **kw):
    a = dict(BASE, q=P, kn=None, vn=None, lens=P, S=4, ws=P, wn=1 << 30, o=P, lse=P, B=2, n_q=8,
             scale=0.1, w=-1, cap=0.0, al=None)
    a.update(kw)
    return L.attn_decode_fp8(a["q"], a["kn"], a["vn"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"],
                             a["lens"], a["S"], a["ws"], a["wn"], a["o"], a["lse"], a["B"],
                             a["n_q"], a["n_kv"], a["d"], a["bs"], a["mb"], a["nb"], a["mx"],
                             a["scale"], a["w"], a["cap"], a["al"], None)


CACHE = [("NULL", dict(kc=None)), ("NULL", dict(vc=None)), ("NULL", dict(ks=None)),
         ("NULL", dict(vs=None)), ("SHAPE", dict(n_kv=0)), ("SHAPE", dict(bs=0)),
         ("SHAPE", dict(bs=(1 << 20) + 1)), ("SHAPE", dict(mb=0)), ("SHAPE", dict(nb=0)),
         ("SHAPE", dict(bs=1 << 16, mb=1 << 15)), ("SHAPE", dict(bt=None, mx=0)),
         ("SHAPE", dict(bt=None, mx=(1 << 30) + 1)), ("SHAPE", dict(mx=-1)),
         ("HEADDIM", dict(d=96)), ("HEADDIM", dict(d=512)), ("ALIGN", dict(kc=P + 8)),
         ("ALIGN", dict(vc=P + 1)), ("ALIGN", dict(ks=P + 2)), ("ALIGN", dict(vs=P + 1)),
         ("ALIGN", dict(bt=P + 2))]

ROWS = [("NULL", dict(k=None)), ("NULL", dict(v=None)), ("SHAPE", dict(B=0)), ("SHAPE", dict(T=0)),
        ("SHAPE", dict(B=(1 << 20) + 1)), ("SHAPE", dict(T=(1 << 24) + 1)),
        ("SHAPE", dict(kt=-128)), ("SHAPE", dict(vh=132)), ("SHAPE", dict(kh=4)),
        ("SHAPE", dict(T=1 << 24, bs=1, mb=1, n_kv=1000)), ("ALIGN", dict(k=P + 8)),
        ("ALIGN", dict(v=P + 2)), ("ALIGN", dict(cu=P + 2)), ("ALIGN", dict(lens=P + 1))]


@pytest.mark.parametrize("name,kw", CACHE + ROWS)
@pytest.mark.parametrize("read", [False, True])
def test_rows_validation(L, E, read, name, kw):
    assert rows(L, read, **kw) == E[name]


def test_rows_validation_of_one_direction(L, E):
    assert rows(L, False, lens=None) == E["NULL"]
    assert rows(L, False, cu=None) == E["SHAPE"]             # one row a sequence: T must be B
    assert rows(L, True, cu=None) == E["NULL"]
    assert rows(L, True, kt=0) == E["SHAPE"]                 # written rows on one another
    assert rows(L, True, vh=64) == E["SHAPE"]


@pytest.mark.parametrize("which", ["k", "v"])
def test_read_into_rows_on_one_another(L, E, which):
    """3 tokens of 2 heads, 128 columns: refused unless every row has a place of
    its own (16 bytes off: what is refused for that has passed the strides)."""
    at = lambda t, h: rows(L, True, **{which: P + 8, which + "t": t, which + "h": h}, T=3)
    assert at(128, 384) == at(256, 128) == at(128, 400) == at(512, 256) == E["ALIGN"]
    assert at(128, 128) == at(128, 376) == at(128, 256) == at(248, 128) == E["SHAPE"]
    for T, n_kv, t, h in ((1, 2, 0, 128), (3, 1, 128, 0)):
        assert rows(L, True, **{which: P + 8, which + "t": t, which + "h": h}, T=T,
                    n_kv=n_kv) == E["ALIGN"]


DECODE = [("NULL", dict(q=None)), ("NULL", dict(lens=None)), ("SHAPE", dict(B=0)),
          ("SHAPE", dict(B=65536)), ("SHAPE", dict(scale=0.0)), ("SHAPE", dict(scale=float("nan"))),
          ("SHAPE", dict(w=-2)), ("SHAPE", dict(cap=-1.0)), ("SHAPE", dict(cap=float("inf"))),
          ("SHAPE", dict(cap=2.0, al=P)), ("GQA", dict(n_q=7)), ("GQA", dict(n_q=130)),
          ("SPLITS", dict(S=-1)), ("SPLITS", dict(S=1025)), ("ALIGN", dict(q=P + 8)),
          ("ALIGN", dict(lens=P + 2)), ("ALIGN", dict(al=P + 2))]


@pytest.mark.parametrize("name,kw", CACHE + DECODE)
@pytest.mark.parametrize("call", [splitkv, decode])
def test_decode_validation(L, E, call, name, kw):
    assert call(L, **kw) == E[name]


def test_decode_outputs_validation(L, E):
    assert splitkv(L, op=None) == E["NULL"] and splitkv(L, lp=None) == E["NULL"]
    assert splitkv(L, op=P + 4) == E["ALIGN"] and splitkv(L, lp=P + 2) == E["ALIGN"]
    assert decode(L, o=None) == E["NULL"] and decode(L, lse=None) == E["NULL"]
    assert decode(L, o=P + 4) == E["ALIGN"] and decode(L, ws=P + 8) == E["ALIGN"]
    assert decode(L, kn=P) == E["NULL"] and decode(L, vn=P) == E["NULL"]      # both or none
    assert decode(L, kn=P + 2, vn=P) == E["ALIGN"]


def test_workspace_bytes(L):
    f = lambda S, B, H, Hk, d: L.attn_decode_fp8_workspace_bytes(S, B, H, Hk, d, 5000, -1)
    assert f(1, 4, 32, 8, 128) == 0 and f(-1, 4, 32, 8, 128) == 0 and f(4, 0, 32, 8, 128) == 0
    for S, B, H, d in [(2, 1, 1, 64), (76, 1, 28, 128), (1024, 65535, 64, 256)]:
        n = f(S, B, H, 1, d)
        assert n == -(-S * B * H * d * 4 // 256) * 256 + S * B * H * 4


def test_binding_takes_only_what_it_knows(L):
    """csrc/binding.cpp on the CPU: everything is refused (NotImplemented), so
    api.py's checks and messages decide."""
    import torch

    from exact_io_aware_order_gb300._lib import binding

    b = binding()
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    u = torch.zeros(2, 16, 3, 64, dtype=torch.uint8)
    s, n = torch.ones(2, 3), torch.zeros(2, dtype=torch.int32)
    for args in ((), (1,) * 10, (x, x, u, u, s, s, n, None, None, 16), (None,) * 10):
        assert b.cache_write_fp8(*args) is NotImplemented
    for args in ((), (u, u, s, s, n, 4, None, None, 16), (None,) * 9, (u, u, s, s, n, "4", None, None, 16)):
        assert b.cache_read_fp8(*args) is NotImplemented
    for args in ((), (x, None, None, u, u, s, s, n, None, 0, None, None, None, None, None, -1, 0.0,
                      None, 16), (None,) * 19):
        assert b.decode_fp8(*args) is NotImplemented
