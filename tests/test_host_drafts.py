"""Host-side checks of rotary positions and of the calls of a decode step with
drafted tokens (no GPU needed, no kernel launched): every refusal that
include/attn.h documents, by its status."""

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


def rope(L, **kw):
    a = dict(q=P, qs=(10240, 1280, 128), qo=P, qos=(10240, 1280, 128), k=P, ks=(2560, 1280, 128),
             ko=P, kos=(2560, 1280, 128), f=P, pos=P, ps=10, B=2, n_q=8, n_kv=2, N=10, d=128,
             rot=128, m=1.0)
    a.update(kw)
    return L.attn_rope(a["q"], *a["qs"], a["qo"], *a["qos"], a["k"], *a["ks"], a["ko"], *a["kos"],
                       a["f"], a["pos"], a["ps"], a["B"], a["n_q"], a["n_kv"], a["N"], a["d"],
                       a["rot"], 0, 0, a["m"], None)


def append(L, **kw):
    a = dict(k=P, ks=(128, 1280), v=P, vs=(128, 1280), q=P, qs=(128, 1280), qo=P, qos=(128, 1280),
             kc=P, vc=P, bt=P, cu=P, lens=P, f=P, pos=P, B=3, T=10, n_q=8, n_kv=2, d=128, rot=128,
             m=1.0, bs=16, mb=8, nb=16, mx=128)
    a.update(kw)
    return L.attn_cache_append(a["k"], a["v"], *a["ks"], *a["vs"], a["q"], *a["qs"], a["qo"],
                               *a["qos"], a["kc"], a["vc"], a["bt"], a["cu"], a["lens"], a["f"],
                               a["pos"], a["B"], a["T"], a["n_q"], a["n_kv"], a["d"], a["rot"], 0,
                               a["m"], a["bs"], a["mb"], a["nb"], a["mx"], None)


ROT = [("SHAPE", dict(rot=8)), ("SHAPE", dict(rot=24)), ("SHAPE", dict(rot=144)),
       ("SHAPE", dict(rot=-16)), ("SHAPE", dict(m=float("inf"))), ("HEADDIM", dict(d=96)),
       ("NULL", dict(f=None)), ("ALIGN", dict(f=P + 4)), ("ALIGN", dict(pos=P + 2))]


@pytest.mark.parametrize("name,kw", ROT + [
    ("NULL", dict(q=None)), ("NULL", dict(qo=None)), ("NULL", dict(k=None)), ("NULL", dict(ko=None)),
    ("SHAPE", dict(B=0)), ("SHAPE", dict(N=0)), ("SHAPE", dict(n_q=0)), ("SHAPE", dict(n_kv=-1)),
    ("SHAPE", dict(B=1 << 20, N=1 << 20)), ("SHAPE", dict(n_q=65536)), ("SHAPE", dict(ps=9)),
    ("SHAPE", dict(ps=-1)), ("SHAPE", dict(qs=(10240, 1284, 128))),
    ("SHAPE", dict(ks=(2560, 1280, -128))), ("SHAPE", dict(qs=(10240, (1 << 40) + 8, 128))),
    ("SHAPE", dict(qos=(10240, 1280, 64))), ("SHAPE", dict(qos=(10232, 1280, 128))),
    ("SHAPE", dict(kos=(0, 1280, 128))), ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(qo=P + 2)),
    ("ALIGN", dict(k=P + 8)), ("ALIGN", dict(ko=P + 4))])
def test_rope_validation(L, E, name, kw):
    assert rope(L, **kw) == E[name]


def test_rope_accepts_what_is_documented(L, E):
    """Refused for their alignment only, which is looked at last."""
    for kw in (dict(qs=(0, 0, 0)), dict(qos=(128, 256, 2048)), dict(qos=(0, 1280, 128), B=1, ps=0),
               dict(n_kv=0, k=None, ko=None), dict(ps=0), dict(pos=None), dict(rot=16)):
        assert rope(L, **{**kw, "q": P + 2}) == E["ALIGN"], kw


@pytest.mark.parametrize("name,kw", ROT + [
    ("NULL", dict(k=None)), ("NULL", dict(v=None)), ("NULL", dict(kc=None)), ("NULL", dict(vc=None)),
    ("NULL", dict(lens=None)), ("NULL", dict(q=None)), ("NULL", dict(qo=None)),
    ("SHAPE", dict(B=0)), ("SHAPE", dict(T=0)), ("SHAPE", dict(B=(1 << 20) + 1)),
    ("SHAPE", dict(T=(1 << 24) + 1)), ("SHAPE", dict(cu=None)), ("SHAPE", dict(n_kv=0)),
    ("SHAPE", dict(n_q=-1)), ("SHAPE", dict(bs=0)), ("SHAPE", dict(mb=0)), ("SHAPE", dict(nb=0)),
    ("SHAPE", dict(bs=1 << 16, mb=1 << 15)), ("SHAPE", dict(bt=None, mx=0)),
    ("SHAPE", dict(bt=None, mx=(1 << 30) + 1)), ("SHAPE", dict(ks=(128, 1284))),
    ("SHAPE", dict(vs=(-128, 1280))), ("SHAPE", dict(qos=(64, 1280))), ("SHAPE", dict(qos=(0, 128))),
    ("ALIGN", dict(k=P + 8)), ("ALIGN", dict(v=P + 2)), ("ALIGN", dict(q=P + 8)),
    ("ALIGN", dict(qo=P + 8)), ("ALIGN", dict(kc=P + 8)), ("ALIGN", dict(vc=P + 8)),
    ("ALIGN", dict(bt=P + 2)), ("ALIGN", dict(cu=P + 1)), ("ALIGN", dict(lens=P + 2))])
def test_append_validation(L, E, name, kw):
    assert append(L, **kw) == E[name]


def test_append_accepts_what_is_documented(L, E):
    for kw in (dict(n_q=0, q=None, qo=None), dict(n_q=0, q=None, qo=None, f=None, rot=0),
               dict(bt=None, bs=0, mb=0, nb=0), dict(cu=None, T=3), dict(qos=(1024, 128)),
               dict(ks=(0, 0))):
        assert append(L, **{**kw, "k": P + 2}) == E["ALIGN"], kw
    assert append(L, n_q=0, q=None, qo=None, f=None) == E["NULL"]          # rot without frequencies
    assert append(L, f=None, rot=0) == E["NULL"]                           # queries without any


def tree(L, **kw):
    a = dict(q=P, kc=P, vc=P, bt=P, lens=P, cu=P, mask=P, ws=P, wn=1 << 40, o=P, lse=P, B=2, T=10,
             n_q=8, n_kv=2, d=128, bs=16, mb=8, nb=16, mx=128, scale=0.1, w=-1, cap=0.0, al=None,
             flags=0)
    a.update(kw)
    return L.attn_decode_tree(a["q"], a["kc"], a["vc"], a["bt"], a["lens"], a["cu"], a["mask"],
                              a["ws"], a["wn"], a["o"], a["lse"], a["B"], a["T"], a["n_q"],
                              a["n_kv"], a["d"], a["bs"], a["mb"], a["nb"], a["mx"], a["scale"],
                              a["w"], a["cap"], a["al"], a["flags"], None)


@pytest.mark.parametrize("name,kw", [
    ("NULL", dict(q=None)), ("NULL", dict(kc=None)), ("NULL", dict(vc=None)), ("NULL", dict(lens=None)),
    ("NULL", dict(cu=None)), ("NULL", dict(o=None)), ("NULL", dict(lse=None)), ("SHAPE", dict(B=0)),
    ("SHAPE", dict(B=65536)), ("SHAPE", dict(T=0)), ("SHAPE", dict(T=(1 << 24) + 1)),
    ("SHAPE", dict(n_q=0)), ("SHAPE", dict(bs=0)), ("SHAPE", dict(mb=0)), ("SHAPE", dict(nb=0)),
    ("SHAPE", dict(bs=1 << 16, mb=1 << 15)), ("SHAPE", dict(bt=None, mx=0)), ("SHAPE", dict(mx=-1)),
    ("SHAPE", dict(bt=None, mx=(1 << 30) + 1)), ("SHAPE", dict(scale=float("nan"))),
    ("SHAPE", dict(w=-2)), ("SHAPE", dict(cap=float("inf"))), ("SHAPE", dict(cap=1.0, al=P)),
    ("SHAPE", dict(flags=2)), ("HEADDIM", dict(d=96)), ("GQA", dict(n_q=7)), ("GQA", dict(n_q=130)),
    ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(kc=P + 8)), ("ALIGN", dict(vc=P + 2)),
    ("ALIGN", dict(bt=P + 2)), ("ALIGN", dict(lens=P + 2)), ("ALIGN", dict(cu=P + 2)),
    ("ALIGN", dict(mask=P + 4)), ("ALIGN", dict(ws=P + 8)), ("ALIGN", dict(o=P + 8)),
    ("ALIGN", dict(lse=P + 2)), ("ALIGN", dict(al=P + 2))])
def test_tree_validation(L, E, name, kw):
    assert tree(L, **kw) == E[name]


def test_tree_workspace_of_refused_arguments(L):
    f = L.attn_decode_tree_workspace_bytes
    for args in ((0, 8, 8, 2, 128, 5000, -1), (1, 0, 8, 2, 128, 5000, -1), (1, 8, 7, 2, 128, 5000, -1),
                 (1, 8, 130, 2, 128, 5000, -1), (1, 8, 8, 2, 96, 5000, -1), (1, 8, 8, 2, 128, -1, -1),
                 (1, 8, 8, 2, 128, 5000, -2), (1, 8, 8, 0, 128, 5000, -1)):
        assert f(*args) == 0


def test_tree_masks():
    """The words from parents, on the CPU: a chain of 64, trees, rows of no sequence."""
    import torch

    import exact_io_aware_order_gb300 as attn
    from drafts_util import signed, tree as parents, words_of

    ps = [parents(n, s, s == 1) for s, n in enumerate([1, 64, 7, 30, 64])]
    cu = [0]
    for p in ps:
        cu.append(cu[-1] + len(p))
    cu.insert(2, cu[2])                                     # an empty sequence
    w = attn.tree_mask(torch.tensor(sum(ps, []) + [0, 5], dtype=torch.int32), torch.tensor(cu, dtype=torch.int32))
    assert w.tolist() == signed(sum((words_of(p) for p in ps), [])) + [0, 0]


def verify(L, **kw):
    a = dict(p=P, ps=100, q=P, qs=100, tok=P, par=P, cu=P, u=P, ul=P, n=P, path=P, nt=P, B=2, T=10, V=100)
    a.update(kw)
    return L.attn_verify_tree(a["p"], a["ps"], a["q"], a["qs"], a["tok"], a["par"], a["cu"], a["u"],
                              a["ul"], a["n"], a["path"], a["nt"], a["B"], a["T"], a["V"], None)


@pytest.mark.parametrize("name,kw", [("NULL", {k: None}) for k in ("p", "tok", "par", "cu", "u", "ul", "n", "path", "nt")] + [
    ("ALIGN", {k: P + 2}) for k in ("p", "q", "tok", "par", "cu", "u", "ul", "n", "path", "nt")] + [
    ("SHAPE", dict(B=0)), ("SHAPE", dict(B=(1 << 20) + 1)), ("SHAPE", dict(T=0)), ("SHAPE", dict(T=(1 << 24) + 1)),
    ("SHAPE", dict(V=0)), ("SHAPE", dict(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31)), ("SHAPE", dict(ps=99)),
    ("SHAPE", dict(qs=99)), ("SHAPE", dict(ps=(1 << 40) + 1))])
def test_verify_validation(L, E, name, kw):
    assert verify(L, **kw) == E[name]


def test_verify_without_drafts(L, E):
    assert verify(L, q=None, qs=0, nt=P + 2) == E["ALIGN"]


def test_binding_takes_only_what_it_knows(L):
    """csrc/binding.cpp on the CPU: everything is refused (NotImplemented), so drafts.py's
    checks and messages decide."""
    import torch

    from exact_io_aware_order_gb300._lib import binding

    b = binding()
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 3, 64, dtype=torch.bfloat16)
    f, n, p = torch.ones(32, dtype=torch.float64), torch.zeros(2, dtype=torch.int32), torch.ones(2, 5)
    u = torch.zeros(2)
    for name, args in (("rope", (x, None, f, None, False, False, 1.0, None, None)),
                       ("cache_append", (x, x, c, c, n, None, None, f, None, x, False, 1.0, None)),
                       ("decode_tree", (x, c, c, n, n, None, None, None, None, None, None, None, -1, 0.0, None, False)),
                       ("verify_tree", (p, n, n, n, u, u, None, None, None, None))):
        call = getattr(b, name)
        for wrong in ((), args, (None,) * len(args), (1,) * len(args), args[:-1]):
            assert call(*wrong) is NotImplemented


def test_tree_masks_of_parents_that_are_none():
    """A parent that is not a smaller index of the sequence is none, and reads nothing outside."""
    import torch

    import exact_io_aware_order_gb300 as attn

    big = 2**31 - 1
    parents = torch.tensor([-1, 1, 0, big, 3, -9, -1, 5, 0, 0], dtype=torch.int32)
    w = attn.tree_mask(parents, torch.tensor([0, 6, 9], dtype=torch.int32))
    assert w.tolist() == [1, 2, 5, 8, 24, 32, 1, 2, 5, 0]
