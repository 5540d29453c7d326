"""The two ways from Python into rotary positions and a decode step with drafted
tokens, csrc/binding.cpp and drafts.py's own marshalling, give the same bits; what
the first does not take, it leaves to the second."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import signed, tree, words_of
from exact_io_aware_order_gb300 import _lib, drafts

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
NAMES = ("rope", "cache_append", "decode_tree", "verify_tree")


class Refuses:
    rope = cache_append = decode_tree = verify_tree = staticmethod(lambda *a: NotImplemented)


class Counts:
    """The binding, counting what it took."""

    def __init__(self):
        self.taken, self.b = 0, _lib.binding()

    def __getattr__(self, name):
        def call(*a):
            r = getattr(self.b, name)(*a)
            self.taken += r is not NotImplemented
            return r
        return call


def step(dev, paged, seed=0):
    """Rotation of a prompt, then append, attention and verification of a step; every result."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF16).to(dev)
    i32 = lambda x: torch.tensor(x, dtype=I32, device=dev)
    f = attn.rope_inv_freq(96, 50000.0, device=dev)
    got = [*attn.rope(rand(2, 30, 6, 128).transpose(1, 2), rand(2, 30, 2, 128).transpose(1, 2), f)]
    got += [attn.rope(rand(6, 41, 128), None, f, i32(list(range(41))), interleaved=True, inverse=True,
                      magnitude=2)[0]]
    lens, nodes = [1000, 3], [9, 30]
    ps = [tree(n, n) for n in nodes]
    cu, kv = i32([0, 9, 39]), i32(lens)
    shape = (80, 16, 2, 128) if paged else (2, 1040, 2, 128)
    kc, vc = rand(*shape), rand(*shape)
    table = torch.randperm(80, generator=g)[:66].view(1, 66).repeat(2, 1).to(I32)
    table[1, :4] = torch.tensor([x for x in range(80) if x not in table[0].tolist()][:4], dtype=I32)
    table = table.to(dev) if paged else None
    qkv = rand(39, 10, 128)
    q, k, v = qkv.split([6, 2, 2], dim=1)
    t = lambda x: x.transpose(0, 1)
    q = attn.cache_append(t(k), t(v), kc, vc, kv, cu, table, f, q=t(q))
    got.append(q)
    words = signed(sum((words_of(p) for p in ps), []))
    mask = torch.tensor(words, dtype=torch.int64, device=dev)
    got += attn.decode_tree(t(q), kc, vc, kv, cu, mask, table)
    got += attn.decode_tree(t(q), kc, vc, kv, cu, None, table, window_left=50, softcap=30,
                            out_dtype=BF16, max_kv_len=1030 if paged else None)
    one = attn.cache_append(k[:2], v[:2], kc, vc, kv + 31, None, table, f, q=qkv[:2, :6])
    got.append(one)
    p = torch.softmax(rand(39, 700).float(), 1)
    d = torch.softmax(rand(39, 700).float(), 1)
    u = torch.rand(39, generator=g).to(dev)
    for draft in (None, d):
        got += attn.verify_tree(p, i32(torch.randint(0, 700, (39,), generator=g).tolist()),
                                i32(sum(ps, [])), cu, u, u[:2], draft)
    attn.check_device_status()
    return got + [kc, vc]


@pytest.mark.parametrize("paged", [True, False])
def test_both_ways_agree(dev, paged, monkeypatch):
    counts = Counts()
    monkeypatch.setattr(drafts, "binding", lambda: counts)
    a = step(dev, paged)
    assert counts.taken == 8
    monkeypatch.setattr(drafts, "binding", Refuses)
    b = step(dev, paged)
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride()
        assert torch.equal(x, y)


def test_other_streams_go_the_long_way(dev, monkeypatch):
    counts = Counts()
    monkeypatch.setattr(drafts, "binding", lambda: counts)
    f = attn.rope_inv_freq(64, device=dev)
    q = torch.randn(1, 2, 9, 64, device=dev).to(BF16)
    want = attn.rope(q, None, f)[0]
    assert counts.taken == 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.rope(q, None, f, stream=side)[0]
    side.synchronize()
    assert counts.taken == 1 and torch.equal(want, got)
    with torch.cuda.stream(side):                            # torch's current stream is the call's
        got = attn.rope(q, None, f)[0]
    side.synchronize()
    assert counts.taken == 2 and torch.equal(want, got)


def test_tensors_without_memory_are_refused_by_drafts(dev):
    f = attn.rope_inv_freq(64, device=dev)
    q = torch.randn(3, 2, 9, 64, device=dev).to(BF16)
    with pytest.raises(Exception):
        torch.vmap(lambda x: attn.rope(x, None, f)[0])(q)
    attn.check_device_status()
