"""The two ways from Python into the 8-bit cache's calls, csrc/binding.cpp and
api.py's own marshalling, give the same bits; what the first does not take, it
leaves to the second."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from exact_io_aware_order_gb300 import _lib, api
from cache_fp8_util import Cache, rows

pytestmark = pytest.mark.gpu


class Refuses:
    cache_write_fp8 = cache_read_fp8 = decode_fp8 = staticmethod(lambda *a: NotImplemented)


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


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def session(dev, paged, alibi):
    """Write, append, decode and read; returns every result."""
    c = Cache(2, 2, 64, [900, 40], 24, paged, seed=5)
    (k, v, ks, vs), table = c.on(dev)
    kn, vn = rows(2, 930, 64, 1).to(dev), rows(2, 930, 64, 2).to(dev)
    cu, lens = i32([0, 890, 920], dev), i32([0, 0], dev)
    attn.cache_write_fp8(kn, vn, k, v, ks, vs, lens, cu, table, block_size=24)
    lens = i32([890, 30], dev)
    q = torch.randn(2, 6, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    sl = torch.tensor([0.5 ** h for h in range(6)], device=dev) if alibi else None
    one = kn[:, :2].transpose(0, 1).contiguous()
    got = [*attn.decode_append_fp8(q, one, one, k, v, ks, vs, lens, table, block_size=24,
                                   alibi_slopes=sl)]
    lens += 1
    got += attn.decode_fp8(q, k, v, ks, vs, lens, table, num_splits=3, window_left=100, scale=0.2,
                           block_size=24, softcap=0 if alibi else 20)
    out = torch.empty(2, 6, 64, device=dev)
    got += attn.decode_fp8(q, k, v, ks, vs, lens, table, out=out, max_kv_len=897 if paged else None,
                           block_size=24)
    assert got[-2] is out
    got += attn.cache_read_fp8(k, v, ks, vs, i32([0, 891, 920], dev), 920, table, block_size=24)
    attn.check_device_status()
    return got + [k, v, ks, vs]


@pytest.mark.parametrize("paged,alibi", [(True, False), (False, True)])
def test_both_ways_give_the_same_bits(dev, monkeypatch, paged, alibi):
    count = Counts()
    monkeypatch.setattr(api, "binding", lambda: count)
    fast = session(dev, paged, alibi)
    assert count.taken == 5                                   # all of the session
    monkeypatch.setattr(api, "binding", lambda: Refuses)
    slow = session(dev, paged, alibi)
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_leaves_the_rest_to_python(dev, monkeypatch):
    """Subclasses, other strides of a cache, numpy numbers, refused calls."""
    count = Counts()
    monkeypatch.setattr(api, "binding", lambda: count)
    c = Cache(1, 2, 64, [40], 16, True, seed=5)
    (k, v, ks, vs), table = c.on(dev)
    ks.fill_(1.0), vs.fill_(1.0)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=dev)
    lens = i32([40], dev)

    class Sub(torch.Tensor):
        pass

    attn.decode_fp8(q.as_subclass(Sub), k, v, ks, vs, lens, table)
    assert count.taken == 0
    with pytest.raises(ValueError):
        attn.decode_fp8(q, k, v, ks[:1], vs, lens, table)
    with pytest.raises(_lib.AttnError):
        attn.decode_fp8(q, k, v, ks, vs, lens, table, softcap=-1.0)
    with pytest.raises(TypeError):
        attn.decode_fp8(q.float(), k, v, ks, vs, lens, table)
    assert count.taken == 0
    attn.decode_fp8(q, k, v, ks, vs, lens, table)
    assert count.taken == 1
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                             # the current stream is followed
        torch.cuda._sleep(1000000)
        o, _ = attn.decode_fp8(q, k, v, ks, vs, lens, table)
        done = torch.cuda.Event()
        done.record()
    assert not done.query() and count.taken == 2
    side.synchronize()
    attn.check_device_status()
