"""The softmax weights of a tree attention with fp32 outputs, one by one: values are unit
vectors, so that O shows each weight, and scores lie in binary fractions, so that they are exact.

Each weight is compared with one whose score is 0, which cancels the sum.  Bound, relative: of
each of the two exp2 two steps of fp32 (2^-22), what three bf16 parts leave (half a step, 2^-8,
three times: below 2^-24), and two additions of three products by the tensor core (2^-23 each);
once the factor that turns scores into powers of two, and with soft-capping two more products and
the series, three roundings of |x| <= 2 (3 * 2 * 2^-24 * ln 2 < 2^-21.9); the products with 1 / l
(2^-23 together).  2 (2^-22 + 2^-24 + 2^-22) + 2^-21.9 + 2^-23 < 2^-19.3.  Two bf16 parts are off
by up to 2^-17."""

import math

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import F64, signed, tree, words_of

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TOL = 2.0 ** -19.3


def a_scale():
    """A scale whose product with log2(e) in fp32 is 1."""
    s = np.float32(math.log(2.0))
    for x in (s, np.nextafter(s, np.float32(1)), np.nextafter(s, np.float32(0))):
        if np.float32(x) * np.float32(1.4426950408889634) == np.float32(1):
            return float(x)
    raise AssertionError("none")


def parts(p, n):
    """p in n bf16 parts."""
    got = torch.zeros_like(p)
    for _ in range(n):
        got = got + (p - got).to(BF16).double()
    return got


@pytest.mark.parametrize("variant", ["plain", "softcap", "alibi"])
@pytest.mark.parametrize("off", [0, 64, 211, None])
@pytest.mark.parametrize("kv", [5, 61, 300, 440])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_each_weight(dev, d, kv, off, variant):
    """Keys off .. off + d (None: the last ones) have values of their own."""
    nodes, n_q, scale = 9, 6, a_scale()
    n = kv + nodes
    m = min(d, n)
    off = n - m if off is None else min(off, n - m)
    g = torch.Generator().manual_seed(d + kv + off)
    x = -torch.randint(0, 129, (n,), generator=g) / 64.0
    x[::16] = 0.0                                            # in every run of keys one of weight 1
    words = words_of(tree(nodes, kv))
    q = torch.zeros(nodes, n_q, d, dtype=BF16)
    q[..., 0] = 1.0
    k, v = torch.zeros(n, d, dtype=BF16), torch.zeros(n, d, dtype=BF16)
    k[:, 0] = x.to(BF16)
    v[off:off + m, :m] = torch.eye(m, dtype=BF16)
    kw = dict(plain=dict(), softcap=dict(softcap=2.0 ** 20),
              alibi=dict(alibi_slopes=torch.zeros(n_q, device=dev)))[variant]
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=dev)
    cache = lambda t: t[None, :, None].contiguous().to(dev)
    o, _ = attn.decode_tree(q.to(dev), cache(k), cache(v), i32([kv]), i32([0, nodes]),
                            torch.tensor(signed(words), dtype=torch.int64, device=dev), scale=scale, **kw)
    o = o.cpu().to(F64)
    want = torch.exp(x.to(F64) * scale)                      # (the scale that the call got is an fp32)
    seen = torch.tensor([[j < kv or (w >> (j - kv)) & 1 for j in range(n)] for w in words], dtype=torch.bool)
    unit = (torch.arange(n) % 16 == 0) & (torch.arange(n) >= off) & (torch.arange(n) < off + m)
    for i in range(nodes):
        at = int((unit & seen[i]).nonzero()[0])
        got = o[i, :, :m] / o[i, :, at - off, None]
        mine = torch.where(seen[i], want, 0.0)[off:off + m]
        assert bool(((got - mine).abs() <= TOL * mine).all()), float(((got - mine).abs() / mine.clamp(min=1e-9)).max())
    attn.check_device_status()


def test_the_bound_tells_two_parts_from_three():
    p = torch.exp2(-torch.arange(129, dtype=F64) / 64)
    assert float(((parts(p, 2) - p).abs() / p).max()) > 2 * TOL
    assert float(((parts(p, 3) - p).abs() / p).max()) < 2.0 ** -24
