"""Decode over an 8-bit cache with 9 to 64 query heads a kv head: every form of
the teams (one for up to 16 heads, two for up to 32, four beyond), at every
head_dim, over lengths that take several tiles a warp and end inside one."""

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
import oracle
from oracle import cache_fp8_ref as C
from cache_fp8_util import assert_cache, rows
from test_gpu_decode_fp8 import close, filled, i32, queries, reference, slopes_of

pytestmark = pytest.mark.gpu

# (query heads a kv head, head_dim, window, softcap, alibi)
FORMS = [(g, 256, -1, 0.0, False) for g in (9, 16, 17, 32, 33, 64)]
FORMS += [(g, d, -1, 0.0, False) for g in (16, 32, 64) for d in (64, 128)]
FORMS += [(16, 256, 700, 0.0, False), (20, 256, -1, 30.0, False), (64, 256, -1, 0.0, True),
          (32, 256, 1000, 0.0, True), (48, 256, 50, 20.0, False), (64, 128, 900, 30.0, False),
          (10, 64, 333, 0.0, True)]


@pytest.mark.parametrize("g,d,window,softcap,alibi", FORMS)
def test_forms(dev, g, d, window, softcap, alibi):
    lens, scale = [2311, 33, 0, 1500, 127], d ** -0.5
    c = filled(lens, 1, d, 16, True, seed=g + d)
    q = queries(len(lens), g, d, seed=g)
    sl = slopes_of(g) if alibi else None
    want, bound, _ = reference(c, q, lens, scale, window, softcap, sl)
    tensors, table = c.on(dev)
    kw = dict(scale=scale, window_left=window, softcap=softcap,
              alibi_slopes=None if sl is None else sl.to(dev))
    for S, most in ((1, None), (5, None), (0, 300), (0, 4000)):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S,
                                 max_kv_len=most, **kw)
        attn.check_device_status()
        close(o, lse, want, bound, f"g={g} d={d} S={S} for {most}")
    assert_cache(tensors, c.ref(), c, "only read")


@pytest.mark.parametrize("g", [9, 24, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append(dev, g, d):
    lens, n_kv = [700, 0, 63], 2
    c = filled(lens, n_kv, d, 24, True, seed=g + d, room=[n + 1 for n in lens])
    q = queries(3, g * n_kv, d, seed=g)
    new = [rows(n_kv, 3, d, s, spread=1.5).permute(1, 0, 2).contiguous() for s in (5, 6)]
    tensors, table = c.on(dev)
    want = c.ref()
    C.write(want, c.geo, new[0].double().numpy(), new[1].double().numpy(), [0, 1, 2, 3], lens)
    after = c.on(dev)[0]
    c.set_from(want)
    ref, bound, _ = reference(c, q, [n + 1 for n in lens], d ** -0.5)
    for S, most, t in ((3, None, tensors), (0, 2999, after)):
        o, lse = attn.decode_append_fp8(q.to(dev), new[0].to(dev), new[1].to(dev), *t,
                                        i32(lens, dev), table, num_splits=S, max_kv_len=most)
        attn.check_device_status()
        close(o, lse, ref, bound, f"append g={g} d={d} S={S}")
        assert_cache(t, want, c, "append")


@pytest.mark.parametrize("g,d", [(4, 256), (16, 64), (16, 256), (32, 128), (64, 256)])
def test_long_cache(dev, g, d):
    """20000 tokens in one split and in the library's division.  The norm of O's
    error: 2e-5 is 160 fp32 steps; sums that the tensor core truncated over all
    tokens were 3e-5 too small."""
    n = 20000
    c = filled([n], 1, d, 64, True, seed=n, spread=0.5)
    q = queries(1, g, d, 1)
    kc, vc = C.values(c.ref(), c.geo, [n])
    want = oracle.decode(q, kc, vc, None, [n], d ** -0.5, 0)
    tensors, table = c.on(dev)
    for S in (1, 0):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32([n], dev), table, num_splits=S)
        attn.check_device_status()
        e = np.linalg.norm(o.double().cpu().numpy() - want[0]) / np.linalg.norm(want[0])
        assert e <= 2e-5, (S, e)
        assert np.abs(lse.double().cpu().numpy() - want[1]).max() <= 2e-5, S
