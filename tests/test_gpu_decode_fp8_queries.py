"""Decode over an 8-bit cache with queries that have channels far larger than
the rest, and keys that are as much smaller there (few such channels, or all but
a few: keys with a large channel): every channel counts alike in the scores,
so the small values of q have to be used as they are."""

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
from oracle import cache_fp8_ref as C
from cache_fp8_util import code_bytes
from test_gpu_decode_fp8 import close, filled, i32, queries, reference

pytestmark = pytest.mark.gpu

AT = 40                                                    # the large channel


def uneven(n_q, n_kv, d, lens, p, rows, paged=True, at=(AT,)):
    """A cache whose keys are 2^-p in the channels `at`, and queries 2^p there in
    the rows given (the others 0 there)."""
    c = filled(lens, n_kv, d, 16, paged, seed=n_q + p)
    at = list(at)
    kv = C.decode_code(c.k.numpy())
    kv[..., at] *= 2.0 ** -p
    c.k.copy_(code_bytes(C.encode_value(kv)).view(c.k.shape))
    q = queries(len(lens), n_q, d, p)
    for h in range(n_q):
        q[:, h, at] = q[:, h, at] * 2.0 ** p if h in rows else 0.0
    return c, q


@pytest.mark.parametrize("p", [4, 7, 12, 20, 30])
@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 64), (28, 4, 128), (6, 2, 256), (9, 1, 64),
                                        (24, 1, 128), (64, 1, 128), (64, 1, 64), (16, 1, 256),
                                        (40, 1, 256)])
def test_one_large_channel(dev, n_q, n_kv, d, p):
    """Scores of deviation 4 or so.  Besides the worst case of every rounding
    (close), the norm of O's error: one rounding of 2^-23 for each step of 32
    products and 8 more in a score of which the products' magnitudes sum to a,
    twice that in a weight (its own and the sum's) -> 2 (d / 32 + 8) 2^-23 a.
    Two 4-bit terms of q alone are off by some 2^(p - 25) in every product."""
    lens = [700, 33]
    c, q = uneven(n_q, n_kv, d, lens, p, range(n_q))
    scale = 4 * d ** -0.5
    want, bound, (kc, _) = reference(c, q, lens, scale)
    tensors, table = c.on(dev)
    for S in (1, 3, 0):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S,
                                 max_kv_len=3000, scale=scale)
        attn.check_device_status()
        close(o, lse, want, bound, f"p={p} S={S}")
        for b, n in enumerate(lens):
            k = np.abs(kc[b, :n]).repeat(n_q // n_kv, axis=1)
            a = scale * np.einsum("hd,nhd->nh", np.abs(q[b].double().numpy()), k).max()
            e = np.linalg.norm(o[b].double().cpu().numpy() - want[0][b]) / np.linalg.norm(want[0][b])
            assert e <= 2 * (d / 32 + 8) * 2.0 ** -23 * a, (p, S, b, e, a)


@pytest.mark.parametrize("p", [9, 12])
@pytest.mark.parametrize("n_q,n_kv,d,few", [(8, 2, 64, 1), (8, 2, 64, 8), (28, 4, 128, 1),
                                            (28, 4, 128, 6), (6, 2, 256, 8), (24, 1, 128, 2),
                                            (64, 1, 64, 3), (16, 1, 256, 8), (40, 1, 256, 1)])
def test_all_channels_but_a_few_large(dev, n_q, n_kv, d, few, p):
    """The other way round, as with keys that have `few` large channels.  Norm of
    O's error as above, and 2^-18 of a base 2 logarithm in every score: twice 2^-18 log
    2 < 2^-17.5 in the weights.  (A norm over the head's row of d values.)"""
    lens = [700, 33]
    c, q = uneven(n_q, n_kv, d, lens, p, range(n_q), at=[i for i in range(d) if i % d >= few])
    scale = 4 * d ** -0.5
    want, bound, (kc, _) = reference(c, q, lens, scale)
    tensors, table = c.on(dev)
    for S in (1, 0):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S,
                                 max_kv_len=3000, scale=scale)
        attn.check_device_status()
        close(o, lse, want, bound, f"p={p} S={S}")
        for b, n in enumerate(lens):
            k = np.abs(kc[b, :n]).repeat(n_q // n_kv, axis=1)
            a = scale * np.einsum("hd,nhd->nh", np.abs(q[b].double().numpy()), k).max()
            e = np.linalg.norm(o[b].double().cpu().numpy() - want[0][b], axis=1)
            e = (e / np.linalg.norm(want[0][b], axis=1)).max()
            assert e <= 2 * (d / 32 + 8) * 2.0 ** -23 * a + 2.0 ** -17.5, (p, S, b, e, a)


@pytest.mark.parametrize("n_q,d", [(8, 64), (8, 128), (5, 256), (20, 128), (40, 256)])
def test_one_row_of_many(dev, n_q, d):
    """A row with a large channel beside rows without one."""
    lens = [300]
    c, q = uneven(n_q, 1, d, lens, 14, [3])
    scale = 4 * d ** -0.5
    want, bound, _ = reference(c, q, lens, scale)
    tensors, table = c.on(dev)
    for S in (1, 0):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S,
                                 max_kv_len=3000, scale=scale)
        attn.check_device_status()
        close(o, lse, want, bound, f"S={S}")


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (40, 1, 256)])
def test_the_next_segment_has_other_queries(dev, n_q, n_kv, d):
    """Equal shares take a block over several sequences: some with large
    channels, some without."""
    lens = [int(n) for n in np.random.default_rng(d).integers(10, 2500, 36)]
    c, q = uneven(n_q, n_kv, d, lens, 16, range(n_q))
    q[::2, :, AT] = 0.0
    scale = 4 * d ** -0.5
    want, bound, _ = reference(c, q, lens, scale)
    tensors, table = c.on(dev)
    o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, max_kv_len=8192, scale=scale)
    attn.check_device_status()
    close(o, lse, want, bound, "segments")
