"""Pins of the 8-bit cache's reference (oracle/cache_fp8_ref.py): the codes
against torch's e4m3 type, the block scale against its definition, and the
write's and the read's bookkeeping on a case small enough to write out."""

import math

import numpy as np
import torch

from oracle import cache_fp8_ref as C


def test_codes_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    got = C.decode_code(codes)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).sum() == 2
    fin = ~np.isnan(want)
    assert np.array_equal(got[fin], want[fin])
    assert np.array_equal(np.signbit(got[fin]), np.signbit(want[fin]))
    assert np.array_equal(C.encode_value(got[fin]), got[fin])      # every value keeps its code


def test_encode_ties_and_limits():
    for x, want in {17.0: 16.0, 19.0: 20.0, 464.0: 448.0, 1e30: 448.0, -math.inf: -448.0,
                    2.0 ** -10: 0.0, 3 * 2.0 ** -10: 2.0 ** -8, 449.0: 448.0}.items():
        assert C.encode_value(np.array([x]))[0] == want, x
    assert np.isnan(C.encode_value(np.array([math.nan]))[0])


def test_block_scale():
    assert C.block_scale(0.0) == 2.0 ** -60 and C.block_scale(2.0 ** 127) == 2.0 ** 60
    for k in (-59, -3, 0, 7, 59):
        edge = 448.0 * math.ldexp(1.0, k)
        assert C.block_scale(edge) == math.ldexp(1.0, k)
        assert C.block_scale(edge * (1 + 2.0 ** -7)) == math.ldexp(1.0, k + 1)


def test_write_and_read_by_hand():
    """Blocks of 2 tokens, one head of width 1, table [1, 0]: tokens 1.0 and
    448.0 share block 1 at scale 1; then 3.0 opens block 0 at scale 2^-7 (3 <=
    448 * 2^-7 = 3.5) as code 384, and 8.0 makes it grow to 2^-5 (8 <= 14):
    codes 96 and 256."""
    cache = {n: np.full((4, 1, 1), 5.0) for n in ("k", "v")}
    cache.update({n + "s": np.full((2, 1), 99.0) for n in ("k", "v")})
    geo = C.Geometry(2, [[1, 0]])
    col = lambda *x: np.array(x).reshape(-1, 1, 1)
    C.write(cache, geo, col(1.0, 448.0), col(1.0, 448.0), [0, 2], [0])
    assert cache["k"].ravel().tolist() == [5.0, 5.0, 1.0, 448.0]
    assert cache["ks"].ravel().tolist() == [99.0, 1.0]
    C.write(cache, geo, col(3.0), col(3.0), [0, 1], [2])
    assert cache["k"].ravel().tolist() == [384.0, 5.0, 1.0, 448.0] and cache["ks"][0, 0] == 2 ** -7
    C.write(cache, geo, col(8.0), col(8.0), [0, 1], [3])
    assert cache["v"].ravel().tolist() == [96.0, 256.0, 1.0, 448.0] and cache["vs"][0, 0] == 2 ** -5
    k, v = C.read(cache, geo, [0, 3], [1], 4)
    assert k[0, :3, 0].tolist() == [448.0, 3.0, 8.0] and np.isnan(k[0, 3, 0])
    kc, _ = C.values(cache, geo, [4])
    assert kc.ravel().tolist() == [1.0, 448.0, 3.0, 8.0]
