"""A key/value cache held in 8 bits: the float64 reference of its write, its
read and the values that decode attends to.

TEST INFRASTRUCTURE ONLY.  The test-suite is the only caller; the CUDA library
never routes through this file and this file imports nothing from the library.

The explainer page "FlashAttention for inference: tiled prefill and split-KV
decoding" (pofe.ai) has no 8-bit cache; the reading taken here is that of the
C header: e4m3 codes, and for each block of ``block_size`` tokens and kv head
one scale 2^k, k the smallest integer in [-60, 60] with amax <= 448 * 2^k over
the finite values written to the block.  A block that is continued keeps the
larger of its scale and the new rows' one; if its scale grows, the codes that
are already there become e4m3(code * old / new).

A cache is a dict: ``k``, ``v`` codes as float64 e4m3 values (rows, n_kv, d),
``ks``, ``vs`` scales (blocks, n_kv); rows and blocks are flat, and
:func:`place` finds a position's row and block for paged and contiguous caches.
"""

from __future__ import annotations

import math

import numpy as np

from .attention_ref import _f64
from .fp8_ref import E4M3_MAX, round_e4m3

__all__ = ["SCALE_EXP", "decode_code", "encode_value", "block_scale", "Geometry", "write", "read",
           "values"]

SCALE_EXP = (-60, 60)


def decode_code(code) -> np.ndarray:
    """The value of each e4m3 code (uint8), by the format's definition: sign,
    4 exponent bits (bias 7), 3 mantissa bits; exponent 0 is subnormal, 0x7f
    and 0xff are NaN."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def encode_value(x) -> np.ndarray:
    """e4m3 of each value as a float64: nearest, ties to even; beyond 448 (and
    infinities) saturate, NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.where(np.isnan(x), 0.0, np.clip(x, -1e4, 1e4))
    return np.where(np.isnan(x), np.nan, round_e4m3(fin))


def block_scale(amax: float) -> float:
    """2^k, k the smallest integer in SCALE_EXP with amax <= 448 * 2^k."""
    k = SCALE_EXP[0]
    while k < SCALE_EXP[1] and amax > E4M3_MAX * math.ldexp(1.0, k):
        k += 1
    return math.ldexp(1.0, k)


class Geometry:
    """Where position t of sequence s lies: paged (a block table) or
    contiguous (max_kv_len rows a sequence)."""

    def __init__(self, block_size, block_table=None, max_kv_len=0):
        self.bs = int(block_size)
        self.table = None if block_table is None else np.asarray(block_table).astype(np.int64)
        self.L = int(max_kv_len)

    def row(self, s, t):
        if self.table is not None:
            return int(self.table[s, t // self.bs]) * self.bs + t % self.bs
        return s * self.L + t

    def block(self, s, t):
        if self.table is not None:
            return int(self.table[s, t // self.bs])
        return s * -(-self.L // self.bs) + t // self.bs


def write(cache: dict, geo: Geometry, k, v, cu_seqlens, kv_lens) -> None:
    """Writes rows [cu[s], cu[s+1]) of k, v (total, n_kv, d) behind the
    kv_lens[s] tokens of sequence s, in place."""
    for name, x in (("k", _f64(k)), ("v", _f64(v))):
        codes, scales = cache[name], cache[name + "s"]
        for s, start in enumerate(int(n) for n in kv_lens):
            a, b = int(cu_seqlens[s]), int(cu_seqlens[s + 1])
            pos, end = start, start + b - a
            while pos < end:
                first = pos // geo.bs * geo.bs
                stop = min(end, first + geo.bs)
                blk = geo.block(s, pos)
                rows = [geo.row(s, t) for t in range(pos, stop)]
                new = x[a + pos - start:a + stop - start]
                for h in range(x.shape[1]):
                    y = new[:, h]
                    fin = np.abs(y[np.isfinite(y)])
                    scale = block_scale(float(fin.max()) if fin.size else 0.0)
                    if pos > first:
                        was = float(scales[blk, h])
                        scale = max(scale, was)
                        if scale > was:
                            old = [geo.row(s, t) for t in range(first, pos)]
                            codes[old, h] = encode_value(codes[old, h] * (was / scale))
                    scales[blk, h] = scale
                    codes[rows, h] = encode_value(y / scale)
                pos = stop


def read(cache: dict, geo: Geometry, cu_seqlens, starts, total: int):
    """(K, V) (n_kv, total, d): row cu[s] + i is position starts[s] + i of
    sequence s; NaN elsewhere."""
    out = []
    for name in ("k", "v"):
        codes, scales = cache[name], cache[name + "s"]
        y = np.full((codes.shape[1], total, codes.shape[2]), np.nan)
        for s in range(len(cu_seqlens) - 1):
            for i in range(int(cu_seqlens[s + 1]) - int(cu_seqlens[s])):
                t = int(starts[s]) + i
                y[:, int(cu_seqlens[s]) + i] = (codes[geo.row(s, t)]
                                                * scales[geo.block(s, t)][:, None])
        out.append(y)
    return tuple(out)


def values(cache: dict, geo: Geometry, kv_lens):
    """The caches' values as a contiguous float64 cache (B, max len, n_kv, d)
    for the attention reference, NaN where no token is."""
    lens = [int(n) for n in kv_lens]
    out = []
    for name in ("k", "v"):
        codes, scales = cache[name], cache[name + "s"]
        y = np.full((len(lens), max(1, max(lens)), *codes.shape[1:]), np.nan)
        for s, n in enumerate(lens):
            if n:
                rows = [geo.row(s, t) for t in range(n)]
                blks = [geo.block(s, t) for t in range(n)]
                y[s, :n] = codes[rows] * scales[blks][:, :, None]
        out.append(y)
    return tuple(out)
