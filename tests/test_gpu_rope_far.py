"""Angles of rotary positions at any position and frequency, against p * inv_freq reduced modulo
a turn in whole numbers."""

import math
from decimal import Decimal, getcontext
from fractions import Fraction

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import F64, assert_bf16

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def turn():
    """2 pi in 80 digits, by Machin's formula."""
    getcontext().prec = 90
    def arctan_of_one_over(n):
        x = Decimal(1) / n
        s, t, k = x, x, 1
        while abs(t) > Decimal(10) ** -88:
            t = -t / (n * n)
            k += 2
            s += t / k
        return s
    return Fraction(8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_positions_and_large_frequencies(dev, sign, interleaved):
    full = turn()
    f = torch.tensor([1.0, 0.99, 3.25, -1e3, 12345.678, 1e6, 2 * math.pi, 2.0 ** 40 / 3,
                      -(2.0 ** 53), 1e-5, -0.3, 1e9 + 0.1, 2.0 ** 33 * math.pi, 77.7, 1e-12, -1e-30,
                      7.0, 5e5, -2e7, 0.0, 1 / 3, 100.0, 1e11, -9.75], dtype=F64) * sign
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1500000001, -1999999999, 10 ** 9, 2 ** 24 + 1, 1, -1, 0, 12345]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, len(pos), 64, generator=g).to(BF16)
    got = attn.rope(x.to(dev), None, f.to(dev), torch.tensor(pos, dtype=torch.int32, device=dev),
                    interleaved=interleaved)[0]
    cos, sin = torch.empty(len(pos), 24, dtype=F64), torch.empty(len(pos), 24, dtype=F64)
    for i, p in enumerate(pos):
        for j, w in enumerate(f.tolist()):
            a = Fraction(w) * p / full
            a = float((a - math.floor(a + Fraction(1, 2))) * full)   # within half a turn of 0
            cos[i, j], sin[i, j] = math.cos(a), math.sin(a)
    y, err = x.to(F64), torch.zeros(2, len(pos), 64, dtype=F64)
    i1, i2 = (slice(0, 48, 2), slice(1, 48, 2)) if interleaved else (slice(0, 24), slice(24, 48))
    x1, x2 = x[..., i1].to(F64), x[..., i2].to(F64)
    y[..., i1], y[..., i2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    # The angle within 2^-24 half turns (2e-7), sines and cosines within 2^-22, three roundings.
    err[..., i1] = err[..., i2] = (x1.abs() + x2.abs()) * 2.0 ** -20
    assert_bf16(got, y, err)
    attn.check_device_status()
