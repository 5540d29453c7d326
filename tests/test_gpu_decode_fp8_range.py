"""Decode over an 8-bit cache whose V scales lie as far apart as they may, 2^-60
and 2^60: the sum of the weights has to follow, whichever comes first."""

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
from test_gpu_decode_fp8 import close, filled, i32, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q", [2, 8, 24, 64])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("large_at", ["first", "middle", "last"])
def test_many_small_values_and_a_few_large_ones(dev, n_q, d, large_at):
    """One block of 16 tokens has the scale 2^60 and scores 8 octaves above the
    others', 2^-60: 16 weights of 1 against 1184 of 2^-8.3, so that the small
    values' tokens carry a fifth of the sum."""
    n, bs = 1200, 16
    c = filled([n], 2, d, bs, True, seed=n_q)
    c.k.zero_()
    c.ks.fill_(1.0)
    c.vs.fill_(2.0 ** -60)
    big = int(c.table[0, {"first": 0, "middle": 40, "last": n // bs - 1}[large_at]])
    c.k[big, :, :, 0] = 0x38                               # 1.0
    c.vs[big] = 2.0 ** 60
    q = torch.zeros(1, n_q, d)
    q[0, :, 0] = 5.75
    q = q.to(torch.bfloat16)
    want, bound, _ = reference(c, q, [n], 1.0)
    assert (np.abs(want[1] - (5.75 + np.log(16 + 1184 * np.exp(-5.75)))) < 1e-9).all()
    tensors, table = c.on(dev)
    for S in (1, 3, 0):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32([n], dev), table, num_splits=S,
                                 max_kv_len=3000, scale=1.0)
        attn.check_device_status()
        # V's codes times 2^60: O's bound is relative to those.
        close(o, lse, want, bound, f"{large_at} S={S}")
