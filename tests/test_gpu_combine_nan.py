"""A split whose partial is NaN makes its own row's result NaN: it is not
taken for an empty split, and it reaches no other row."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,D,at", [(1, 128, 0), (3, 64, 2), (148, 128, 77), (1024, 256, 1023)])
@pytest.mark.parametrize("others_empty", [False, True])
def test_nan_split(dev, S, D, at, others_empty):
    gen = torch.Generator().manual_seed(S)
    op, lp = torch.randn(S, 2, 3, D, generator=gen), torch.randn(S, 2, 3, generator=gen)
    if others_empty:
        lp[:, 1, 2], op[:, 1, 2] = -float("inf"), 0.0
    want, lwant = attn.combine(op.to(dev), lp.to(dev))
    op[at, 1, 2], lp[at, 1, 2] = float("nan"), float("nan")
    o, lse = attn.combine(op.to(dev), lp.to(dev))
    attn.check_device_status()
    assert bool(torch.isnan(o[1, 2]).all()) and bool(torch.isnan(lse[1, 2]))
    rest = torch.ones(2, 3, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.equal(o[rest], want[rest]) and torch.equal(lse[rest], lwant[rest])
