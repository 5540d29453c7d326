"""Long caches with one row tile an item, where 226 KB hold an odd number of key and value tiles: a
tile that were overwritten before its products are through would show in some run of many."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from test_gpu_decode_tree import BF16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", [dict(), dict(softcap=50.0), dict(alibi=True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,n_q,n_kv,nodes", [(128, 8, 8, 32), (128, 28, 4, 6), (64, 16, 8, 64), (256, 8, 4, 20)])
def test_many_runs(dev, d, n_q, n_kv, nodes, dtype, variant):
    c = Case(dev, [12000, 5000], [nodes, 3], n_q, n_kv, d, 16, True, "tree", seed=1, **variant)
    c.check(*c.run(dtype))
    a = {**c.args(), "out_dtype": dtype}
    want = attn.decode_tree(**a)
    real = c.cu[-1]
    for _ in range(150):
        o, lse = attn.decode_tree(**a)
        assert torch.equal(o[:real], want[0][:real]) and torch.equal(lse[:real], want[1][:real])
    attn.check_device_status()
