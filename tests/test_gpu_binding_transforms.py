"""The 8-bit cache's calls inside torch's function transforms: a Python
exception, as from the framework's other calls, and the process lives on."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from cache_fp8_util import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["decode", "append", "write", "read", "scales", "bf16"])
@pytest.mark.parametrize("transform", [torch.vmap, torch.func.grad])
def test_transformed_tensors_raise(dev, op, transform):
    c = Cache(2, 2, 64, [40, 9], 16, True, seed=5)
    (k, v, ks, vs), table = c.on(dev)
    ks.fill_(1.0), vs.fill_(1.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    lens = i32([30, 8])
    q, new = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device=dev) for h in (4, 2))
    out = torch.empty(2, 40, 64, dtype=torch.bfloat16, device=dev)
    calls = {
        "decode": (lambda x: attn.decode_fp8(x, k, v, ks, vs, lens, table), q),
        "append": (lambda x: attn.decode_append_fp8(q, x, x, k, v, ks, vs, lens, table), new),
        "write": (lambda x: attn.cache_write_fp8(x, x, k, v, ks, vs, lens, None, table), new),
        "read": (lambda x: attn.cache_read_fp8(k, v, x, vs, i32([0, 30, 38]), 40, table), ks),
        "scales": (lambda x: attn.decode_fp8(q, k, v, x, vs, lens, table), ks),
        "bf16": (lambda x: attn.decode_splitkv(x, out[:, :, None], out[:, :, None], lens), q),
    }
    call, x = calls[op]
    many = x[None].repeat(3, *[1] * x.dim()) if transform is torch.vmap else x
    with pytest.raises(RuntimeError):
        transform(lambda t: (call(t), t.float().sum())[1])(many)
    o, _ = attn.decode_fp8(q, k, v, ks, vs, lens, table)
    attn.check_device_status()
    assert o.shape == q.shape
