"""Every call that takes a block table refuses one without columns."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [None, 64])
def test_table_without_columns(dev, most):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    none, lens, cu = torch.empty(2, 0, dtype=torch.int32, device=dev), i32(0, 0), i32(0, 1, 2)
    q, new = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device=dev) for h in (4, 2))
    c16 = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    c8, s = c16.to(torch.uint8), torch.ones(4, 2, device=dev)
    kw = dict(block_table=none, max_kv_len=most)
    for call in (lambda: attn.decode(q, c16, c16, lens, **kw),
                 lambda: attn.decode_splitkv(q, c16, c16, lens, num_splits=2, **kw),
                 lambda: attn.decode_append(q, new, new, c16, c16, lens, **kw),
                 lambda: attn.decode_noalloc(q, c16, c16, lens, **kw),
                 lambda: attn.decode_fp8(q, c8, c8, s, s, lens, **kw),
                 lambda: attn.decode_fp8_splitkv(q, c8, c8, s, s, lens, num_splits=2, **kw),
                 lambda: attn.decode_append_fp8(q, new, new, c8, c8, s, s, lens, **kw),
                 lambda: attn.cache_write_fp8(new, new, c8, c8, s, s, lens, None, none),
                 lambda: attn.cache_read_fp8(c8, c8, s, s, cu, 2, none)):
        with pytest.raises(ValueError, match="column"):
            call()
    attn.check_device_status()
