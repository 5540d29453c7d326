"""The 8-bit cache's calls refuse whole numbers beyond 32 bits."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn

pytestmark = pytest.mark.gpu


def test_beyond_32_bits(dev):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    lens, cu, table = i32(20, 3), i32(0, 20, 23), i32(0, 1, 2, 3).view(2, 2)
    q, new = (torch.zeros(2, h, 64, dtype=torch.bfloat16, device=dev) for h in (4, 2))
    c = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device=dev)
    s, flat = torch.ones(4, 2, device=dev), c.view(2, 32, 2, 64)
    one = torch.ones(2, 1, 2, device=dev)
    far = 2 ** 32
    paged = (c, c, s, s, lens, table)
    for call in (lambda: attn.decode_fp8(q, *paged, window_left=far + 5),
                 lambda: attn.decode_fp8(q, *paged, num_splits=far + 2),
                 lambda: attn.decode_fp8(q, *paged, max_kv_len=far + 32),
                 lambda: attn.decode_fp8(q, flat, flat, one, one, lens, block_size=far + 16),
                 lambda: attn.decode_fp8_splitkv(q, *paged, num_splits=far + 2),
                 lambda: attn.decode_fp8_splitkv(q, *paged, num_splits=2, window_left=far),
                 lambda: attn.decode_append_fp8(q, new, new, *paged, window_left=-far),
                 lambda: attn.cache_write_fp8(new, new, flat, flat, one, one, lens,
                                              block_size=far + 16),
                 lambda: attn.cache_read_fp8(c, c, s, s, cu, far + 23, table)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    attn.check_device_status()
