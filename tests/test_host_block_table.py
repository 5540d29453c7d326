"""A block table without columns is refused: its address is null, which the C
entry points take for a contiguous cache of max_kv_len rows a sequence."""

import pytest
import torch

from exact_io_aware_order_gb300 import api


def test_table_without_columns():
    assert torch.empty(2, 0, dtype=torch.int32).data_ptr() == 0
    with pytest.raises(ValueError, match="column"):
        api._columns(torch.empty(2, 0, dtype=torch.int32))
    assert api._columns(torch.empty(2, 3, dtype=torch.int32)) == 3


def test_fp8_cache_with_a_table_without_columns():
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=torch.uint8), torch.ones(4, 2)
    check = lambda table: api._cache_fp8(torch.device("cpu"), codes, codes, scales, scales, table,
                                         None, 2)
    with pytest.raises(ValueError, match="column"):
        check(torch.empty(2, 0, dtype=torch.int32))
    table = torch.zeros(2, 5, dtype=torch.int32)
    ptrs, geom = check(table)
    assert ptrs[4] == table.data_ptr() != 0 and geom == (16, 5, 4, 80)
