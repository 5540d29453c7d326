"""Whole numbers that do not fit the C entry points' 32 bits are refused and
not taken modulo 2^32: a block size taken so would index the scales by other
blocks than the ones whose count was checked."""

import pytest
import torch

from exact_io_aware_order_gb300 import api


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 64 + 1])
def test_beyond_32_bits(x):
    with pytest.raises(ValueError, match="32 bits"):
        api._int32(x, "x")


def test_within_32_bits():
    for x in (0, -1, 2 ** 31 - 1, -2 ** 31):
        assert api._int32(x, "x") == x


def test_block_size_of_a_contiguous_cache():
    codes, one = torch.zeros(1, 100, 2, 64, dtype=torch.uint8), torch.ones(1, 1, 2)
    check = lambda bs, s: api._cache_fp8(torch.device("cpu"), codes, codes, s, s, None, bs, 1)
    assert check(128, one)[1] == (128, 0, 0, 100)
    assert check(16, torch.ones(1, 7, 2))[1] == (16, 0, 0, 100)
    with pytest.raises(ValueError, match="32 bits"):     # one block, but 16 in 32 bits
        check(2 ** 32 + 16, one)


def test_other_numbers_are_no_whole_numbers():
    for x in (2.0, "3", None):
        with pytest.raises(TypeError):
            api._int32(x, "x")
