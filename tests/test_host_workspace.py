"""attn_decode_fp8_workspace_bytes is 0 for what attn_decode_fp8 refuses: a
caller that asks first sets no memory aside for it (the size of 1000 splits
of a batch of 70000 would be 37 TB)."""

import pytest

from exact_io_aware_order_gb300 import _lib, build

GOOD = dict(S=4, B=2, n_q=32, n_kv=8, d=128, most=5000, window=-1)


@pytest.fixture(scope="module")
def size():
    build.build()
    f = _lib.lib().attn_decode_fp8_workspace_bytes

    def call(**kw):
        a = dict(GOOD, **kw)
        return f(a["S"], a["B"], a["n_q"], a["n_kv"], a["d"], a["most"], a["window"])

    return call


@pytest.mark.parametrize("kw", [dict(S=-1), dict(S=1025), dict(S=1000, B=70000), dict(B=0),
                                dict(n_kv=0), dict(n_kv=70000, n_q=140000), dict(n_q=7),
                                dict(n_q=33), dict(n_q=8 * 65), dict(d=0), dict(d=96),
                                dict(d=1 << 30), dict(most=-1), dict(most=(1 << 30) + 1),
                                dict(window=-2)])
def test_nothing_for_what_is_refused(size, kw):
    assert size(**kw) == 0


def test_what_is_not(size):
    rows = 4 * 2 * 32
    assert size() == rows * 128 * 4 + rows * 4
    assert size(S=1) == 0
    assert size(window=0) == size(most=0) == size(most=1 << 30) == size()
    assert size(S=1024, B=65535, n_q=64, n_kv=1, d=256) > 1 << 40
