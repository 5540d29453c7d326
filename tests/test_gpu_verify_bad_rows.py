"""Verification of rows without weight: the next token is the last entry, as documented, and a row
whose entries are not numbers is flagged."""

import pytest

import exact_io_aware_order_gb300 as attn
from exact_io_aware_order_gb300._lib import status_codes
from test_gpu_verify_tree import Case

pytestmark = pytest.mark.gpu


def flagged():
    with pytest.raises(attn.AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V", [10, 9000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0, 2.0])
def test_rows_that_are_not_numbers(dev, bad, V, drafts):
    """The row that the next token would be drawn from holds nothing but what counts as 0: its last
    entry, flagged.  A row of zeros gives that too, without a flag; so do bad rows that are not
    reached, and ones with weight elsewhere."""
    c = Case([3, 2, 4], V, drafts, seed=2, chain=True)
    c.u[:] = 1 - 2.0 ** -24
    c.p[3:5] = c.p[3:5].clamp(max=0) * 0                      # sequence 1: zeros
    c.p[6:9] = bad                                            # sequence 2: nodes that are not reached
    if drafts:
        c.q[5, c.tokens[6]] = 1.0
    c.p[5, c.tokens[6]] = 0.0
    attn.check_device_status()
    n, _, token = (x.tolist() for x in attn.verify_tree(*c.args(dev)))
    assert n[2] == 0 and token[1] == V - 1
    attn.check_device_status()
    c.p[2, V // 2:] = bad                                     # sequence 0's last node: half of it
    attn.verify_tree(*c.args(dev))
    attn.check_device_status()
    c.p[0] = bad
    c.p[0, 0] = 0.0
    n, path, token = (x.tolist() for x in attn.verify_tree(*c.args(dev)))
    assert n[0] == 0 and path[0] == [0] + [-1] * 63 and token[0] == V - 1
    flagged()
    c.tokens[1] = 0                                           # (refused, its weight is 0)
    c.p[0, V - 1] = 0.5                                       # some weight: drawn, without a flag
    token = attn.verify_tree(*c.args(dev))[2].tolist()
    assert token[0] == V - 1
    attn.check_device_status()
