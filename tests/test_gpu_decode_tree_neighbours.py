"""A row of the tree attention depends on its own sequence alone, bit for bit: not on what ran
before the call, on other sequences' queries (lengths being equal), or on keys that no node sees.

Rows of a 128-row product that belong to no node (128 is no multiple of the query heads of a kv
head, or a sequence has fewer nodes) and masked columns hold whatever was there; what is left
there here is large, so that any part it takes shows: the rows beside it would raise the
reference of their exponentials, or take the other form of tanh."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from test_gpu_decode_tree import BF16, F32, Case

pytestmark = pytest.mark.gpu


def leave(dev, d, size):
    """A call over all of the GPU whose queries, all 128 rows of each tile, are this large."""
    c = Case(dev, [20000], [32], 16, 2, d, 16, True, "tree", seed=1, junk=False)
    c.q = (c.q.float() * size).to(BF16)
    c.run(BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [3, 5, 7])
def test_what_ran_before(dev, g, d, softcap, dtype):
    c = Case(dev, [20000, 3000, 300], [40, 64, 25], 2 * g, 2, d, 16, True, "tree", seed=2, softcap=softcap)
    leave(dev, d, 0.0)
    first = c.run(dtype)
    c.check(*first)
    for size in (100.0, 1.0, 1000.0):
        leave(dev, d, size)
        again = c.run(dtype)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    attn.check_device_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("variant", [dict(), dict(softcap=50.0), dict(alibi=True), dict(window=700)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_other_sequences_queries(dev, d, variant, dtype):
    c = Case(dev, [1500, 6000, 800], [9, 30, 21], 8, 2, d, 16, True, "tree", seed=3, **variant)
    was, (o, lse) = c.q.clone(), c.run(dtype)
    c.check(o, lse)
    for b in range(3):
        mine = slice(c.cu[b], c.cu[b] + c.nodes[b])
        for size in (0.0, 100.0):
            c.q = (was.float() * size).to(BF16)
            c.q[mine] = was[mine]
            again = c.run(dtype)
            assert torch.equal(o[mine], again[0][mine]) and torch.equal(lse[mine], again[1][mine])
    attn.check_device_status()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("variant", [dict(), dict(softcap=50.0), dict(alibi=True)])
def test_keys_that_no_node_sees(dev, variant, d):
    c = Case(dev, [1500, 70], [40, 33], 8, 2, d, 16, True, "any", seed=4, **variant)
    hidden = [3, 17, 32]
    words = [w & ~sum(1 << j for j in hidden) for ws in c.words for w in ws]
    c.words = [words[:40], words[40:]]
    c.mask[:73] = words
    rows = torch.cat([c.rows(b, n + 40)[n:][hidden] for b, n in enumerate(c.lens)])
    o, lse = c.run(F32)
    c.check(o, lse)
    for fill in (0.0, 1000.0, float("inf"), float("nan")):
        c.kc.view(-1, 2, d)[rows] = fill
        again = c.run(F32)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    attn.check_device_status()
