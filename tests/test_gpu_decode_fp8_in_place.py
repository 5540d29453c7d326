"""Decode steps whose query, new token, lengths and block table stay in the same
buffers and are changed there by other kernels right before each step (a
captured graph's way of working).  The decode of a small step reads them while
its write runs, so it has to see this step's, not the one's before."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from cache_fp8_util import Cache, rows
from test_gpu_decode_fp8 import i32, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n_kv,g,d", [(1, 1, 4, 128), (2, 4, 7, 64), (5, 2, 16, 256)])
@pytest.mark.parametrize("graph", [False, True])
def test_buffers_changed_in_place(dev, B, n_kv, g, d, graph):
    bs, steps = 4, 48
    c = Cache(B, n_kv, d, [steps] * B, bs, True, seed=B)
    apart, table = c.on(dev)
    joined = [t.clone() for t in apart]
    q = [queries(B, n_kv * g, d, s).to(dev) for s in range(steps)]
    new = [rows(n_kv, B, d, 100 + s).permute(1, 0, 2).contiguous().to(dev) for s in range(steps)]
    kw = dict(max_kv_len=3000)
    want = []
    for i in range(steps):
        lens = i32([i] * B, dev)
        attn.cache_write_fp8(new[i], new[i], *apart, lens, None, table)
        torch.cuda.synchronize()
        want.append(attn.decode_fp8(q[i], *apart, lens + 1, table, **kw))
        torch.cuda.synchronize()
    # A table that knows no block before its first token (0 stands there).
    qb, nb, lens = torch.empty_like(q[0]), torch.empty_like(new[0]), i32([-1] * B, dev)
    tb = torch.zeros_like(table)
    step = torch.zeros(1, dtype=torch.int64, device=dev)
    q_all, new_all = torch.stack(q), torch.stack(new)
    block = torch.arange(table.shape[1], device=dev)

    def one():
        qb.copy_(q_all.index_select(0, step)[0])
        nb.copy_(new_all.index_select(0, step)[0])
        tb.copy_(torch.where(block <= step // bs, table, 0))
        lens.add_(1)
        step.add_(1)
        return attn.decode_append_fp8(qb, nb, nb, *joined, lens, tb, **kw)

    got = []
    if graph:
        start = [t.clone() for t in joined]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one()
        torch.cuda.current_stream().wait_stream(side)
        lens.fill_(-1), step.zero_()
        for a, b in zip(joined, start):
            a.copy_(b)
        replayed = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replayed):
            out = one()
        for i in range(steps):
            replayed.replay()
            got.append([t.clone() for t in out])
    else:
        for i in range(steps):
            got.append(one())
    torch.cuda.synchronize()
    attn.check_device_status()
    for i in range(steps):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1]), i
    for a, b in zip(joined, apart):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
