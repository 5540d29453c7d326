"""Decode steps with drafted tokens, one after another as a user makes them: the nodes' keys
and values into the cache, attention of the trees, verification, the accepted path's keys and
values behind the cached tokens, lengths advanced on the device; each result against its
64-bit form, and steps captured into a graph against steps that are not."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import F64, assert_bf16, tree, tree_attention, turned, words_of
from test_gpu_verify_tree import reference

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
N_Q, N_KV, D, V, BLOCK = 6, 2, 128, 260, 16


class Step:
    """What a step is given: trees, their tokens' projections and probabilities."""

    def __init__(self, nodes, seed):
        g = torch.Generator().manual_seed(seed)
        total = sum(nodes)
        self.nodes, self.cu = nodes, [sum(nodes[:i]) for i in range(len(nodes) + 1)]
        self.parents = [tree(n, seed + 10 * b) for b, n in enumerate(nodes)]
        self.qkv = torch.randn(total, N_Q + 2 * N_KV, D, generator=g).to(BF16)
        logits = torch.randn(total, V, generator=g)
        self.p = torch.softmax(logits, 1)
        self.d = torch.softmax(logits + 0.1 * torch.randn(total, V, generator=g), 1)
        up = [self.cu[b] + max(j, 0) for b, t in enumerate(self.parents) for j in t]
        self.tokens = torch.multinomial(self.d[up], 1, generator=g)[:, 0].to(I32)
        self.u, self.u_last = torch.rand(total, generator=g), torch.rand(len(nodes), generator=g)

    def tensors(self):
        return [self.qkv, self.p, self.d, self.tokens, torch.tensor(sum(self.parents, []), dtype=I32),
                torch.tensor(self.cu, dtype=I32), self.u, self.u_last]


def rows_of_paths(path, num, cu, total):
    """The accepted paths' rows, packed, and their cu_seqlens; nothing waits for the device."""
    n = num + 1
    new = torch.cat([torch.zeros_like(cu[:1]), n.cumsum(0).to(I32)])
    i = torch.arange(path.shape[1], device=path.device)
    real = i < n[:, None]
    to = torch.where(real, new[:-1, None] + i, total).long()
    rows = torch.zeros(total + 1, dtype=torch.int64, device=path.device)
    rows.scatter_(0, to.flatten(), torch.where(real, cu[:-1, None] + path, 0).long().flatten())
    return rows[:total], new


def step(x, kc, vc, kv, table, f):
    """One step; kv is advanced."""
    qkv, p, d, tokens, parents, cu, u, u_last = x
    q, k, v = (t.transpose(0, 1) for t in qkv.split([N_Q, N_KV, N_KV], dim=1))
    mask = attn.tree_mask(parents, cu)
    deep = sum(((mask >> j) & 1) for j in range(64)).to(I32) - 1
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(len(parents), device=cu.device, dtype=I32),
                             right=True)
    q = attn.cache_append(k, v, kc, vc, kv, cu, table, f, positions=kv[seq] + deep, q=q).transpose(0, 1)
    o, lse = attn.decode_tree(q.contiguous(), kc, vc, kv, cu, mask, table)
    num, path, token = attn.verify_tree(p, tokens, parents, cu, u, u_last, d)
    rows, new = rows_of_paths(path, num, cu, len(parents))
    attn.cache_append(k[:, rows], v[:, rows], kc, vc, kv, new, table, f)
    kv += num + 1
    return q, o, lse, num, path, token


def state(dev, lens, room, seed=0):
    g = torch.Generator().manual_seed(seed)
    per = -(-room // BLOCK)
    table = torch.randperm(per * len(lens), generator=g).to(I32).view(len(lens), per)
    shape = (per * len(lens), BLOCK, N_KV, D)
    kc, vc = torch.randn(*shape, generator=g).to(BF16), torch.randn(*shape, generator=g).to(BF16)
    return [t.to(dev) for t in (kc, vc, torch.tensor(lens, dtype=I32), table)]


def contents(kc, vc, table, b, n):
    j = torch.arange(n)
    r = table[b].cpu().long()[j // BLOCK] * BLOCK + j % BLOCK
    return kc.cpu().view(-1, N_KV, D)[r], vc.cpu().view(-1, N_KV, D)[r]


def test_steps_in_a_row(dev):
    f = attn.rope_inv_freq(64, 10000.0, device=dev)
    lens = [0, 37, 500]
    kc, vc, kv, table = state(dev, lens, 900)
    held = [contents(kc, vc, table, b, n) for b, n in enumerate(lens)]   # what has to be there
    slack = [torch.zeros(n, N_KV, D, dtype=F64) for n in lens]           # and how exactly
    held = [[k.to(F64), v] for k, v in held]
    accepted = 0
    for i, nodes in enumerate([[12, 1, 30], [64, 7, 3], [2, 64, 20], [9, 9, 9]]):
        s = Step(nodes, 100 + i)
        was = kv.tolist()
        kc_was, vc_was = kc.clone(), vc.clone()
        x = [t.to(dev) for t in s.tensors()]
        q, o, lse, num, path, token = step(x, kc, vc, kv, table, f)
        # The tree's own keys and values, as attention saw them, from a cache of their own.
        q1, k1, v1 = (t.transpose(0, 1) for t in x[0].split([N_Q, N_KV, N_KV], dim=1))
        deep = [bin(w).count("1") - 1 for t in s.parents for w in words_of(t)]
        pos = [was[b] + deep[s.cu[b] + j] for b, n in enumerate(nodes) for j in range(n)]
        attn.cache_append(k1, v1, kc_was, vc_was, torch.tensor(was, dtype=I32, device=dev), x[5], table, f,
                          positions=torch.tensor(pos, dtype=I32, device=dev))
        pos = torch.tensor(pos)
        want, err = turned(s.qkv[:, :N_Q].transpose(0, 1), pos, f.cpu())
        assert_bf16(q.transpose(0, 1), want, err, "queries")
        kr, kerr = (t.transpose(0, 1) for t in turned(s.qkv[:, N_Q:N_Q + N_KV].transpose(0, 1), pos, f.cpu()))
        for b, n in enumerate(nodes):
            sl = slice(s.cu[b], s.cu[b] + n)
            K, W = contents(kc_was, vc_was, table, b, was[b] + n)
            assert_bf16(K, torch.cat([held[b][0], kr[sl]]), torch.cat([slack[b], kerr[sl]]), "keys")
            assert torch.equal(W, torch.cat([held[b][1], s.qkv[sl, N_Q + N_KV:]]))
            ro, rl, A, X, _ = tree_attention(q[sl].cpu(), K, W, was[b], words_of(s.parents[b]), D ** -0.5)
            # Scores: D / 16 additions good to 2^-22 of X, exponentials 2^-20; weights in three
            # bf16 parts, sums over 16 keys at a time 2^-23.
            e = D / 16 * X * 2.0 ** -22 + 2.0 ** -20
            tol = A * (2.0 ** -16 + 2 * e + (was[b] + n + 16) / 16 * 2.0 ** -23)
            assert bool(((o[sl].cpu().to(F64) - ro).abs() <= tol).all())
            assert bool(((lse[sl].cpu().to(F64) - rl).abs() <= 2 * e + 2.0 ** -21 * (1 + rl.abs())).all())
            n_acc, way, tok = reference(s.p[sl], s.d[sl], s.tokens[sl].tolist(), s.parents[b],
                                        s.u[sl], s.u_last[b])
            assert (int(num[b]), path[b].tolist(), int(token[b])) == (n_acc, way, tok)
            accepted += n_acc
            rows = [s.cu[b] + j for j in way[:n_acc + 1]]
            assert [int(pos[t]) for t in rows] == list(range(was[b], was[b] + n_acc + 1))
            held[b] = [torch.cat([held[b][0], kr[rows]]), torch.cat([held[b][1], s.qkv[rows, N_Q + N_KV:]])]
            slack[b] = torch.cat([slack[b], kerr[rows]])
            assert int(kv[b]) == was[b] + n_acc + 1
    assert accepted >= 6                                      # (the inputs reach it)
    for b, n in enumerate(kv.tolist()):
        K, W = contents(kc, vc, table, b, n)
        assert_bf16(K, held[b][0], slack[b], "keys in the end")
        assert torch.equal(W, held[b][1])
    attn.check_device_status()


def test_captured_steps(dev):
    f = attn.rope_inv_freq(128, 10000.0, device=dev)
    lens, nodes = [3, 700, 64, 0], [20, 5, 64, 1]
    steps = [Step(nodes, 200 + i) for i in range(4)]
    eager = state(dev, lens, 1100, seed=1)
    want = [[t.clone() for t in step([t.to(dev) for t in s.tensors()], *eager[:3], eager[3], f)] for s in steps]
    mine = state(dev, lens, 1100, seed=1)
    start = [t.clone() for t in mine]
    x = [t.to(dev) for t in steps[0].tensors()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, *mine[:3], mine[3], f)                       # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, *mine[:3], mine[3], f)
    for a, b in zip(mine, start):
        a.copy_(b)
    for s, w in zip(steps, want):
        for a, b in zip(x, s.tensors()):
            a.copy_(b)
        graph.replay()
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    for a, b in zip(mine, eager):
        assert torch.equal(a, b)
    attn.check_device_status()
