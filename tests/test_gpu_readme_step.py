"""README's decode step with drafted tokens runs as it is printed, and gives what its calls are
documented to give."""

import os

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from conftest import ROOT
from drafts_util import F64, assert_bf16, tree, tree_attention, turned, words_of
from test_gpu_verify_tree import reference

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def printed_step():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    a = text.index("# a decode step with drafted tokens")
    return text[a:text.index("attn.check_device_status()", a)]


@pytest.mark.parametrize("n_q,n_kv,nodes,sliced", [(6, 2, [12, 1, 9], False), (22, 2, [12, 1, 9], True),
                                                   (8, 1, [64, 30], True), (4, 4, [7, 0, 5], True)])
def test_printed_step(dev, n_q, n_kv, nodes, sliced):
    """With as many nodes as heads too, where axes that are exchanged have the right sizes."""
    d, V, block = 128, 260, 16
    g = torch.Generator().manual_seed(n_q)
    total, B = sum(nodes), len(nodes)
    cu = [sum(nodes[:i]) for i in range(B + 1)]
    lens = [0, 37, 500][:B]
    trees = [tree(n, 10 * b + 1) if n else [] for b, n in enumerate(nodes)]
    qkv = torch.randn(total, n_q + 2 * n_kv, d, generator=g).to(BF16)
    logits = torch.randn(total, V, generator=g)
    p = torch.softmax(logits, 1)
    dp = torch.softmax(logits + 0.1 * torch.randn(total, V, generator=g), 1)
    up = [cu[b] + max(j, 0) for b, t in enumerate(trees) for j in t]
    tokens = torch.multinomial(dp[up], 1, generator=g)[:, 0].to(I32)
    u, u_last = torch.rand(total, generator=g), torch.rand(B, generator=g)
    per = 40
    table = torch.randperm(per * B, generator=g).to(I32).view(B, per)
    kc, vc = (torch.randn(per * B, block, n_kv, d, generator=g).to(BF16) for _ in range(2))
    f = attn.rope_inv_freq(d, device=dev)
    q, k, v = qkv.to(dev).split([n_q, n_kv, n_kv], dim=1)
    if not sliced:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    names = dict(torch=torch, attn=attn, parents=torch.tensor(sum(trees, []), dtype=I32, device=dev),
                 cu_nodes=torch.tensor(cu, dtype=I32, device=dev), q=q, k_new=k, v_new=v,
                 k_cache=kc.to(dev), v_cache=vc.to(dev), kv_lens=torch.tensor(lens, dtype=I32, device=dev),
                 block_table=table.to(dev), f=f, target_probs=p.to(dev), draft_tokens=tokens.to(dev),
                 u_accept=u.to(dev), u_sample=u_last.to(dev), draft_probs=dp.to(dev))
    exec(printed_step(), names)
    got_q, o, token = (names[x].cpu() for x in ("q", "o", "token"))
    n_new = names["kv_lens"].tolist()
    for b, n in enumerate(nodes):
        if n == 0:
            assert int(token[b]) == -1 and n_new[b] == lens[b]
            continue
        sl, words = slice(cu[b], cu[b] + n), words_of(trees[b])
        pos = torch.tensor([lens[b] + bin(w).count("1") - 1 for w in words])
        want, err = turned(qkv[sl, :n_q].transpose(0, 1), pos, f.cpu())
        assert_bf16(got_q[sl].transpose(0, 1), want, err, "queries")
        kr, kerr = turned(qkv[sl, n_q:n_q + n_kv].transpose(0, 1), pos, f.cpu())
        j = torch.arange(lens[b] + n)
        r = table[b].long()[j // block] * block + j % block
        K = torch.cat([kc.view(-1, n_kv, d)[r[:lens[b]]].to(F64), kr.transpose(0, 1)])
        W = torch.cat([vc.view(-1, n_kv, d)[r[:lens[b]]], qkv[sl, n_q + n_kv:]])
        ro, _, A, X, _ = tree_attention(got_q[sl], K, W, lens[b], words, d ** -0.5)
        # The nodes' keys were rounded to bf16: a score is off by 2^-8 of its sum of magnitudes X
        # (all else, as in the tests of decode_tree, by less than 2^-12 of it), a weight and the
        # sum of weights by e to that.
        tol = A * (torch.exp(torch.tensor(2 * X * (2.0 ** -8 + 2.0 ** -12))).item() - 1 + 2.0 ** -14)
        assert bool(((o[sl].to(F64) - ro).abs() <= tol).all())
        num, way, tok = reference(p[sl], dp[sl], tokens[sl].tolist(), trees[b], u[sl], u_last[b])
        assert int(token[b]) == tok and n_new[b] == lens[b] + num + 1
        rows = [cu[b] + x for x in way[:num + 1]]
        at = r[lens[b]:lens[b] + num + 1]
        assert_bf16(names["k_cache"].cpu().view(-1, n_kv, d)[at].transpose(0, 1),
                    kr[:, [x - cu[b] for x in rows]], kerr[:, [x - cu[b] for x in rows]], "keys")
        assert torch.equal(names["v_cache"].cpu().view(-1, n_kv, d)[at], qkv[rows, n_q + n_kv:])
    attn.check_device_status()
