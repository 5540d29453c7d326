"""New keys and values into a bf16 cache, rotated on the way, against the formula."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import assert_bf16, turned
from exact_io_aware_order_gb300._lib import status_codes

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Case:
    def __init__(self, dev, lens, new, n_q, n_kv, d, block, paged, seed=0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.n_kv, self.d, self.block = lens, new, n_kv, d, block
        B, self.total = len(lens), sum(new) + extra
        room = [a + b for a, b in zip(lens, new)]
        if paged:
            need = [-(-n // block) for n in room]
            order = torch.randperm(sum(need) + 3, generator=g).to(torch.int32)
            self.table = torch.full((B, max(max(need), 1) + 1), -7, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = order[at:at + n]
                at += n
            shape = (sum(need) + 3, block, n_kv, d)
        else:
            self.table, shape = None, (B, max(max(room), 1) + 2, n_kv, d)
        rand = lambda *s: torch.randn(*s, generator=g).to(BF16)
        self.kc, self.vc = rand(*shape), rand(*shape)
        self.qkv = rand(self.total, n_q + 2 * n_kv, d)
        self.q, self.k, self.v = self.qkv.split([n_q, n_kv, n_kv], dim=1)
        self.cu = [sum(new[:i]) for i in range(B + 1)]
        self.dev = dev

    def row(self, s, slot):
        if self.table is None:
            return s * self.kc.shape[1] + slot
        return int(self.table[s, slot // self.block]) * self.block + slot % self.block

    def run(self, f=None, positions=None, with_q=True, one=False, **kw):
        """Runs the call; returns (q_out tokens first or None, caches) on the CPU."""
        dev = self.dev
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        qkv = self.qkv.to(dev)
        q, k, v = qkv.split([self.q.shape[1], self.n_kv, self.n_kv], dim=1)
        kc, vc = self.kc.to(dev), self.vc.to(dev)
        table = None if self.table is None else self.table.to(dev)
        flip = (lambda x: x) if one else (lambda x: x.transpose(0, 1))
        q_out = torch.full(q.shape, 3.0, dtype=BF16, device=dev) if with_q else None
        r = attn.cache_append(flip(k), flip(v), kc, vc, i32(self.lens),
                              None if one else i32(self.cu), table,
                              None if f is None else f.to(dev),
                              None if positions is None else i32(positions),
                              q=flip(q) if with_q else None,
                              q_out=flip(q_out) if with_q else None, **kw)
        assert (r is None) == (not with_q)
        return None if not with_q else q_out.cpu(), kc.cpu(), vc.cpu()

    def check(self, got, f, positions, skip=(), **kw):
        q, kc, vc = got
        k_was, v_was = self.kc.view(-1, self.n_kv, self.d), self.vc.view(-1, self.n_kv, self.d)
        kc, vc = kc.view(-1, self.n_kv, self.d), vc.view(-1, self.n_kv, self.d)
        rows, toks, pos = [], [], []
        for s, n in enumerate(self.new):
            for i in range(n):
                t = self.cu[s] + i
                toks.append(t)
                pos.append(self.lens[s] + i if positions is None else positions[t])
                if s not in skip:
                    rows.append((self.row(s, self.lens[s] + i), t))
        where = torch.tensor(pos, dtype=torch.int64)
        toks = torch.tensor(toks, dtype=torch.int64)
        if q is not None:
            want, err = turned(self.q[toks].transpose(0, 1), where, f, **kw)
            assert_bf16(q[toks].transpose(0, 1), want, err, "q")
            rest = torch.ones(self.total, dtype=torch.bool)
            rest[toks] = False
            assert bool((q[rest] == 3).all())                # rows of no sequence stay
        want_k, want_v, touched = k_was.clone(), v_was.clone(), torch.zeros(len(k_was), dtype=torch.bool)
        at = {int(t): i for i, t in enumerate(toks)}
        if rows:
            r, t = torch.tensor([a for a, _ in rows]), torch.tensor([b for _, b in rows])
            touched[r] = True
            want_v[r] = self.v[t]
            if f is None:
                want_k[r] = self.k[t]
                assert torch.equal(kc, want_k)
            else:
                w, err = turned(self.k[t].transpose(0, 1), where[[at[int(x)] for x in t]], f, **kw)
                assert_bf16(kc[r].transpose(0, 1), w, err, "k")
        assert torch.equal(vc, want_v)
        assert torch.equal(kc[~touched], k_was[~touched])     # nothing else changes


@pytest.mark.parametrize("paged,block", [(True, 1), (True, 16), (True, 24), (True, 128), (False, 0)])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 128, True), (128, 32, False), (256, 256, False)])
def test_ragged(dev, paged, block, d, rot, inter):
    c = Case(dev, [0, 17, 100, 5, 0, 33], [3, 0, 70, 1, 130, 0], 5, 2, d, block or 16, paged, seed=1, extra=4)
    f = attn.rope_inv_freq(rot, device="cpu")
    c.check(c.run(f, interleaved=inter, magnitude=1.5), f, None, interleaved=inter, magnitude=1.5)
    pos = [(7 * t) % 900000 - 50 for t in range(c.total)]
    c.check(c.run(f, pos, interleaved=inter), f, pos, interleaved=inter)
    attn.check_device_status()


@pytest.mark.parametrize("B", [1, 3, 64])
def test_one_token_a_sequence(dev, B):
    lens = [(37 * b) % 50 for b in range(B)]
    c = Case(dev, lens, [1] * B, 8, 2, 128, 16, True, seed=2)
    f = attn.rope_inv_freq(128, device="cpu")
    c.check(c.run(f, one=True), f, None)
    c.check(c.run(f, with_q=False, one=True), f, None)
    attn.check_device_status()


def test_without_rotation(dev):
    c = Case(dev, [4, 0], [9, 30], 1, 3, 64, 16, True, seed=3)
    c.check(c.run(None, with_q=False), None, None)


def test_many_sequences(dev):
    """More sequences than one round of probes, most of them empty."""
    new = [(i % 7 == 3) * (i % 5) for i in range(1500)]
    c = Case(dev, [i % 11 for i in range(1500)], new, 2, 1, 64, 4, True, seed=4)
    f = attn.rope_inv_freq(64, device="cpu")
    c.check(c.run(f), f, None)
    attn.check_device_status()


def test_queries_in_place_and_graph(dev):
    c = Case(dev, [20, 3], [6, 11], 4, 2, 128, 16, True, seed=5)
    f = attn.rope_inv_freq(128, device=dev)
    want = c.run(f.cpu())
    dv = lambda x: x.to(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    kc, vc, q, k, v = dv(c.kc), dv(c.vc), dv(c.q.contiguous()), dv(c.k), dv(c.v)
    lens, cu, table = i32(c.lens), i32(c.cu), dv(c.table)
    was = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.cache_append(k.transpose(0, 1), v.transpose(0, 1), kc, vc, lens, cu, table, f,
                          q=q.transpose(0, 1), q_out=q.transpose(0, 1))
    q.copy_(was)
    graph.replay()
    for a, b in zip((q, kc, vc), want):
        assert torch.equal(a.cpu(), b)
    lens.add_(1)                                             # the next replay's slots are one on
    q.copy_(was)
    graph.replay()
    c.lens = [n + 1 for n in c.lens]
    for a, b in zip((q,), c.run(f.cpu())[:1]):
        assert torch.equal(a.cpu(), b)


def flagged():
    with pytest.raises(attn.AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]


def test_flags(dev):
    f = attn.rope_inv_freq(64, device="cpu")
    c = Case(dev, [5, 9, 0], [4, 6, 5], 2, 1, 64, 4, True, seed=6)
    ok = c.table.clone()
    c.table[1, 2:] = -1                                      # sequence 1's slots 9 .. 14
    c.check(c.run(f), f, None, skip=(1,))
    flagged()
    c.table[1, 2:] = c.kc.shape[0]
    c.check(c.run(f), f, None, skip=(1,))
    flagged()
    c.table = ok
    for bad in (-1, c.table.shape[1] * 4 - 5, 2**31 - 1):     # 6 tokens do not fit
        c.lens = [5, bad, 0]
        got = c.run(f, positions=[1] * c.total)
        c.check(got, f, [1] * c.total, skip=(1,))
        flagged()
    c.lens = [5, 9, 0]
    good = c.cu
    for cu in ([1, 4, 10, 15], [0, 9, 4, 15], [0, 4, 10, 99], [-3, 4, 10, 15]):
        c.cu = cu
        c.run(f)                                             # stays in bounds
        flagged()
    c.cu = good


def test_refusals(dev):
    c = Case(dev, [4, 0], [3, 3], 2, 2, 64, 4, True, seed=7)
    f = attn.rope_inv_freq(64, device=dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    base = dict(k_new=c.k.to(dev).transpose(0, 1), v_new=c.v.to(dev).transpose(0, 1),
                k_cache=c.kc.to(dev), v_cache=c.vc.to(dev), kv_lens=i32(c.lens), cu_seqlens=i32(c.cu),
                block_table=c.table.to(dev), inv_freq=f, q=c.q.to(dev).transpose(0, 1))
    attn.cache_append(**base)
    for kw, exc in [(dict(k_new=None), TypeError), (dict(k_new=base["k_new"].float()), TypeError),
                    (dict(v_new=base["v_new"][:, :5]), ValueError), (dict(k_cache=base["k_cache"].float()), TypeError),
                    (dict(v_cache=base["v_cache"][:2]), ValueError), (dict(cu_seqlens=i32([0, 6])), ValueError),
                    (dict(cu_seqlens=None), ValueError), (dict(block_table=i32([[0, 1]])), ValueError),
                    (dict(block_table=torch.empty(2, 0, dtype=torch.int32, device=dev)), ValueError),
                    (dict(block_table=None), ValueError), (dict(inv_freq=None), ValueError),
                    (dict(inv_freq=f[:4].clone()), attn.AttnError), (dict(positions=i32([1])), ValueError),
                    (dict(q=base["q"][:, :4]), ValueError), (dict(q=None, q_out=base["q"]), ValueError),
                    (dict(q_out=base["q"][:1].expand(2, 6, 64)), attn.AttnError),
                    (dict(k_cache=base["k_cache"][:, :, :1].contiguous(), v_cache=base["v_cache"][:, :, :1].contiguous()), ValueError),
                    (dict(kv_lens=base["kv_lens"].long()), TypeError)]:
        with pytest.raises(exc):
            attn.cache_append(**{**base, **kw})
    attn.check_device_status()
