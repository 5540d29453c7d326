"""Attention of trees of drafted tokens over a cache, against the formula in 64 bits.

Bounds.  A score is d / 16 tensor-core additions of exact products, each good to 2^-22 of
the sum of magnitudes X; tanh and the bias add 2^-21 of the cap and of the bias; the
exponential and its argument 2^-20.  A weight enters the product with V good to 2^-16
(fp32 O) or 2^-8 (bf16 O), and keys / 16 additions lose 2^-23 each of A = sum p |v|.
So O is within A (w + 2 e) + 2^-21 Ab, e the score's error, and rounds to bf16 by 2^-8."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import F64, signed, tree, tree_attention, words_of
from exact_io_aware_order_gb300._lib import status_codes

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, dev, lens, nodes, n_q, n_kv, d, block=16, paged=True, kind="tree", seed=0,
                 extra=3, window=-1, softcap=0.0, alibi=False, junk=True):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.lens, self.nodes, self.d, self.block = dev, lens, nodes, d, block
        self.n_q, self.n_kv = n_q, n_kv
        self.window, self.softcap = window, softcap
        B, self.total = len(lens), sum(nodes) + extra
        self.cu = [sum(nodes[:i]) for i in range(B + 1)]
        rand = lambda *s: torch.randn(*s, generator=g).to(BF16)
        self.q = rand(self.total, n_q, d)
        amp = 1 + 4 * (torch.rand(n_kv, d, generator=g) < 0.05)
        self.k = [(rand(a + b, n_kv, d) * amp).to(BF16) for a, b in zip(lens, nodes)]
        self.v = [rand(a + b, n_kv, d) for a, b in zip(lens, nodes)]
        self.slopes = torch.rand(n_q, generator=g) if alibi else None
        self.words = []
        for b, n in enumerate(nodes):
            if kind == "any":                                # bits at random: empty rows among them
                w = [int(x) for x in torch.randint(0, 2**62, (n,), generator=g)]
                w = [0 if i % 3 == 1 else x for i, x in enumerate(w)]
            else:
                w = words_of(tree(n, seed + b, kind == "chain")) if n else []
            self.words.append(w)
        self.mask = None if kind == "chain" else sum(self.words, []) + [-1 & (2**64 - 1)] * extra
        fill = float("nan") if junk else 0.0                 # slots that nothing may read
        if paged:
            need = [-(-(a + b) // block) for a, b in zip(lens, nodes)]
            order = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
            self.table = torch.full((B, max(need) + 1), -9, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = order[at:at + n]
                at += n
            shape = (sum(need) + 2, block, n_kv, d)
        else:
            self.table, shape = None, (B, max(a + b for a, b in zip(lens, nodes)) + 2, n_kv, d)
        self.kc, self.vc = torch.full(shape, fill, dtype=BF16), torch.full(shape, fill, dtype=BF16)
        for b in range(B):
            r = self.rows(b, len(self.k[b]))
            self.kc.view(-1, n_kv, d)[r], self.vc.view(-1, n_kv, d)[r] = self.k[b], self.v[b]

    def rows(self, b, n):
        j = torch.arange(n)
        if self.table is None:
            return b * self.kc.shape[1] + j
        return self.table[b].long()[j // self.block] * self.block + j % self.block

    def args(self):
        dev = self.dev
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        mask = None if self.mask is None else torch.tensor(signed(self.mask), dtype=torch.int64, device=dev)
        return dict(q=self.q.to(dev), k_cache=self.kc.to(dev), v_cache=self.vc.to(dev),
                    kv_lens=i32(self.lens), cu_nodes=i32(self.cu), tree_mask=mask,
                    block_table=None if self.table is None else self.table.to(dev),
                    window_left=self.window, softcap=self.softcap,
                    alibi_slopes=None if self.slopes is None else self.slopes.to(dev))

    def run(self, dtype=F32, **kw):
        out = torch.full((self.total, self.n_q, self.d), 7.0, dtype=dtype, device=self.dev)
        lse = torch.full((self.total, self.n_q), 7.0, device=self.dev)
        a = {**self.args(), "out_dtype": dtype, "out": out, "lse": lse, **kw}
        o, l = attn.decode_tree(**a)
        return o.cpu(), l.cpu()

    def check(self, o, lse, skip=()):
        wide = o.dtype is F32
        for b, (n, kv) in enumerate(zip(self.nodes, self.lens)):
            if b in skip or n == 0:
                continue
            sl = slice(self.cu[b], self.cu[b] + n)
            ro, rl, A, X, Ab = tree_attention(self.q[sl], self.k[b], self.v[b], kv, self.words[b],
                                              self.d ** -0.5, self.window, self.softcap, self.slopes)
            e = self.d / 16 * X * 2.0 ** -22 + self.softcap * 2.0 ** -21 + 2.0 ** -20
            tol = A * ((2.0 ** -16 if wide else 2.0 ** -8) + 2 * e + (kv + n + 16) / 16 * 2.0 ** -23) + Ab * 2.0 ** -21
            if not wide:
                tol = tol + (ro.abs() + tol) * 2.0 ** -8
            d = (o[sl].to(F64) - ro).abs()
            assert bool((d <= tol).all()), f"sequence {b}: {float((d - tol).max()):.3e} beyond the bound"
            empty = torch.isneginf(rl)
            assert torch.equal(torch.isneginf(lse[sl]), empty) and bool((o[sl][empty] == 0).all())
            worst = (lse[sl].to(F64) - rl)[~empty].abs()
            bound = (2 * e + 2.0 ** -21 * (1 + rl.abs()))[~empty]
            if self.slopes is not None:
                bound = bound + 2.0 ** -21 * 64 * float(self.slopes.max())
            assert bool((worst <= bound).all()), f"LSE of sequence {b}: {float(worst.max()):.3e}"
        if self.cu[-1] < self.total:                          # rows of no sequence stay
            assert bool((o[self.cu[-1]:] == 7).all()) and bool((lse[self.cu[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("block,paged", [(16, True), (1, True), (24, True), (100, True), (256, True), (0, False)])
def test_short(dev, block, paged, kind, d, dtype):
    """Lengths around a key tile's border, no tokens, no nodes, one node, 64 nodes."""
    c = Case(dev, [0, 1, 63, 127, 128, 90, 300, 0, 511], [1, 64, 2, 3, 1, 60, 0, 37, 64], 6, 2, d, block or 16,
             paged, kind, seed=1)
    o, lse = c.run(dtype)
    c.check(o, lse)
    o2, lse2 = c.run(dtype, max_kv_len=600 if paged else None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    attn.check_device_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n_q,n_kv,d", [(1, 1, 128), (28, 4, 128), (64, 1, 64), (16, 8, 256), (40, 1, 256), (48, 2, 128)])
@pytest.mark.parametrize("nodes", [[1], [5, 33], [64, 64, 17]])
def test_heads(dev, nodes, n_q, n_kv, d, dtype):
    """One row to 4096 rows a kv head; lengths that are cut over many blocks."""
    lens = [2500, 700, 4][:len(nodes)]
    c = Case(dev, lens, nodes, n_q, n_kv, d, 16, True, "tree", seed=2)
    c.check(*c.run(dtype))
    attn.check_device_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("variant", [dict(window=0), dict(window=3), dict(window=63), dict(window=64), dict(window=500),
                                     dict(softcap=20.0), dict(window=100, softcap=50.0), dict(alibi=True),
                                     dict(alibi=True, window=40)])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_variants(dev, kind, variant, d, dtype):
    c = Case(dev, [0, 5, 130, 1700, 64], [20, 64, 9, 31, 1], 6, 2, d, 24, True, kind, seed=3, **variant)
    if variant.get("window", -1) >= 0:
        # What lies in front of every node's window may hold anything.
        for b, n in enumerate(c.lens):
            r = c.rows(b, max(0, n - c.window))
            c.kc.view(-1, c.n_kv, d)[r] = c.vc.view(-1, c.n_kv, d)[r] = float("nan")
            c.k[b][:max(0, n - c.window)] = c.v[b][:max(0, n - c.window)] = 0.0
    c.check(*c.run(dtype))
    attn.check_device_status()


@pytest.mark.parametrize("lens,nodes,block", [([30720], [32], 16), ([32768, 40, 9000], [64, 1, 7], 64)])
def test_long(dev, lens, nodes, block):
    c = Case(dev, lens, nodes, 14, 2, 128, block, True, "tree", seed=4, extra=0)
    for dtype in (F32, BF16):
        c.check(*c.run(dtype))
    attn.check_device_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_that_grow(dev, d, dtype):
    """Maxima that rise by 30 nats every few keys, in rows' own places: the reference of the
    exponentials is raised at tile borders and inside tiles, and O rescaled."""
    c = Case(dev, [700, 40], [20, 64], 4, 1, d, 16, True, "any", seed=15)
    for b, n in enumerate(c.lens):
        k = torch.zeros_like(c.k[b])
        step = torch.arange(len(k)) // 37
        k[:, 0, 0] = (step.float() * 30 - 250).to(BF16)
        k[:, 0, 1] = (-step.float() * 30).to(BF16)
        c.k[b] = k
        c.kc.view(-1, 1, d)[c.rows(b, len(k))] = k
    c.q.zero_()
    c.q[:, :, 0] = d ** 0.5
    c.q[::3, :, 0], c.q[::3, :, 1] = 0.0, d ** 0.5            # every third row falls instead
    c.check(*c.run(dtype))
    c.check(*c.run(dtype, max_kv_len=800))
    attn.check_device_status()


def test_many_sequences(dev):
    n = 700
    lens, nodes = [(i * 37) % 300 for i in range(n)], [(i * 11) % 7 for i in range(n)]
    c = Case(dev, lens, nodes, 2, 1, 64, 16, True, "tree", seed=5)
    c.check(*c.run(BF16))
    c.check(*c.run(F32, max_kv_len=5000))
    attn.check_device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hint", [300, None])
def test_row_tiles_in_turn(dev, d, hint):
    """Items of one and of two row tiles one after another in a block, whole or cut."""
    nodes = [1, 64, 3, 40, 2, 64, 64, 1, 1, 33] * 30
    lens = [(i * 53) % 400 for i in range(len(nodes))]
    c = Case(dev, lens, nodes, 8, 2, d, 16, True, "tree", seed=14)
    for kw in (dict(), dict(out_dtype=BF16)):
        dtype = kw.get("out_dtype", F32)
        c.check(*c.run(dtype, max_kv_len=hint))
    attn.check_device_status()


def test_far_cache_rows(dev):
    """A block whose elements lie past 2^32: offsets are 64 bits."""
    block, n_kv, d = 256, 8, 256
    blocks = (1 << 32) // (block * n_kv * d) + 3              # 8.6 GB a cache
    kc = torch.zeros(blocks, block, n_kv, d, dtype=BF16, device=dev)
    vc = torch.zeros_like(kc)
    c = Case(dev, [400], [6], 16, n_kv, d, block, True, "tree", seed=6, extra=0)
    where = torch.tensor([blocks - 1, blocks - 2])
    for b, n in enumerate((256, 150)):
        src = c.table[0, b]
        kc[where[b], :n], vc[where[b], :n] = c.kc[src, :n].to(dev), c.vc[src, :n].to(dev)
    o, lse = attn.decode_tree(**{**c.args(), "k_cache": kc, "v_cache": vc,
                                 "block_table": where.to(torch.int32).to(dev)[None].contiguous()})
    c.check(o.cpu(), lse.cpu())
    attn.check_device_status()


def test_one_node_is_a_decode(dev):
    c = Case(dev, [1000, 37], [1, 1], 8, 2, 128, 16, True, "chain", seed=7, extra=0)
    a = c.args()
    o, lse = attn.decode_tree(**a)
    po, pl = attn.decode(a["q"], a["k_cache"], a["v_cache"], a["kv_lens"] + 1, a["block_table"])
    assert float((o - po).abs().max()) <= 2e-2 and float((lse - pl).abs().max()) <= 1e-3
    attn.check_device_status()


def test_results_repeat(dev):
    c = Case(dev, [20000, 3000, 70], [40, 64, 11], 16, 2, 128, 16, True, "tree", seed=8)
    first = c.run(F32)
    c.check(*first)
    for _ in range(5):
        again = c.run(F32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    attn.check_device_status()


def test_graph_and_streams(dev):
    """A captured call replayed as the cache grows, beside calls on another stream with a
    workspace of their own."""
    c = Case(dev, [2000, 900], [16, 16], 8, 2, 128, 16, True, "tree", seed=9, extra=0, junk=False)
    a = c.args()
    nb = c.table.shape[1] * 16
    out, lse = torch.empty(32, 8, 128, device=dev), torch.empty(32, 8, device=dev)
    want = {}
    for add in (0, -3, -700):
        want[add] = attn.decode_tree(**{**a, "kv_lens": a["kv_lens"] + add})
    attn.check_device_status()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    lens = a["kv_lens"].clone()
    with torch.cuda.graph(graph):
        attn.decode_tree(**{**a, "kv_lens": lens}, out=out, lse=lse)
    other.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for add in (0, -3, -700, 0):
        lens.copy_(a["kv_lens"] + add)
        torch.cuda.synchronize()
        got = attn.decode_tree(**a, stream=other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[add][0]) and torch.equal(lse, want[add][1])
        assert torch.equal(got[0], want[0][0])
        attn.check_device_status()


def flagged():
    with pytest.raises(attn.AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]


@pytest.mark.parametrize("long", [False, True])
def test_flags(dev, long):
    c = Case(dev, [3000 if long else 70, 9, 40], [4, 6, 5], 4, 2, 64, 16, True, "tree", seed=10)
    for bad in (-1, c.table.shape[1] * 16 - 5, 2**31 - 1):
        c.lens[1], was = bad, c.lens[1]
        o, lse = c.run(F32)
        c.lens[1] = was
        c.check(o, lse, skip=(1,))
        assert bool((o[4:10] == 0).all()) and bool(torch.isneginf(lse[4:10]).all())
        flagged()
    good = c.table.clone()
    for entry in (-1, c.kc.shape[0], 2**31 - 1):
        c.table[1, 0] = entry
        o, lse = c.run(F32)
        c.table.copy_(good)
        c.check(o, lse, skip=(1,))
        flagged()
    cu = c.cu
    for bad in ([1, 4, 10, 15], [0, 9, 4, 15], [0, 4, 10, 99], [-3, 4, 10, 15]):
        c.cu = bad
        c.run(F32)
        flagged()
    c.cu = cu


def test_more_than_64_nodes(dev):
    c = Case(dev, [50], [64], 2, 2, 64, 16, True, "chain", seed=11, extra=6)
    full = c.run(F32)
    c.check(*full)
    c.cu = [0, 70]
    o, lse = c.run(F32)
    flagged()
    assert torch.equal(o[:64], full[0][:64]) and bool((o[64:] == 7).all())


def test_workspace(dev):
    c = Case(dev, [3000], [8], 8, 2, 128, 16, True, "tree", seed=12, extra=0)
    from exact_io_aware_order_gb300._lib import lib
    n = lib().attn_decode_tree_workspace_bytes(1, 8, 8, 2, 128, c.table.shape[1] * 16, -1)
    assert n > 0 and lib().attn_decode_tree_workspace_bytes(1, 8, 8, 2, 128, 300, -1) == 0
    want = c.run(F32)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    got = c.run(F32, workspace=ws)
    assert torch.equal(want[0], got[0])
    with pytest.raises(attn.AttnError) as e:
        c.run(F32, workspace=ws[:n - 16])
    assert e.value.status == status_codes()["ATTN_ERR_SCRATCH"]
    attn.check_device_status()


def test_refusals(dev):
    c = Case(dev, [40, 9], [4, 6], 8, 2, 64, 16, True, "tree", seed=13, extra=0)
    a = c.args()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    attn.decode_tree(**a)
    for kw, exc in [(dict(q=a["q"].float()), TypeError), (dict(q=a["q"][:, :, :32]), ValueError),
                    (dict(q=a["q"][:, :7].contiguous()), attn.AttnError), (dict(q=a["q"].cpu()), ValueError),
                    (dict(k_cache=a["k_cache"].float()), TypeError), (dict(v_cache=a["v_cache"][:1]), ValueError),
                    (dict(kv_lens=i32([1])), ValueError), (dict(cu_nodes=i32([0, 10])), ValueError),
                    (dict(tree_mask=a["tree_mask"].int()), TypeError), (dict(tree_mask=a["tree_mask"][:5]), ValueError),
                    (dict(block_table=None), ValueError), (dict(block_table=i32([[0]])), ValueError),
                    (dict(block_table=torch.empty(2, 0, dtype=torch.int32, device=dev)), ValueError),
                    (dict(max_kv_len=2**40), ValueError), (dict(max_kv_len=-1), attn.AttnError),
                    (dict(scale=0.0), attn.AttnError), (dict(window_left=-2), attn.AttnError),
                    (dict(softcap=-1.0), attn.AttnError), (dict(softcap=2.0, alibi_slopes=torch.ones(8, device=dev)), attn.AttnError),
                    (dict(alibi_slopes=torch.ones(7, device=dev)), ValueError), (dict(out_dtype=torch.float16), ValueError),
                    (dict(out=torch.empty(10, 8, 64, dtype=BF16, device=dev)), TypeError),
                    (dict(lse=torch.empty(10, 7, device=dev)), ValueError), (dict(workspace=a["q"]), TypeError)]:
        with pytest.raises(exc):
            attn.decode_tree(**{**a, **kw})
    attn.check_device_status()
