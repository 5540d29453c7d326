"""Verification of drafted tokens against its definition in whole numbers (Python's), which
outputs have to equal."""

import random

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import tree
from exact_io_aware_order_gb300._lib import status_codes

pytestmark = pytest.mark.gpu
ONE = 1 << 60
I32 = torch.int32


def fixed(x):
    x = float(x)
    return int(x * ONE) if 0 <= x < 2 else 0                 # a power of two: exact, then down


def reference(p, q, tokens, parents, u, u_last):
    """One sequence; p, q (n, V) fp32 on the CPU (q or None)."""
    n, V = p.shape
    if n == 0:
        return 0, [-1] * 64, -1
    row = lambda t: [fixed(x) for x in t.tolist()]
    at, path = 0, [0]
    w, Z, C, pr, qr = row(p[0]), ONE, [], row(p[0]), None if q is None else row(q[0])
    for i in range(1, n):
        if parents[i] != at or not 0 <= tokens[i] < V:
            continue
        x = tokens[i]
        qz = Z if q is None else qr[x] * Z >> 60
        if qz * fixed(u[i]) >> 60 < w[x]:
            at = i
            path.append(i)
            w, Z, C, pr, qr = row(p[i]), ONE, [], row(p[i]), None if q is None else row(q[i])
        elif q is None:
            Z = max(Z - w[x], 0)
            w[x] = 0
        else:
            if C and C[-1] + Z < 8 * ONE:
                C[-1] += Z
            else:
                C.append(Z)
            w = [max(a - sum(b * c >> 60 for c in C), 0) for a, b in zip(pr, qr)]
            Z = sum(w)
    if sum(w) == 0:
        w = row(p[at])
    T, c, token = sum(w) * fixed(u_last) >> 60, 0, V - 1
    for v, a in enumerate(w):
        c += a
        if c > T:
            token = v
            break
    return len(path) - 1, path + [-1] * (64 - len(path)), token


class Case:
    def __init__(self, nodes, V, drafts, seed, chain=False, near=0.3, peak=2.0, extra=2):
        g = torch.Generator().manual_seed(seed)
        self.nodes, self.V = nodes, V
        total = sum(nodes) + extra
        logits = peak * torch.randn(total, V, generator=g)
        self.p = torch.softmax(logits, 1)
        q = torch.softmax(logits + near * torch.randn(total, V, generator=g), 1)
        self.q = q if drafts else None
        rng = random.Random(seed)
        self.cu = [sum(nodes[:i]) for i in range(len(nodes) + 1)]
        self.parents, self.tokens = [], []
        for b, n in enumerate(nodes):
            t = tree(n, seed + b, chain) if n else []
            for i, up in enumerate(t):
                row = q[self.cu[b] + max(up, 0)]
                if drafts:
                    self.tokens.append(int(torch.multinomial(row, 1, generator=g)))
                else:
                    self.tokens.append(int(torch.topk(row, min(3, V)).indices[rng.randrange(min(3, V))]))
            self.parents += t
        self.parents += [-1] * extra
        self.tokens += [0] * extra
        self.u, self.u_last = torch.rand(total, generator=g), torch.rand(len(nodes), generator=g)

    def args(self, dev):
        i32 = lambda x: torch.tensor(x, dtype=I32, device=dev)
        return [self.p.to(dev), i32(self.tokens), i32(self.parents), i32(self.cu), self.u.to(dev),
                self.u_last.to(dev), None if self.q is None else self.q.to(dev)]

    def want(self):
        out = []
        for b, n in enumerate(self.nodes):
            s = slice(self.cu[b], self.cu[b] + n)
            out.append(reference(self.p[s], None if self.q is None else self.q[s], self.tokens[s],
                                 self.parents[s], self.u[s], self.u_last[b]))
        return [list(x) for x in zip(*out)]

    def check(self, dev, args=None):
        got = attn.verify_tree(*(args or self.args(dev)))
        want = self.want()
        for name, g, w in zip(("num_accepted", "path", "next_token"), got, want):
            assert g.tolist() == w, name
        return want


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 1000, 8191, 8192, 8193, 32000])
def test_sizes(dev, V, drafts):
    c = Case([1, 0, 6, 64, 2, 17], V, drafts, seed=V)
    c.check(dev)
    attn.check_device_status()


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("chain", [False, True])
def test_walks(dev, chain, drafts):
    """Many trees, small vocabulary: long paths, many refusals, every level of them."""
    taken = set()
    for seed in range(6):
        c = Case([1 + (7 * i + seed) % 64 for i in range(40)], 13, drafts, seed, chain,
                 near=(0.0, 0.1, 1.0)[seed % 3], peak=(0.2, 2.0)[seed % 2])
        taken |= set(c.check(dev)[0])
    assert {0, 1, 2, 3} <= taken                              # the inputs reach these
    attn.check_device_status()


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("batch,V", [(80, 8200), (640, 9)])
def test_large_batches(dev, batch, V, drafts):
    """More sequences than are on the GPU at once."""
    c = Case([1 + i % 4 for i in range(batch)], V, drafts, seed=batch, near=0.3)
    c.check(dev)
    attn.check_device_status()


def test_many_refusals(dev):
    """A root with 63 children that are all refused, p and q nearly apart: Z stays near 1, and C
    passes 8 again and again."""
    V = 300
    c = Case([64, 64], V, True, seed=10)
    c.parents = ([-1] + [0] * 63) * 2 + [-1] * 2
    c.p[:, :150], c.q[:, 150:] = 1e-9, 1e-9
    c.p /= c.p.sum(1, keepdim=True)
    c.q /= c.q.sum(1, keepdim=True)
    c.tokens = [i % 150 for i in range(len(c.tokens))]
    w = c.check(dev)
    assert w[0] == [0, 0] and min(w[2]) >= 150
    c.p[64:] = c.q[64:] * 0.9999 + c.p[64:] * 0.0001          # and one with most of it in common
    c.u[:] = 1 - 2.0 ** -24
    c.check(dev)
    attn.check_device_status()


def test_large_vocabulary(dev):
    c = Case([5, 12], 151936, True, seed=1)
    c.check(dev)


def test_strides_and_alignment(dev):
    """Rows of a wider buffer, from an odd column on."""
    for drafts in (False, True):
        c = Case([9, 30], 9001, drafts, seed=2)
        a = c.args(dev)
        for i in (0, 6):
            if a[i] is not None:
                wide = torch.full((c.p.shape[0], 9050), 0.7, device=dev)
                wide[:, 13:9014] = a[i]
                a[i] = wide[:, 13:9014]
        c.check(dev, a)


def test_edges_of_the_draw(dev):
    """u of 0 and the largest below 1; leading and trailing zeros; probabilities far below 2^-60."""
    V = 9000
    for u in (0.0, 1 - 2.0 ** -24, 0.5):
        c = Case([1, 1, 1, 1], V, False, seed=3)
        c.p[0, :5000] = 0
        c.p[0, -1000:] = 0
        c.p[1] = 0
        c.p[1, 4321] = 1.0
        c.p[2] = 1e-30
        c.p[2, 8000] = 1e-18
        c.p[3] = 0                                            # nothing at all: the last entry
        c.u_last[:] = u
        w = c.check(dev)
        assert w[2][1] == 4321 and w[2][2] in (8000, V - 1) and w[2][3] == V - 1


def test_equal_distributions(dev):
    """p == q: every chain is accepted whatever u, and nothing is left after a refusal."""
    c = Case([10, 10], 500, True, seed=4, chain=True, near=0.0)
    c.q = c.p.clone()
    c.u[:] = 1 - 2.0 ** -24
    w = c.check(dev)
    assert w[0] == [9, 9]
    c.u[:] = 1.0                                              # not below 1: refused, residual empty
    w = c.check(dev)
    assert w[0] == [0, 0]


def test_distribution(dev):
    """Accepted or drawn, the first token is distributed as the target's: 60000 draws of a small
    vocabulary, each entry within 5 standard deviations."""
    V, B = 6, 60000
    g = torch.Generator(device=dev).manual_seed(5)
    p = torch.tensor([0.4, 0.05, 0.25, 0.1, 0.0, 0.2], device=dev)
    q = torch.tensor([0.1, 0.3, 0.2, 0.1, 0.2, 0.1], device=dev)
    for drafts in (True, False):
        # A root with three children.
        tokens = torch.multinomial(q, B * 4, replacement=True, generator=g).view(B, 4).to(I32)
        if not drafts:
            tokens = torch.tensor([0, 2, 0, 5], dtype=I32, device=dev).repeat(B, 1)
        parents = torch.tensor([-1, 0, 0, 0], dtype=I32, device=dev).repeat(B, 1).view(-1)
        cu = torch.arange(B + 1, dtype=I32, device=dev) * 4
        n, path, token = attn.verify_tree(
            p.repeat(4 * B, 1), tokens.view(-1).contiguous(), parents, cu,
            torch.rand(4 * B, generator=g, device=dev), torch.rand(B, generator=g, device=dev),
            q.repeat(4 * B, 1) if drafts else None)
        first = torch.where(n > 0, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], token)
        share = torch.bincount(first.long(), minlength=V).double() / B
        sd = (p.double() * (1 - p.double()) / B).sqrt()
        assert bool(((share - p.double()).abs() <= 5 * sd + 1e-12).all()), share.tolist()
        assert int(n.max()) == 1
    attn.check_device_status()


def test_not_probabilities(dev):
    """NaN, infinities, negative ones and ones from 2 on count as 0."""
    c = Case([3, 3], 50, True, seed=6)
    for t in (c.p, c.q):
        t[0, :5] = torch.tensor([float("nan"), float("inf"), -0.5, 2.0, -float("inf")])
    c.tokens[1] = 3
    c.check(dev)


def test_graph(dev):
    c = Case([20, 6, 1], 9000, True, seed=7)
    a = c.args(dev)
    out = [torch.empty(3, dtype=I32, device=dev), torch.empty(3, 64, dtype=I32, device=dev),
           torch.empty(3, dtype=I32, device=dev)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.verify_tree(*a, num_accepted=out[0], path=out[1], next_token=out[2])
    for seed in range(4):
        c.u = torch.rand(c.u.shape, generator=torch.Generator().manual_seed(seed))
        a[4].copy_(c.u)
        graph.replay()
        assert [x.tolist() for x in out] == c.want()


def flagged():
    with pytest.raises(attn.AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]


def test_flags(dev):
    c = Case([10, 12], 40, True, seed=8)
    good, toks = list(c.parents), list(c.tokens)
    for i, bad in ((3, 3), (3, 9), (5, -1), (2, -7), (4, 2**31 - 1)):
        c.parents[i] = bad
        args = c.args(dev)
        c.parents[i] = -5                                     # the definition: never reached
        for g, w in zip(attn.verify_tree(*args), c.want()):
            assert g.tolist() == w
        flagged()
        c.parents = list(good)
    c.parents[10] = 0                                         # a root with a parent
    attn.verify_tree(*c.args(dev))
    flagged()
    c.parents = list(good)
    for i, bad in ((1, -1), (1, 40), (14, 2**31 - 1)):
        c.tokens[i] = bad
        c.check(dev)
        flagged()
        c.tokens = list(toks)
    for cu in ([1, 10, 22], [0, 30, 22], [0, 10, 99], [0, -4, 22]):
        c.cu = cu
        attn.verify_tree(*c.args(dev))
        flagged()


def test_refusals(dev):
    c = Case([4, 3], 30, True, seed=9)
    a = c.args(dev)
    names = ("target_probs", "draft_tokens", "parents", "cu_nodes", "u_accept", "u_sample", "draft_probs")
    base = dict(zip(names, a))
    for kw, exc in [(dict(target_probs=a[0].double()), TypeError), (dict(target_probs=a[0][0]), ValueError),
                    (dict(target_probs=a[0].cpu()), ValueError), (dict(target_probs=a[0].t()), ValueError),
                    (dict(draft_probs=a[6][:, :29]), ValueError), (dict(draft_probs=a[6].half()), TypeError),
                    (dict(draft_tokens=a[1].long()), TypeError), (dict(parents=a[2][:3]), ValueError),
                    (dict(cu_nodes=a[3][:1]), ValueError), (dict(cu_nodes=a[3].long()), TypeError),
                    (dict(u_accept=a[4].double()), TypeError), (dict(u_sample=a[5][:1]), ValueError),
                    (dict(target_probs=a[0][:1].expand(9, 30)), attn.AttnError),
                    (dict(path=torch.empty(2, 63, dtype=I32, device=dev)), ValueError),
                    (dict(next_token=torch.empty(2, device=dev)), TypeError)]:
        with pytest.raises(exc):
            attn.verify_tree(**{**base, **kw})
    attn.check_device_status()
