"""Verification of rows that are no probabilities, whose sums are 8 and more: they stop at 8 -
2^-60.  Against the definition in Python's whole numbers."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from test_gpu_verify_tree import I32, ONE, Case, fixed

pytestmark = pytest.mark.gpu
MOST = 8 * ONE - 1


def reference(p, q, tokens, parents, u, u_last):
    """One sequence, as include/attn.h has it; sums of nonnegative numbers that stop at MOST."""
    n, V = p.shape
    row = lambda t: [fixed(x) for x in t.tolist()]
    total = lambda w: min(sum(w), MOST)
    at, path = 0, [0]
    w, Z, C = row(p[0]), ONE, []
    for i in range(1, n):
        if parents[i] != at:
            continue
        x = tokens[i]
        qr = None if q is None else row(q[at])
        qz = Z if q is None else qr[x] * Z >> 60
        if qz * fixed(u[i]) >> 60 < w[x]:
            at = i
            path.append(i)
            w, Z, C = row(p[i]), ONE, []
        elif q is None:
            Z = max(Z - w[x], 0)
            w[x] = 0
        else:
            if C and C[-1] + Z < 8 * ONE:
                C[-1] += Z
            else:
                C.append(Z)
            w = [max(a - sum(b * c >> 60 for c in C), 0) for a, b in zip(row(p[at]), qr)]
            Z = total(w)
    if sum(w) == 0:
        w = row(p[at])
    T, c, token = total(w) * fixed(u_last) >> 60, 0, V - 1
    for v, a in enumerate(w):
        c = min(c + a, MOST)
        if c > T:
            token = v
            break
    return len(path) - 1, path + [-1] * (64 - len(path)), token


def check(dev, c):
    got = [x.tolist() for x in attn.verify_tree(*c.args(dev))]
    for b, n in enumerate(c.nodes):
        s = slice(c.cu[b], c.cu[b] + n)
        want = reference(c.p[s], None if c.q is None else c.q[s], c.tokens[s], c.parents[s], c.u[s],
                         c.u_last[b])
        assert (got[0][b], got[1][b], got[2][b]) == want, b


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V", [9, 40, 700, 9000])
def test_large_sums(dev, V, drafts):
    """Entries up to 2 that sum to 4 (below the limit), 8 - 2^-21, 8, 16, 17, 40 and more, in the
    first entries (one thread's), everywhere, and in the last ones."""
    for seed, big in enumerate((2.0, 4.0, 8.0 - 2.0 ** -21, 8.0, 15.9, 16.0, 17.0, 40.0, 500.0)):
        c = Case([1, 6, 20, 3], V, drafts, seed=seed)
        for t in (c.p, c.q) if drafts else (c.p,):
            for r in range(0, len(t), 2):
                n = min(V, max(5, int(big / 1.5)))
                at = (0, V - n, (V - n) // 2)[r // 2 % 3]
                t[r] = 0
                t[r, at:at + n] = min(big / n, 1.999)
                t[r, at] += min(0.001, 1.9995 - float(t[r, at]))
        c.u *= 0.9
        for last in (0.0, 0.3, 0.5, 0.9, 1 - 2.0 ** -24):
            c.u_last[:] = last
            check(dev, c)
    attn.check_device_status()


def test_at_the_limit(dev):
    """Four entries of 2 - 2^-23: 8 - 2^-21, the largest such sum that fits; one of 2^-21 more ends
    at 8 - 2^-60, and another changes nothing."""
    c = Case([1, 1, 1], 6, False, seed=1)
    c.p[:] = 0
    c.p[:3, :4] = 2 - 2.0 ** -23
    c.p[1, 4], c.p[2, 4], c.p[2, 5] = 2.0 ** -21, 2.0 ** -21, 1.5
    for last in (0.0, 0.25, 0.74, 0.76, 1 - 2.0 ** -24):
        c.u_last[:] = last
        check(dev, c)
    attn.check_device_status()
