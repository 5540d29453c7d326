"""Plain forms in 64 bits of rotary positions and of a decode step with drafted
tokens, for the tests; CPU tensors."""

import random

import torch

F64 = torch.float64


def turned(x, pos, inv_freq, interleaved=False, sign=1.0, magnitude=1.0):
    """x (heads, tokens, d) by pos (tokens,), as products of complex numbers; and how
    far an fp32 computation may be off before its last rounding: cos and sin come
    from an angle within 2^-24 half turns (2e-7 rad), themselves within 2^-22, and
    the two products and the sum round three times at 2^-24: below 2^-20 of the
    pair's |x1| + |x2| times the magnitude."""
    f, r = inv_freq.to(F64), 2 * inv_freq.shape[0]
    x = x.to(F64)
    a = sign * pos.to(F64)[:, None] * f
    z = magnitude * torch.complex(a.cos(), a.sin())
    y, err = x.clone(), torch.zeros_like(x)
    i1, i2 = ((slice(0, r, 2), slice(1, r, 2)) if interleaved
              else (slice(0, r // 2), slice(r // 2, r)))
    c = torch.complex(x[..., i1].clone(), x[..., i2].clone()) * z
    e = (x[..., i1].abs() + x[..., i2].abs()) * abs(magnitude) * 2.0 ** -20
    y[..., i1], y[..., i2] = c.real, c.imag
    err[..., i1], err[..., i2] = e, e
    return y, err


def assert_bf16(got, want, err, what=""):
    """Within half a bf16 step (2^-8 of the value) of a value within err of want."""
    d = (got.cpu().to(F64) - want).abs()
    tol = err + (want.abs() + err) * 2.0 ** -8
    assert bool((d <= tol).all()), f"{what}: off by {float((d - tol).max()):.3e} beyond the bound"


def tree(n, seed, chain=False):
    """Parents of n nodes (the root's is -1)."""
    rng = random.Random(seed)
    return [-1] + [i - 1 if chain or rng.random() < 0.4 else rng.randrange(i) for i in range(1, n)]


def words_of(parents):
    """Mask words of a tree: each node's ancestors and itself."""
    w = []
    for i, j in enumerate(parents):
        w.append((w[j] if j >= 0 else 0) | 1 << i)
    return w


def signed(words):
    return [w - (1 << 64) if w >> 63 else w for w in words]


def tree_attention(q, k, v, kv_len, words, scale, window=-1, softcap=0.0, slopes=None):
    """One sequence in 64 bits: q (n, n_q, d), k, v (kv_len + n, n_kv, d), a mask word a
    node.  Returns O (n, n_q, d), LSE (n, n_q) and, for bounds, A = sum p |v| like O, X the
    largest sum of |q_i k_i| * scale, and Ab = sum p |bias| |v|."""
    n, n_q, d = q.shape
    n_kv, L = k.shape[1], k.shape[0]
    g = n_q // n_kv
    j = torch.arange(L)
    bits = torch.tensor([[(w >> u) & 1 for u in range(n)] for w in words], dtype=torch.bool).view(n, n)
    seen = torch.cat([torch.ones(n, kv_len, dtype=torch.bool), bits], dim=1)
    depth = (bits.sum(dim=1) - 1).clamp(min=0)
    kp = torch.cat([j[:kv_len], kv_len + depth])
    dist = (kv_len + depth)[:, None] - kp[None]
    if window >= 0:
        seen &= dist <= window
    Q, K, V = q.to(F64), k.to(F64).repeat_interleave(g, 1), v.to(F64).repeat_interleave(g, 1)
    K = torch.where(seen.any(0)[:, None, None], K, 0.0)
    V = torch.where(seen.any(0)[:, None, None], V, 0.0)
    x = torch.einsum("nhd,lhd->nhl", Q, K) * scale
    X = float(torch.einsum("nhd,lhd->nhl", Q.abs(), K.abs()).nan_to_num().max()) * scale if L else 0.0
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
    bias = torch.zeros(n, 1, L, dtype=F64)
    if slopes is not None:
        bias = slopes.to(F64)[None, :, None] * dist[:, None].to(F64)
        x = x - bias
    x = torch.where(seen[:, None], x, -torch.inf)
    lse = torch.logsumexp(x, dim=2)
    p = torch.where(seen[:, None], torch.exp(x - torch.where(lse == -torch.inf, 0.0, lse)[..., None]), 0.0)
    o = torch.einsum("nhl,lhd->nhd", p, V)
    A = torch.einsum("nhl,lhd->nhd", p, V.abs())
    Ab = torch.einsum("nhl,lhd->nhd", p * bias.abs(), V.abs())
    return o, lse, A, X, Ab
