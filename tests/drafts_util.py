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
