"""Builds 8-bit caches for the tests and compares them with the reference."""

import numpy as np
import torch

from oracle import cache_fp8_ref as C


class Cache:
    """Codes, scales and block table on the CPU, every byte random (NaN codes
    and NaN scales among them) until something is written."""

    def __init__(self, B, n_kv, d, room, block_size, paged=True, seed=0, extra=2):
        gen = torch.Generator().manual_seed(1000 + seed)
        self.B, self.n_kv, self.d, self.bs, self.paged = B, n_kv, d, block_size, paged
        self.room = max(1, max(room))
        per = -(-self.room // block_size)
        if paged:
            need = [-(-n // block_size) for n in room]
            nb = sum(need) + extra
            perm = torch.randperm(nb, generator=gen).to(torch.int32)
            self.table = torch.full((B, per), nb - 1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = perm[at:at + n]
                at += n
            shape, sshape = (nb, block_size, n_kv, d), (nb, n_kv)
        else:
            self.table, shape, sshape = None, (B, self.room, n_kv, d), (B, per, n_kv)
        rb = lambda: torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8)
        self.k, self.v = rb(), rb()
        self.ks = torch.full(sshape, float("nan"))
        self.vs = self.ks.clone()
        self.geo = C.Geometry(block_size, self.table, self.room)

    def on(self, dev):
        """(k, v, ks, vs) on the device, and the block table (or None)."""
        return ([t.to(dev) for t in (self.k, self.v, self.ks, self.vs)],
                None if self.table is None else self.table.to(dev))

    def ref(self):
        """The reference's dict, flat."""
        flat = lambda t: C.decode_code(t.numpy()).reshape(-1, self.n_kv, self.d)
        sc = lambda t: t.double().numpy().reshape(-1, self.n_kv).copy()
        return {"k": flat(self.k), "v": flat(self.v), "ks": sc(self.ks), "vs": sc(self.vs)}

    def set_from(self, ref):
        """Takes the reference's state as this cache's."""
        for n in ("k", "v"):
            getattr(self, n).copy_(code_bytes(ref[n]).view(getattr(self, n).shape))
            s = getattr(self, n + "s")
            s.copy_(torch.from_numpy(ref[n + "s"]).float().view(s.shape))


def code_bytes(values):
    """e4m3 codes of e4m3 values (the sign of a zero kept)."""
    return torch.from_numpy(np.ascontiguousarray(values)).float().to(torch.float8_e4m3fn).view(
        torch.uint8)


def assert_cache(got, want_ref, before: Cache, what=""):
    """Device tensors (k, v, ks, vs) against the reference's state; what the
    reference left alone has to be the same bytes as before."""
    start = before.ref()
    for i, n in enumerate(("k", "v")):
        g = got[i].cpu()
        old = getattr(before, n)
        same = ((start[n] == want_ref[n]) & (np.signbit(start[n]) == np.signbit(want_ref[n]))) | (
            np.isnan(start[n]) & np.isnan(want_ref[n]))
        want = torch.where(torch.from_numpy(same).view(old.shape), old,
                           code_bytes(want_ref[n]).view(old.shape))
        nan = ((want & 127) == 127) & ((g & 127) == 127)       # a NaN's sign is free
        bad = (g != want) & ~nan
        assert not bad.any(), f"{what}: {int(bad.sum())} codes of {n} differ"
        gs, ws = got[2 + i].cpu().double().numpy().reshape(-1), want_ref[n + "s"].reshape(-1)
        assert np.array_equal(gs, ws, equal_nan=True), f"{what}: scales of {n} differ"


def rows(n_kv, total, d, seed, spread=2.0):
    """(n_kv, total, d) bf16 whose tokens differ in size by powers of e."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n_kv, total, d, generator=gen)
    return (x * torch.exp(spread * torch.randn(n_kv, total, 1, generator=gen))).to(torch.bfloat16)


def token_major(x):
    """(n_kv, total, d) to the reference's (total, n_kv, d) in float64."""
    return x.double().permute(1, 0, 2).numpy()


def decode_bound(q, k, v, scale, softcap=0.0, slopes=None, window_left=-1):
    """How far a decode's O and LSE may be from exact for one sequence: q (n_q,
    d), k, v (n, n_kv, d) float64, n > 0.  Worst case, counting u = 2^-23 (a
    step of fp32 arithmetic that may truncate) for every rounding:
      a score s_j: the d products' sum and six roundings (scales, change of
        base), (d + 6) u sum_i |q_i k_ji| scale; with soft-capping 8 u cap more
        (tanh within 4 ulp, its argument and product); an ALiBi bias 2 u |bias|;
      a weight: that, the exponential and the 22-bit product operand 8 u, and
        the subtraction of the reference 2 u (|s_j| + |s|max)        -> w_j
      O: sum p_j |v_j| (w_j + mean w), and a rounding for each step of 16 tokens,
        the merges and the division, (n / 16 + 32) u sum p_j |v_j|
      LSE: mean w, (n / 4 + 16) u for the sum's steps, 2 u |LSE|.
    Returns (bound of O (n_q, d), bound of LSE (n_q,))."""
    u = 2.0 ** -23
    n_q, d = q.shape
    n, g = k.shape[0], n_q // k.shape[1]
    lo = max(0, n - 1 - window_left) if window_left >= 0 else 0
    kr, vr = np.repeat(k[lo:], g, axis=1), np.repeat(v[lo:], g, axis=1)   # (tokens, n_q, d)
    s = scale * np.einsum("hd,nhd->hn", q, kr)
    w = (d + 6) * u * scale * np.einsum("hd,nhd->hn", np.abs(q), np.abs(kr))
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
        w = w + 8 * u * softcap
    if slopes is not None:
        bias = -np.asarray(slopes)[:, None] * np.arange(n - 1 - lo, -1, -1)[None]
        s = s + bias
        w = w + 2 * u * np.abs(bias)
    top = s.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(s - top).sum(axis=1))
    p = np.exp(s - lse[:, None])
    w = w + 8 * u + 2 * u * (np.abs(s) + np.abs(top))
    mean = (p * w).sum(axis=1)
    av = np.abs(vr)
    ob = np.einsum("hn,nhd->hd", p * (w + mean[:, None] + (n / 16 + 32) * u), av)
    return ob, mean + (n / 4 + 16) * u + 2 * u * np.abs(lse)
