"""Decode over an 8-bit cache (attn_decode_fp8_splitkv, attn_decode_fp8) against
the float64 oracle on the values that the cache stands for: the combined
result, every split's partials, the append, and a run of all the cache's
operators together."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
from exact_io_aware_order_gb300._lib import AttnError, status_codes
import oracle
from oracle import cache_fp8_ref as C
from cache_fp8_util import Cache, assert_cache, decode_bound, rows, token_major
from gpu_util import nan_like, split_ranges

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def filled(lens, n_kv, d, bs, paged, seed, room=None, spread=1.0):
    """A cache that the reference filled with lens[b] tokens, the rest random
    codes and NaN scales."""
    c = Cache(len(lens), n_kv, d, room or lens, bs, paged, seed=seed)
    ref = c.ref()
    total = max(1, sum(lens))
    k, v = rows(n_kv, total, d, seed + 1, spread=0.2), rows(n_kv, total, d, seed + 2, spread=spread)
    cu = np.concatenate([[0], np.cumsum(lens)])
    C.write(ref, c.geo, token_major(k), token_major(v), cu, [0] * len(lens))
    c.set_from(ref)
    return c


def queries(B, n_q, d, seed):
    return torch.randn(B, n_q, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def slopes_of(n_q):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)], dtype=torch.float32)


def reference(c, q, lens, scale, window=-1, softcap=0.0, slopes=None):
    kc, vc = C.values(c.ref(), c.geo, lens)
    sl = None if slopes is None else slopes.double().numpy()
    o, lse = oracle.decode(q, kc, vc, None, lens, scale, 0, window_left=window, softcap=softcap,
                           alibi_slopes=sl)
    bo, bl = np.zeros_like(o), np.zeros_like(lse)
    qd = q.double().numpy()
    for b, n in enumerate(lens):
        if n:
            bo[b], bl[b] = decode_bound(qd[b], kc[b, :n], vc[b, :n], scale, softcap, sl, window)
    return (o, lse), (bo, bl), (kc, vc)


def close(o, lse, want, bound, what):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    inf = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(lse), inf), f"{what}: -inf pattern of LSE differs"
    eo, el = np.abs(o - want[0]), np.abs(lse[~inf] - want[1][~inf])
    assert np.isfinite(o).all() and np.isfinite(lse[~inf]).all(), what
    assert (eo <= bound[0]).all(), f"{what}: O off by {eo.max():.3e}, {(eo / np.maximum(bound[0], 1e-300)).max():.2f} of the bound"
    assert (el <= bound[1][~inf]).all(), f"{what}: LSE off by {el.max():.3e}"


# (lens, splits, block size, head_dim, query heads, kv heads, paged, window, softcap, alibi)
CASES = [
    ([300], 2, 16, 128, 28, 4, True, -1, 0.0, False),
    ([0, 1, 15, 16, 17, 63, 64, 65], 3, 16, 128, 8, 2, True, -1, 0.0, False),
    ([63, 64, 65, 200, 0], 2, 16, 64, 4, 4, True, -1, 0.0, False),     # one query head a kv head
    ([5, 1000], 100, 16, 128, 16, 1, True, -1, 0.0, False),            # many empty splits
    ([1, 2, 3, 130], 1, 1, 128, 2, 1, True, -1, 0.0, False),           # one-token blocks
    ([777, 1], 5, 7, 64, 6, 3, True, -1, 0.0, False),                  # odd blocks
    ([777, 90], 3, 24, 128, 14, 2, True, -1, 0.0, False),              # blocks ending inside a tile
    ([500, 33], 4, 48, 256, 4, 2, True, -1, 0.0, False),
    ([4096], 1, 64, 128, 28, 4, True, -1, 0.0, False),
    ([0, 1, 17, 3000], 4, 32, 256, 16, 8, True, -1, 0.0, False),
    ([777, 1], 5, 7, 256, 4, 2, True, -1, 0.0, False),
    ([1, 300], 4, 16, 128, 8, 2, False, -1, 0.0, False),               # contiguous
    ([2049, 700], 33, 100, 64, 8, 2, False, -1, 0.0, False),
    ([400, 399], 2, 64, 256, 16, 2, False, -1, 0.0, False),
    ([600, 31], 3, 16, 128, 9, 1, True, -1, 0.0, False),               # 9 .. 64 heads a kv head
    ([600, 31], 3, 16, 64, 17, 1, True, -1, 0.0, False),
    ([600, 31], 3, 16, 128, 32, 1, True, -1, 0.0, False),
    ([300, 1], 2, 16, 256, 33, 1, True, -1, 0.0, False),
    ([700, 64], 3, 128, 128, 128, 2, True, -1, 0.0, False),
    ([900, 50, 0], 4, 16, 128, 8, 2, True, 100, 0.0, False),           # windows
    ([900, 50], 4, 10, 128, 48, 2, True, 0, 0.0, False),               # the query's own token only
    ([1500], 3, 64, 64, 8, 2, False, 333, 0.0, False),
    ([900, 50], 4, 24, 256, 16, 8, True, 255, 50.0, False),            # window and cap
    ([900, 50], 4, 16, 128, 28, 4, True, -1, 20.0, False),
    ([900, 50], 4, 16, 64, 48, 2, True, -1, 30.0, False),
    ([900, 50, 1], 4, 16, 128, 8, 2, True, -1, 0.0, True),             # ALiBi
    ([900, 50, 1], 4, 128, 64, 64, 2, True, 77, 0.0, True),
    ([1200], 5, 100, 256, 12, 4, False, -1, 0.0, True),
]


@pytest.mark.parametrize("lens,S,bs,d,n_q,n_kv,paged,window,softcap,alibi", CASES)
def test_decode(dev, lens, S, bs, d, n_q, n_kv, paged, window, softcap, alibi):
    B, scale = len(lens), d ** -0.5
    c = filled(lens, n_kv, d, bs, paged, seed=sum(lens) + S)
    q = queries(B, n_q, d, seed=S)
    sl = slopes_of(n_q) if alibi else None
    want, bound, (kc, vc) = reference(c, q, lens, scale, window, softcap, sl)
    tensors, table = c.on(dev)
    op, lp = nan_like((S, B, n_q, d), dev), nan_like((S, B, n_q), dev)
    kw = dict(scale=scale, window_left=window, softcap=softcap, block_size=bs,
              alibi_slopes=None if sl is None else sl.to(dev))
    attn.decode_fp8_splitkv(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S, o_partial=op,
                            lse_partial=lp, **kw)
    o, lse = attn.combine(op, lp)
    attn.check_device_status()
    what = f"lens={lens} S={S} bs={bs} d={d} {n_q}/{n_kv}"
    close(o, lse, want, bound, what + " combined")
    # Every split's partials: the same bound on its own tokens.
    ranges = [split_ranges(n, S, window) for n in lens]
    opr, lpr = oracle.decode_partials(q, kc, vc, None, lens, scale, 0, ranges, softcap=softcap,
                                      alibi_slopes=None if sl is None else sl.double().numpy())
    for s in range(S):
        bo, bl = np.zeros_like(opr[s]), np.zeros_like(lpr[s])
        for b, n in enumerate(lens):
            x, y = ranges[b][s]
            if y > x:
                far = (n - y) * (sl.double().numpy() if alibi else 0.0)   # |bias| of the last token
                bo[b], bl[b] = decode_bound(q[b].double().numpy(), kc[b, x:y], vc[b, x:y], scale,
                                            softcap, sl.double().numpy() if alibi else None)
                if alibi:  # and of the distance to the query, rounded once in each score
                    bl[b] = bl[b] + 4 * 2.0 ** -23 * far
                    bo[b] = bo[b] + 8 * 2.0 ** -23 * far[:, None] * np.abs(vc[b, x:y]).max()
        close(op[s], lp[s], (opr[s], lpr[s]), (bo, bl), what + f" split {s}")
    # One call, given or allocated outputs: the same bits.
    for out in (None, nan_like((B, n_q, d), dev)):
        o2, lse2 = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S, out=out,
                                   **kw)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    # The library's division: one block a pair, or shares of the tiles for the
    # blocks that this many tokens would take (a paged cache's max_kv_len).
    for most in ([300, 600, 4000, 100000] if paged else [None]):
        o3, lse3 = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, max_kv_len=most,
                                   out=nan_like((B, n_q, d), dev), lse=nan_like((B, n_q), dev), **kw)
        attn.check_device_status()
        close(o3, lse3, want, bound, what + f" shares for {most}")
    assert_cache(tensors, c.ref(), c, what)                 # only read


@pytest.mark.parametrize("B", [150, 1024, 1025])
def test_many_sequences_in_shares(dev, B):
    """Lengths from none to some hundred over many sequences (1025: beyond the
    shares' scan), first and last ones empty, two kv heads."""
    gen = torch.Generator().manual_seed(B)
    lens = (torch.randint(0, 3, (B,), generator=gen) * torch.randint(0, 160, (B,), generator=gen))
    lens[[0, 1, B - 1]] = 0
    lens[B // 2] = 900
    lens = lens.tolist()
    c = filled(lens, 2, 64, 16, True, seed=B)
    q = queries(B, 6, 64, 1)
    want, bound, _ = reference(c, q, lens, 0.125)
    tensors, table = c.on(dev)
    for most in (900, 20000):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, max_kv_len=most,
                                 scale=0.125, out=nan_like((B, 6, 64), dev),
                                 lse=nan_like((B, 6), dev))
        attn.check_device_status()
        close(o, lse, want, bound, f"{B} sequences, shares for {most}")
    none = torch.zeros(B, dtype=torch.int32, device=dev)
    o, lse = attn.decode_fp8(q.to(dev), *tensors, none, table, out=nan_like((B, 6, 64), dev),
                             lse=nan_like((B, 6), dev))
    attn.check_device_status()
    assert bool((o == 0).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("paged,n,n_q,n_kv,d", [(False, 30720, 28, 4, 128), (True, 30720, 8, 2, 64),
                                                (True, 100000, 4, 1, 128)])
def test_long_cache(dev, paged, n, n_q, n_kv, d):
    """The policy's split count, and one split."""
    c = filled([n], n_kv, d, 64, paged, seed=n, spread=0.5)
    q = queries(1, n_q, d, 1)
    want, bound, _ = reference(c, q, [n], d ** -0.5)
    tensors, table = c.on(dev)
    for S in (0, 1):
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32([n], dev), table, num_splits=S,
                                 block_size=64)
        attn.check_device_status()
        close(o, lse, want, bound, f"n={n} S={S}")
        # The weights' sum carries fp32 rounding only: the typical error is far
        # below the worst case.  2e-5 of the norm is 160 fp32 steps.
        e = np.linalg.norm(o.double().cpu().numpy() - want[0]) / np.linalg.norm(want[0])
        assert e <= 2e-5, (S, e)


def test_offsets_beyond_32_bits(dev):
    """A paged cache of more than 2^32 bytes: the sequence's blocks lie at
    its two ends."""
    n_kv, d, bs = 8, 128, 64
    nb = (1 << 32) // (bs * n_kv * d) + 40
    small = filled([300], n_kv, d, bs, True, seed=5)
    k = torch.zeros((nb, bs, n_kv, d), dtype=torch.uint8, device=dev)
    v = torch.zeros_like(k)
    ks, vs = torch.ones((nb, n_kv), device=dev), torch.ones((nb, n_kv), device=dev)
    where = [nb - 1, 0, nb - 2, nb // 2, nb - 3]
    for j, w in enumerate(where):
        src = int(small.table[0, j])
        k[w], v[w] = small.k[src].to(dev), small.v[src].to(dev)
        ks[w], vs[w] = small.ks[src].to(dev), small.vs[src].to(dev)
    q = queries(1, 32, d, 3)
    want, bound, _ = reference(small, q, [300], d ** -0.5)
    table = i32([where], dev)
    o, lse = attn.decode_fp8(q.to(dev), k, v, ks, vs, i32([300], dev), table, num_splits=2)
    attn.check_device_status()
    close(o, lse, want, bound, "far blocks")
    new = rows(n_kv, 1, d, 8).permute(1, 0, 2).contiguous()
    attn.cache_write_fp8(new.to(dev), new.to(dev), k, v, ks, vs, i32([300], dev), None, table)
    kr, _ = attn.cache_read_fp8(k, v, ks, vs, i32([0, 301], dev), 301, table)
    attn.check_device_status()
    ref = small.ref()
    C.write(ref, small.geo, new.double().numpy(), new.double().numpy(), [0, 1], [300])
    kw, _ = C.read(ref, small.geo, [0, 301], [0], 301)
    assert np.array_equal(kr.double().cpu().numpy(), kw)


@pytest.mark.parametrize("n_q", [8, 32])
def test_scales_far_apart(dev, n_q):
    """V's blocks between 2^-40 and 2^40 and queries far from 1: the result
    follows the largest values, and no weight over- or underflows."""
    lens, n_kv, d, bs = [400], 2, 128, 16
    c = filled(lens, n_kv, d, bs, True, seed=11)
    gen = torch.Generator().manual_seed(1)
    c.vs[torch.isfinite(c.vs)] = 2.0 ** torch.randint(-40, 41, c.vs[torch.isfinite(c.vs)].shape,
                                                      generator=gen).float()
    for amp, scale in ((1.0, 0.1), (2.0 ** 40, 0.1 * 2.0 ** -40), (2.0 ** -60, 0.1 * 2.0 ** 60)):
        q = (queries(1, n_q, d, 2).float() * amp).to(torch.bfloat16)
        want, bound, _ = reference(c, q, lens, scale)
        tensors, table = c.on(dev)
        for S in (1, 3, 0):
            o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=S,
                                     max_kv_len=2000, scale=scale)
            attn.check_device_status()
            # each weight's product with its scale keeps 22 bits, or 2^-36 of the largest
            floor = 2.0 ** -30 * max(lens) * 448.0 * 2.0 ** 40
            close(o, lse, want, (bound[0] + floor * 2.0 ** -3, bound[1]), f"amp={amp} S={S}")


def test_scales_need_not_be_powers_of_two(dev):
    lens, n_kv, d = [333], 2, 64
    c = filled(lens, n_kv, d, 16, True, seed=12)
    c.ks.mul_(1.37)
    c.vs.mul_(0.71)
    q = queries(1, 8, d, 2)
    want, bound, _ = reference(c, q, lens, d ** -0.5)
    tensors, table = c.on(dev)
    o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, num_splits=2)
    attn.check_device_status()
    close(o, lse, want, bound, "other scales")


@pytest.mark.parametrize("S", [3, 0])
@pytest.mark.parametrize("n_q", [8, 24])
def test_nan_in_live_and_masked_places(dev, n_q, S):
    """A NaN value in an attended token reaches the outputs that it belongs to
    (V: its own column; K: the whole row); left of the window, or past the
    end, it reaches nothing."""
    n, n_kv, d, bs, W = 200, 2, 64, 16, 50
    c = filled([n], n_kv, d, bs, True, seed=13)
    q = queries(1, n_q, d, 5)
    base, table = c.on(dev)
    run = lambda t, **kw: attn.decode_fp8(q.to(dev), *t, i32([n], dev), table, num_splits=S,
                                       max_kv_len=2000, **kw)
    o0, l0 = run(base)
    w0, wl0 = run(base, window_left=W)
    bad = [t.clone() for t in base]
    row = lambda t: (int(c.table[0, t // bs]), t % bs)
    for t in (3, n - 2 - W):                                # outside the window
        for x in bad[:2]:
            x[row(t)] = 0x7F
    w1, wl1 = run(bad, window_left=W)
    assert torch.equal(w1, w0) and torch.equal(wl1, wl0)
    bad = [t.clone() for t in base]
    b, s = row(n - 3)
    bad[1][b, s, 1, 9] = 0xFF                               # V of kv head 1, column 9
    o1, l1 = run(bad)
    hit = torch.zeros_like(o1, dtype=torch.bool)
    hit[:, n_q // 2:, 9] = True
    assert bool(torch.isnan(o1[hit]).all()) and torch.equal(o1[~hit], o0[~hit])
    assert torch.equal(l1, l0)
    bad = [t.clone() for t in base]
    bad[0][b, s, 0, 4] = 0x7F                               # K of kv head 0
    o2, l2 = run(bad)
    attn.check_device_status()
    assert bool(torch.isnan(o2[:, :n_q // 2]).all()) and bool(torch.isnan(l2[:, :n_q // 2]).all())
    assert torch.equal(o2[:, n_q // 2:], o0[:, n_q // 2:])


APPENDS = [
    ([0, 1, 15, 16, 31], 3, 16, 128, 8, 2, True, -1, 0.0, False),
    ([63, 64, 200], 2, 64, 64, 4, 4, True, -1, 0.0, False),
    ([0, 2, 3], 1, 1, 128, 2, 1, True, -1, 0.0, False),
    ([776, 0], 5, 7, 64, 6, 3, True, -1, 0.0, False),
    ([0, 99], 2, 300, 128, 28, 4, False, -1, 0.0, False),
    ([0, 31, 700], 4, 24, 256, 16, 8, True, 100, 30.0, False),
    ([500, 40], 4, 128, 64, 64, 2, True, -1, 0.0, True),
]


@pytest.mark.parametrize("lens,S,bs,d,n_q,n_kv,paged,window,softcap,alibi", APPENDS)
def test_append(dev, lens, S, bs, d, n_q, n_kv, paged, window, softcap, alibi):
    B, scale = len(lens), d ** -0.5
    c = filled(lens, n_kv, d, bs, paged, seed=sum(lens) + 3, room=[n + 1 for n in lens])
    q = queries(B, n_q, d, seed=S)
    sl = slopes_of(n_q) if alibi else None
    kn = rows(n_kv, B, d, 5, spread=1.5).permute(1, 0, 2).contiguous()
    vn = rows(n_kv, B, d, 6, spread=1.5).permute(1, 0, 2).contiguous()
    tensors, table = c.on(dev)
    kw = dict(scale=scale, window_left=window, softcap=softcap, block_size=bs,
              alibi_slopes=None if sl is None else sl.to(dev), num_splits=S)
    o, lse = attn.decode_append_fp8(q.to(dev), kn.to(dev), vn.to(dev), *tensors, i32(lens, dev),
                                    table, **kw)
    attn.check_device_status()
    want = c.ref()
    C.write(want, c.geo, kn.double().numpy(), vn.double().numpy(), list(range(B + 1)), lens)
    assert_cache(tensors, want, c, f"append {lens}")
    after = [n + 1 for n in lens]
    c.set_from(want)
    ref, bound, _ = reference(c, q, after, scale, window, softcap, sl)
    close(o, lse, ref, bound, f"append {lens}")
    # The same as the write and the decode apart, bit for bit.
    o2, lse2 = attn.decode_fp8(q.to(dev), *tensors, i32(after, dev), table, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # Again (the token is there already: the same bytes), in shares.
    kw["num_splits"] = 0
    o3, lse3 = attn.decode_append_fp8(q.to(dev), kn.to(dev), vn.to(dev), *tensors, i32(lens, dev),
                                      table, max_kv_len=3000 if paged else None, **kw)
    attn.check_device_status()
    close(o3, lse3, ref, bound, f"append {lens} in shares")
    assert_cache(tensors, want, c, f"append {lens} again")


def test_append_to_a_full_cache_is_flagged_and_not_written(dev):
    c = filled([64, 10], 1, 64, 16, False, seed=1, room=[64, 64])
    tensors, _ = c.on(dev)
    new = rows(1, 2, 64, 1).permute(1, 0, 2).contiguous()
    q = queries(2, 4, 64, 1)
    o, lse = attn.decode_append_fp8(q.to(dev), new.to(dev), new.to(dev), *tensors,
                                    i32([64, 10], dev), block_size=16, num_splits=2)
    with pytest.raises(AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]
    want = c.ref()
    C.write(want, c.geo, new.double().numpy(), new.double().numpy(), [0, 0, 0], [0, 0])
    C.write(want, C.Geometry(16, None, 64), new.double().numpy()[1:], new.double().numpy()[1:],
            [0, 0, 1], [64, 10])
    assert_cache(tensors, want, c, "full")
    c.set_from(want)
    ref, bound, _ = reference(c, q, [64, 11], 64 ** -0.5)
    close(o, lse, ref, bound, "full")                       # the full one attends what it holds


def test_bad_block_is_flagged_in_bounds(dev):
    c = filled([100], 2, 128, 16, True, seed=2)
    tensors, table = c.on(dev)
    q = queries(1, 8, 128, 1).to(dev)
    good, _ = attn.decode_fp8(q, *tensors, i32([100], dev), table, num_splits=2)
    for bad, S in ((-1, 2), (c.k.shape[0], 0), (1 << 30, 1)):
        t = table.clone()
        t[0, 3] = bad
        attn.decode_fp8(q, *tensors, i32([100], dev), t, num_splits=S, max_kv_len=1000)
        with pytest.raises(AttnError) as e:
            attn.check_device_status()
        assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]
    for n, S in ((-5, 2), (113, 0), (1 << 30, 1), (-1, 0)):  # lengths outside [0, 112]
        attn.decode_fp8(q, *tensors, i32([n], dev), table, num_splits=S, max_kv_len=1000)
        with pytest.raises(AttnError) as e:
            attn.check_device_status()
        assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]
    again, _ = attn.decode_fp8(q, *tensors, i32([100], dev), table, num_splits=2)
    attn.check_device_status()
    assert torch.equal(good, again)


def test_prompt_steps_and_read_back_together(dev):
    """A serving run: two packed prompts written, decode steps appended, the
    sequences read back; the decode over the cache equals the framework's bf16
    decode over what is read back, and prefill's last row over it, up to those
    kernels' rounding of the weights to bf16: half a step, 2^-8 of each weight,
    so 2^-8 sum p |v| (the values reach 32 here)."""
    n_q, n_kv, d, bs, steps = 8, 2, 128, 16, 40
    prompt = [75, 130]
    c = Cache(2, n_kv, d, [n + steps for n in prompt], bs, True, seed=21)
    tensors, table = c.on(dev)
    k = rows(n_kv, sum(prompt), d, 1, spread=0.5)
    v = rows(n_kv, sum(prompt), d, 2, spread=0.5)
    lens = i32([0, 0], dev)
    attn.cache_write_fp8(k.to(dev), v.to(dev), *tensors, lens, i32([0, 75, 205], dev), table)
    lens += i32(prompt, dev)
    want = c.ref()
    C.write(want, c.geo, token_major(k), token_major(v), [0, 75, 205], [0, 0])
    for t in range(steps):
        kn = rows(n_kv, 2, d, 50 + t, spread=1.0).permute(1, 0, 2).contiguous()
        q = queries(2, n_q, d, 300 + t)
        o, lse = attn.decode_append_fp8(q.to(dev), kn.to(dev), (-kn).to(dev), *tensors, lens, table)
        C.write(want, c.geo, kn.double().numpy(), -kn.double().numpy(), [0, 1, 2],
                [n + t for n in prompt])
        lens += 1
    attn.check_device_status()
    assert_cache(tensors, want, c, "run")
    c.set_from(want)
    total = [n + steps for n in prompt]
    ref, bound, (kv, vv) = reference(c, q, total, d ** -0.5)
    close(o, lse, ref, bound, "last step")
    # Read back: the framework's bf16 attention over the same values.
    size, _ = oracle.decode(q, kv, np.abs(vv), None, total, d ** -0.5, 0)
    bound16 = (bound[0] + 2.0 ** -8 * size, np.full_like(bound[1], 1e-3))
    cu = i32([0, total[0], sum(total)], dev)
    kr, vr = attn.cache_read_fp8(*tensors, cu, sum(total), table)
    L = max(total)
    kc = torch.zeros((2, L, n_kv, d), dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    for b in range(2):
        one = i32([0, total[b]], dev)
        attn.cache_read_fp8(*tensors, one, total[b], table[b:b + 1],
                            k_out=kc[b, :total[b]].transpose(0, 1),
                            v_out=vc[b, :total[b]].transpose(0, 1))
        a = int(cu[b])
        assert torch.equal(kc[b, :total[b]].transpose(0, 1), kr[:, a:a + total[b]])
    o16, l16 = attn.decode(q.to(dev), kc, vc, lens)
    qq = torch.zeros((n_q, sum(total), d), dtype=torch.bfloat16, device=dev)
    for b in range(2):
        qq[:, int(cu[b + 1]) - 1] = q[b].to(dev)
    op, lp = attn.prefill_varlen(qq, kr, vr, cu)
    attn.check_device_status()
    close(o16, l16, ref, bound16, "bf16 decode over what was read back")
    last = [int(x) - 1 for x in cu[1:]]
    close(op[:, last].transpose(0, 1), lp[:, last].transpose(0, 1), ref, bound16,
          "prefill over what was read back")


def test_other_stream_and_its_workspace(dev):
    """stream= with allocated outputs and workspace: the workspace belongs to
    that stream, so allocations on the caller's stream made right after the
    call do not disturb it."""
    lens = [3000] * 4
    c = filled([3000] * 4, 2, 128, 64, True, seed=31)
    tensors, table = c.on(dev)
    q = queries(4, 16, 128, 1).to(dev)
    ln = i32(lens, dev)
    want = attn.decode_fp8(q, *tensors, ln, table, num_splits=8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for _ in range(5):
            torch.cuda._sleep(100000)
            o, lse = attn.decode_fp8(q, *tensors, ln, table, num_splits=8, stream=stream)
            junk = [torch.full((8 * 4 * 16 * 129,), float("nan"), device=dev) for _ in range(4)]
            side.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            del junk
    attn.check_device_status()


def test_two_streams_at_once(dev):
    c = filled([2000, 100], 2, 128, 16, True, seed=32)
    tensors, table = c.on(dev)
    q = [queries(2, 8, 128, s).to(dev) for s in range(2)]
    ln = i32([2000, 100], dev)
    want = [attn.decode_fp8(x, *tensors, ln, table) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, s in zip(q, streams):
            got.append(attn.decode_fp8(x, *tensors, ln, table, stream=s))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_captured_steps_replay(dev):
    """Decode steps captured into one graph (append, attend, count up), and a
    second graph of the same calls with its own buffers, replayed in turn."""
    n_kv, n_q, d, bs, B = 2, 8, 128, 16, 3
    start = [5, 16, 130]
    c = filled(start, n_kv, d, bs, True, seed=41, room=[n + 8 for n in start])
    q, kn = queries(B, n_q, d, 1).to(dev), rows(n_kv, B, d, 2).permute(1, 0, 2).contiguous().to(dev)
    eager, table = c.on(dev)
    lens = i32(start, dev)
    want = []
    for _ in range(6):
        want.append([t.clone() for t in attn.decode_append_fp8(q, kn, kn, *eager, lens, table,
                                                               num_splits=4)])
        lens += 1
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        mine, ln = c.on(dev)[0], i32(start, dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = attn.decode_append_fp8(q, kn, kn, *mine, ln, table, num_splits=4)
            ln += 1
        graphs.append((g, out, mine, ln))
    for i in range(6):
        for g, out, mine, ln in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out, mine, ln in graphs:
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1]), i
    for g, out, mine, ln in graphs:
        for a, b in zip(mine, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(ln, lens)
    attn.check_device_status()


def test_same_call_same_bits(dev):
    c = filled([5000, 10, 777], 2, 128, 16, True, seed=51)
    tensors, table = c.on(dev)
    q = queries(3, 28, 128, 4)[:, :14].contiguous().to(dev)
    first = attn.decode_fp8(q, *tensors, i32([5000, 10, 777], dev), table)
    for _ in range(5):
        o, lse = attn.decode_fp8(q, *tensors, i32([5000, 10, 777], dev), table)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n_q", [8, 24])
def test_query_that_is_not_finite(dev, n_q, bad):
    """An infinity or a NaN in q makes its own row NaN and no other."""
    c = filled([300], 2, 64, 16, True, seed=61)
    tensors, table = c.on(dev)
    q = queries(1, n_q, 64, 7).to(dev)
    for S in (1, 0):
        kw = dict(num_splits=S, max_kv_len=3000)
        want = attn.decode_fp8(q, *tensors, i32([300], dev), table, **kw)
        q2 = q.clone()
        q2[0, 3, 17] = bad
        o, lse = attn.decode_fp8(q2, *tensors, i32([300], dev), table, **kw)
        attn.check_device_status()
        assert bool(torch.isnan(o[0, 3]).all()) and bool(torch.isnan(lse[0, 3]))
        rest = [h for h in range(n_q) if h != 3]
        assert torch.equal(o[0, rest], want[0][0, rest])
        assert torch.equal(lse[0, rest], want[1][0, rest])


def test_tiny_and_zero_queries(dev):
    """Rows of zeros, and of bf16 subnormals: uniform weights."""
    c = filled([77], 2, 128, 16, True, seed=62)
    tensors, table = c.on(dev)
    q = queries(1, 8, 128, 8)
    q[0, 0] = 0.0
    q[0, 1] = 1e-39
    q[0, 5] = -0.0
    want, bound, _ = reference(c, q, [77], 0.1)
    o, lse = attn.decode_fp8(q.to(dev), *tensors, i32([77], dev), table, scale=0.1)
    attn.check_device_status()
    close(o, lse, want, bound, "tiny queries")


def test_queries_with_one_large_value(dev):
    """A row whose largest value is 2^12 times the others: the two e4m3 terms
    still carry the others (2^-15 of the maximum and above exactly)."""
    c = filled([333], 2, 128, 32, True, seed=63)
    tensors, table = c.on(dev)
    q = queries(1, 8, 128, 9)
    q[0, :, 40] = 0.0
    big = q.clone()
    big[0, 2, 40] = 4096.0
    scale = 0.05
    want, bound, (kv, vv) = reference(c, big, [333], scale)
    # below 2^-15 of the row's maximum a value of q may be off by 2^-23 of it
    d_s = scale * 2.0 ** -23 * 4096.0 * np.abs(kv[0]).sum(axis=2).max()
    o, lse = attn.decode_fp8(big.to(dev), *tensors, i32([333], dev), table, scale=scale)
    attn.check_device_status()
    extra = 2 * d_s * np.abs(vv[0]).max()
    close(o, lse, want, (bound[0] + extra, bound[1] + d_s), "one large value")


def test_captured_shares_follow_the_lengths(dev):
    """A step captured with num_splits 0 divides the tokens by the lengths of
    the replay, not of the capture: sequences that grow, and ones that are
    replaced by others between replays (an empty one among them)."""
    n_kv, n_q, d, bs, B = 2, 8, 128, 16, 4
    at = [[5, 16, 130, 1000], [1000, 0, 700, 3], [0, 0, 0, 0], [1000, 1000, 1000, 1000]]
    c = filled([1000] * B, n_kv, d, bs, True, seed=42, room=[1001] * B)
    q = queries(B, n_q, d, 1).to(dev)
    tensors, table = c.on(dev)
    lens = i32(at[0], dev)
    call = lambda: attn.decode_fp8(q, *tensors, lens, table, max_kv_len=4000)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for now in at + at[:1]:
        lens.copy_(i32(now, dev))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b), now
        want, bound, _ = reference(c, q.cpu(), now, d ** -0.5)
        close(*got, want, bound, str(now))
    attn.check_device_status()


FIRST_CALL = """
import torch
import exact_io_aware_order_gb300 as attn
dev = torch.device("cuda", 0)
k = torch.zeros(8, 16, 2, 64, dtype=torch.uint8, device=dev)
v, ks = k.clone(), torch.zeros(8, 2, device=dev)
vs, table = ks.clone(), torch.arange(8, dtype=torch.int32, device=dev).view(1, 8)
x = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=dev)
lens = torch.zeros(1, dtype=torch.int32, device=dev)
q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=dev)
attn.cache_write_fp8(x, x, k, v, ks, vs, lens, None, table)
lens += 1
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, lse = attn.decode_append_fp8(q, x, x, k, v, ks, vs, lens, table, max_kv_len=5000)
g.replay()
torch.cuda.synchronize()
attn.check_device_status()
assert bool((o == 1).all()), o
print("replayed")
"""


def test_first_decode_of_a_process_is_captured():
    """Nothing of the decode's set-up gets in the way of a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stdout + r.stderr


def test_two_threads_at_once(dev):
    """The calls drop the interpreter's lock while they launch."""
    lens = [2000, 100]
    c = filled(lens, 2, 128, 16, True, seed=33)
    tensors, table = c.on(dev)
    q = [queries(2, 8, 128, s).to(dev) for s in range(2)]
    ln = i32(lens, dev)
    want = [attn.decode_fp8(x, *tensors, ln, table) for x in q]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i].append(attn.decode_fp8(q[i], *tensors, ln, table))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 50
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("n_q", [4, 20])
@pytest.mark.parametrize("S", [2, 0])
def test_scales_of_zero(dev, n_q, S):
    """A cache that is zero as it was allocated, scales too, and blocks of zeros
    among written ones: values of 0, whatever the codes' scale."""
    lens = [3000, 33]
    q = queries(2, n_q, 64, 3)
    kw = dict(num_splits=S, max_kv_len=3000)
    for some in (False, True):
        c = filled(lens, 2, 64, 16, True, seed=71)
        zero = torch.zeros(len(c.ks), dtype=torch.bool)
        zero[::2] = True
        zero = zero if some else torch.ones_like(zero)
        for codes, scales in ((c.k, c.ks), (c.v, c.vs)):
            codes[zero], scales[zero] = 0, 0.0
        tensors, table = c.on(dev)
        want, bound, _ = reference(c, q, lens, 0.125)
        o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, **kw)
        attn.check_device_status()
        close(o, lse, want, bound, f"zero scales, some {some}")
        if not some:
            assert not o.any()


@pytest.mark.parametrize("B,n_kv,d,lo,hi", [
    (36, 8, 64, 300, 300),     # a block for each pair
    (36, 8, 64, 10, 2500),     # too uneven for that
    (40, 1, 128, 0, 900),      # more sequences than a warp has lanes, several blocks a pair
    (33, 2, 256, 500, 600),
    (304, 1, 128, 33, 64),     # as many pairs as blocks
    (305, 1, 128, 33, 64),     # one more
    (2, 3, 128, 31, 33),       # fewer tiles than pairs have blocks
])
def test_every_division(dev, B, n_kv, d, lo, hi):
    """num_splits 0 over batches for which each pair takes one block, several,
    or parts of shared ones."""
    gen = np.random.default_rng(B)
    lens = [int(n) for n in gen.integers(lo, hi + 1, B)]
    n_q = 2 * n_kv
    c = filled(lens, n_kv, d, 16, True, seed=B)
    tensors, table = c.on(dev)
    q = queries(B, n_q, d, 5)
    want, bound, _ = reference(c, q, lens, d ** -0.5)
    o, lse = attn.decode_fp8(q.to(dev), *tensors, i32(lens, dev), table, max_kv_len=8192)
    attn.check_device_status()
    close(o, lse, want, bound, f"{B} x {n_kv}, {lo} to {hi}")


@pytest.mark.parametrize("B,n_kv", [(1, 2), (6, 2), (40, 16)])
def test_steps_in_a_row(dev, B, n_kv):
    """Steps one behind the other, each attending what the one before wrote, with
    scales that grow in the block being filled, against the write, a pause and the
    decode (a decode of a small step starts while its write runs)."""
    d, bs, steps = 64, 16, 24
    start = [(7 * b) % 23 for b in range(B)]
    c = filled(start, n_kv, d, bs, True, seed=81, room=[n + steps for n in start])
    apart, table = c.on(dev)
    joined = [t.clone() for t in apart]
    q = queries(B, 4 * n_kv, d, 1).to(dev)
    new = [(rows(n_kv, B, d, 100 + i).permute(1, 0, 2) * 2.0 ** (i / 2)).contiguous().to(dev)
           for i in range(steps)]
    want = []
    lens = i32(start, dev)
    for x in new:
        attn.cache_write_fp8(x, x, *apart, lens, None, table)
        lens += 1
        torch.cuda.synchronize()
        want.append(attn.decode_fp8(q, *apart, lens, table, max_kv_len=3000))
        torch.cuda.synchronize()
    got = []
    lens = [i32([n + i for n in start], dev) for i in range(steps)]
    torch.cuda.synchronize()
    for x, ln in zip(new, lens):
        got.append(attn.decode_append_fp8(q, x, x, *joined, ln, table, max_kv_len=2999))
    torch.cuda.synchronize()
    attn.check_device_status()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i
    for a, b in zip(joined, apart):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
