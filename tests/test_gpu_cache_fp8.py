"""The 8-bit cache's write and read (attn_cache_write_fp8, attn_cache_read_fp8)
against the float64 reference.  Both are exact but for the one rounding that
defines a code, so codes and scales are compared byte for byte, and so is
everything that a call has to leave alone (codes and scales start as random
bytes and NaN)."""

import numpy as np
import pytest
import torch

import exact_io_aware_order_gb300 as attn
from exact_io_aware_order_gb300._lib import AttnError, status_codes
from oracle import cache_fp8_ref as C
from cache_fp8_util import Cache, assert_cache, rows, token_major

pytestmark = pytest.mark.gpu


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def write_both(c, dev, k, v, lens, cu, tensors=None, table=None):
    """One write on the device and in the reference, from c's state."""
    if tensors is None:
        tensors, table = c.on(dev)
    attn.cache_write_fp8(k.to(dev), v.to(dev), *tensors, i32(lens, dev), cu.to(dev), table,
                         block_size=c.bs)
    ref = c.ref()
    C.write(ref, c.geo, token_major(k), token_major(v), cu.tolist(), lens)
    return tensors, table, ref


# (cached tokens, new tokens, block size, head_dim, kv heads, paged)
WRITES = [
    ([0], [1], 16, 128, 1, True),
    ([0, 5, 16, 31, 40], [16, 11, 1, 3, 0], 16, 128, 2, True),
    ([0, 7, 63], [200, 1, 130], 64, 64, 3, True),
    ([3, 0, 100], [70, 45, 9], 24, 256, 2, True),
    ([0, 2], [9, 5], 1, 128, 4, True),              # one token a block
    ([5, 6, 0], [40, 1, 13], 7, 64, 5, True),       # odd blocks
    ([130, 0], [300, 1000], 256, 128, 2, True),     # blocks read twice
    ([0, 999], [1500, 2], 1000, 64, 1, False),      # a last block cut short
    ([0, 17, 64], [33, 48, 1], 16, 128, 2, False),
    ([1, 0], [99, 100], 32, 256, 3, False),
]


@pytest.mark.parametrize("lens,new,bs,d,n_kv,paged", WRITES)
def test_write(dev, lens, new, bs, d, n_kv, paged):
    c = Cache(len(lens), n_kv, d, [a + b for a, b in zip(lens, new)], bs, paged, seed=sum(new))
    # What is cached already, written by the reference.
    ref = c.ref()
    old = rows(n_kv, max(1, sum(lens)), d, seed=1)
    C.write(ref, c.geo, token_major(old), token_major(-old), cu_of(lens).tolist(), [0] * len(lens))
    c.set_from(ref)
    total = sum(new)
    k, v = rows(n_kv, total, d, seed=2, spread=4.0), rows(n_kv, total, d, seed=3)
    got, _, want = write_both(c, dev, k, v, lens, cu_of(new))
    attn.check_device_status()
    assert_cache(got, want, c, f"write {lens}+{new} bs={bs}")


def test_write_many_sequences(dev):
    """More sequences than one search step spans, some without rows."""
    gen = torch.Generator().manual_seed(5)
    B = 1500
    new = (torch.randint(0, 4, (B,), generator=gen) * torch.randint(0, 9, (B,), generator=gen)).tolist()
    lens = torch.randint(0, 40, (B,), generator=gen).tolist()
    c = Cache(B, 1, 64, [a + b for a, b in zip(lens, new)], 16, True, seed=7)
    ref = c.ref()
    old = rows(1, sum(lens), 64, seed=4)
    C.write(ref, c.geo, token_major(old), token_major(old), cu_of(lens).tolist(), [0] * B)
    c.set_from(ref)
    k, v = rows(1, sum(new), 64, seed=8), rows(1, sum(new), 64, seed=9)
    got, _, want = write_both(c, dev, k, v, lens, cu_of(new))
    attn.check_device_status()
    assert_cache(got, want, c, "1500 sequences")


@pytest.mark.parametrize("paged,bs,d", [(True, 16, 128), (False, 5, 64), (True, 64, 256)])
def test_token_by_token(dev, paged, bs, d):
    """One token a call, sizes rising over five powers of ten: the blocks'
    scales grow and their codes move with them."""
    N, n_kv, B = 70, 2, 2
    c = Cache(B, n_kv, d, [N, N], bs, paged, seed=bs)
    tensors, table = c.on(dev)
    want = c.ref()
    for t in range(N):
        k = rows(n_kv, B, d, seed=100 + t).float() * 10.0 ** (t / 14)
        k = k.to(torch.bfloat16).permute(1, 0, 2).contiguous()       # (B, n_kv, d)
        v = (-0.5 * k.float()).to(torch.bfloat16)
        attn.cache_write_fp8(k.to(dev), v.to(dev), *tensors, i32([t, t], dev), None, table,
                             block_size=bs)
        C.write(want, c.geo, k.double().numpy(), v.double().numpy(), [0, 1, 2], [t, t])
    attn.check_device_status()
    assert_cache(tensors, want, c, "token by token")


def test_division_into_calls_does_not_matter_without_growth(dev):
    c = Cache(1, 2, 128, [200], 16, True, seed=3)
    x = torch.randn(2, 200, 128, generator=torch.Generator().manual_seed(1))
    x[:, ::1, 0] = 4.0 * x.abs().amax()                 # every token has the same maximum
    x = x.to(torch.bfloat16).to(dev)
    whole, table = c.on(dev)
    attn.cache_write_fp8(x, x, *whole, i32([0], dev), i32([0, 200], dev), table)
    parts, _ = c.on(dev)
    at = 0
    for n in (1, 14, 2, 50, 16, 117):
        part = x[:, at:at + n]
        attn.cache_write_fp8(part, part, *parts, i32([at], dev), i32([0, n], dev), table)
        at += n
    attn.check_device_status()
    for a, b in zip(whole, parts):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_values_at_the_limits(dev):
    """Infinities, NaN, zeros, subnormals, the largest bf16, scales at both
    ends of their range."""
    inf, nan = float("inf"), float("nan")
    n_kv, d, bs = 1, 64, 16
    x = torch.zeros(n_kv, 9 * bs, d)
    x[0, 0:16] = torch.randn(16, d, generator=torch.Generator().manual_seed(0))
    x[0, 3, 5], x[0, 4, 6], x[0, 5, 7] = inf, -inf, nan      # block 0
    x[0, 16:32] = 0.0                                        # block 1: zeros
    x[0, 17, 1] = -0.0
    x[0, 32:48] = 1e-39                                      # block 2: bf16 subnormals
    x[0, 48:64] = 3.3e38                                     # block 3: beyond 448 * 2^60
    x[0, 50, 2] = 1.0
    x[0, 64:80] = nan                                        # block 4: nothing finite
    x[0, 70, 3] = inf
    x[0, 80:96] = 448.0                                      # block 5: an edge of a scale
    x[0, 96:112] = 450.0                                     # block 6: one step above it
    x[0, 112:128] = 448.0 * 2.0 ** -60                       # block 7: the smallest scale's edge
    x[0, 128:144] = 448.0 * 2.0 ** 60                        # block 8: the largest scale's edge
    k = x.to(torch.bfloat16)
    for bs_ in (bs, 48):
        c = Cache(1, n_kv, d, [9 * bs], bs_, True, seed=9)
        got, _, want = write_both(c, dev, k, -k, [0], cu_of([9 * bs]))
        attn.check_device_status()
        assert_cache(got, want, c, f"limits bs={bs_}")


def test_strided_rows(dev):
    """Keys and values as views of a fused projection (total, (n_q + 2 n_kv) d)
    and of a (total, n_kv, d) tensor."""
    n_q, n_kv, d, total = 8, 2, 128, 75
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn(total, (n_q + 2 * n_kv) * d, generator=gen).to(torch.bfloat16).to(dev)
    heads = qkv.view(total, n_q + 2 * n_kv, d)
    k, v = heads[:, n_q:n_q + n_kv].transpose(0, 1), heads[:, n_q + n_kv:].transpose(0, 1)
    assert not k.is_contiguous()
    c = Cache(2, n_kv, d, [30, 60], 16, True, seed=1)
    cu, lens = i32([0, 20, 75], dev), i32([10, 5], dev)
    ref = c.ref()
    old = rows(n_kv, 15, d, seed=6)
    C.write(ref, c.geo, token_major(old), token_major(old), [0, 10, 15], [0, 0])
    c.set_from(ref)
    a, table = c.on(dev)
    b, _ = c.on(dev)
    attn.cache_write_fp8(k, v, *a, lens, cu, table)
    attn.cache_write_fp8(k.contiguous(), v.contiguous(), *b, lens, cu, table)
    attn.check_device_status()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # Read back into views with gaps: (total, n_kv, d) in a wider tensor.
    wide = torch.full((total, 3 * n_kv, d), 7.0, dtype=torch.bfloat16, device=dev)
    ko, vo = wide[:, :n_kv].transpose(0, 1), wide[:, 2 * n_kv:].transpose(0, 1)
    attn.cache_read_fp8(*a, cu, total, table, starts=lens, k_out=ko, v_out=vo)
    kr, vr = attn.cache_read_fp8(*a, cu, total, table, starts=lens)
    attn.check_device_status()
    assert torch.equal(ko, kr) and torch.equal(vo, vr)
    assert bool((wide[:, n_kv:2 * n_kv] == 7.0).all())
    # A value is within half an e4m3 step (2^-4 of it, or 2^-10 of the scale).
    big = max(float(a[2][torch.isfinite(a[2])].max()), 0)
    assert bool(((kr.float() - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * big).all())


@pytest.mark.parametrize("bs,d,n_kv,paged", [(16, 128, 2, True), (64, 64, 3, True),
                                             (24, 256, 1, False), (1, 128, 1, True),
                                             (300, 64, 2, False), (7, 128, 4, True)])
def test_read(dev, bs, d, n_kv, paged):
    """Any part of each sequence, rows behind the last sequence left alone,
    NaN codes back as NaN."""
    lens = [40, 0, 333, 17, 64]
    c = Cache(5, n_kv, d, lens, bs, paged, seed=bs)
    ref = c.ref()
    old = rows(n_kv, sum(lens), d, seed=3, spread=8.0)
    old[0, 7, 3] = float("nan")
    C.write(ref, c.geo, token_major(old), token_major(-old), cu_of(lens).tolist(), [0] * 5)
    c.set_from(ref)
    tensors, table = c.on(dev)
    for starts, n in (([0] * 5, lens), ([3, 0, 100, 16, 1], [20, 0, 233, 1, 63])):
        total = sum(n) + 5
        out = [torch.full((n_kv, total, d), 3.0, dtype=torch.bfloat16, device=dev) for _ in "kv"]
        attn.cache_read_fp8(*tensors, cu_of(n).to(dev), total, table,
                            starts=None if starts == [0] * 5 else i32(starts, dev), block_size=bs,
                            k_out=out[0], v_out=out[1])
        attn.check_device_status()
        want = C.read(ref, c.geo, cu_of(n).tolist(), starts, total)
        for g, w in zip(out, want):
            w[:, sum(n):] = 3.0
            assert np.array_equal(g.double().cpu().numpy(), w, equal_nan=True)


def test_read_of_written_equals_the_value_rounded_once(dev):
    """Write, read, write again: the second write changes nothing (a value
    read back is its own code)."""
    c = Cache(1, 2, 128, [500], 32, True, seed=4)
    tensors, table = c.on(dev)
    k, v = rows(2, 500, 128, 1).to(dev), rows(2, 500, 128, 2).to(dev)
    cu, zero = i32([0, 500], dev), i32([0], dev)
    attn.cache_write_fp8(k, v, *tensors, zero, cu, table)
    kr, vr = attn.cache_read_fp8(*tensors, cu, 500, table)
    again = [t.clone() for t in tensors]
    attn.cache_write_fp8(kr, vr, *again, zero, cu, table)
    kr2, vr2 = attn.cache_read_fp8(*again, cu, 500, table)
    attn.check_device_status()
    assert torch.equal(kr, kr2) and torch.equal(vr, vr2)


# ---- what the kernels report ----

def flagged(dev):
    with pytest.raises(AttnError) as e:
        attn.check_device_status()
    assert e.value.status == status_codes()["ATTN_ERR_DEVICE"]
    attn.check_device_status()                           # read and cleared


@pytest.mark.parametrize("bad", ["too_long", "negative", "block", "cu_order", "cu_total"])
def test_bad_lists_are_flagged(dev, bad):
    """A bad sequence is flagged and not written; the good one beside it is
    (where its rows are still known)."""
    lens, new = [4, 10], [6, 20]
    c = Cache(2, 1, 64, [10, 30], 16, True, seed=2)
    ref = c.ref()
    old = rows(1, 14, 64, 1)
    C.write(ref, c.geo, token_major(old), token_major(old), [0, 4, 14], [0, 0])
    c.set_from(ref)
    tensors, table = c.on(dev)
    cu = [0, 6, 26]
    want = c.ref()
    k = rows(1, 26, 64, 2)
    if bad == "too_long":
        lens = [4, 13]                                   # 13 + 20 > 32
        C.write(want, c.geo, token_major(k), token_major(k), [0, 6, 6], lens)
    elif bad == "negative":
        lens = [4, -1]
        C.write(want, c.geo, token_major(k), token_major(k), [0, 6, 6], [4, 0])
    elif bad == "block":
        table[1, 1] = c.k.shape[0]                       # positions 16 .. 29 of sequence 1
        C.write(want, c.geo, token_major(k), token_major(k), [0, 6, 12], lens)
    elif bad == "cu_order":
        cu, lens = [0, 26, 6], [30, 10]                  # sequence 0 does not fit, 1 has no rows
    elif bad == "cu_total":
        cu = [0, 6, 27]                                  # clamped to 26
        C.write(want, c.geo, token_major(k), token_major(k), [0, 6, 26], lens)
    attn.cache_write_fp8(k.to(dev), k.to(dev), *tensors, i32(lens, dev), i32(cu, dev), table)
    flagged(dev)
    assert_cache(tensors, want, c, bad)
    # The read: the same lists, nothing of a bad sequence comes back.
    out = torch.full((1, 26, 64), 5.0, dtype=torch.bfloat16, device=dev)
    attn.cache_read_fp8(*tensors, i32(cu, dev), 26, table, starts=i32(lens, dev), k_out=out,
                        v_out=out.clone())
    flagged(dev)
    if bad in ("too_long", "negative"):
        assert bool((out[:, 6:] == 5.0).all())
    if bad == "block":
        assert bool((out[:, 12:] == 5.0).all())


def test_python_refusals(dev):
    c = Cache(2, 2, 128, [32, 32], 16, True)
    (k, v, ks, vs), table = c.on(dev)
    x = torch.zeros(2, 10, 128, dtype=torch.bfloat16, device=dev)
    lens, cu = i32([0, 0], dev), i32([0, 5, 10], dev)
    ok = dict(kv_lens=lens, cu_seqlens=cu, block_table=table)
    W = attn.cache_write_fp8
    with pytest.raises(TypeError):
        W(x.float(), x, k, v, ks, vs, **ok)
    with pytest.raises(TypeError):
        W(x, x, k.view(torch.int8), v, ks, vs, **ok)
    with pytest.raises(TypeError):
        W(x, x, k, v, ks.half(), vs, **ok)
    with pytest.raises(TypeError):
        W(x, x, k, v, ks, vs, kv_lens=lens.long(), cu_seqlens=cu, block_table=table)
    with pytest.raises(ValueError):
        W(x, x[:1], k, v, ks, vs, **ok)                         # shapes differ
    with pytest.raises(ValueError):
        W(x[..., ::2], x[..., ::2], k, v, ks, vs, **ok)         # rows not contiguous
    with pytest.raises(ValueError):
        W(x, x, k, v, ks[:-1], vs, **ok)                        # scales too few
    with pytest.raises(ValueError):
        W(x, x, k, v[:-1], ks, vs, **ok)
    with pytest.raises(ValueError):
        W(x, x, k, v, ks, vs, kv_lens=lens, cu_seqlens=cu[:2], block_table=table)
    with pytest.raises(ValueError):
        W(x, x, k, v, ks, vs, kv_lens=lens, block_table=table)  # 10 rows, 2 sequences
    with pytest.raises(ValueError):
        W(x, x, k, v, ks, vs, block_size=32, **ok)              # not the cache's
    with pytest.raises(ValueError):
        W(x, x, k.transpose(1, 2), v, ks, vs, **ok)             # cache not contiguous
    with pytest.raises(ValueError):
        W(x.cpu(), x, k, v, ks, vs, **ok)
    with pytest.raises(ValueError):                             # contiguous: block_size missing
        W(x, x, k[:2], v[:2], ks[:2], vs[:2], kv_lens=lens, cu_seqlens=cu)
    with pytest.raises(ValueError):
        attn.cache_read_fp8(k, v, ks, vs, cu, 10, table, k_out=x[:, :9])
    with pytest.raises(ValueError):
        attn.cache_read_fp8(k, v, ks, vs, cu, 10, table, starts=i32([0], dev))
    with pytest.raises(AttnError) as e:                         # rows on one another
        attn.cache_read_fp8(k, v, ks, vs, cu, 10, table,
                            k_out=x[:, :1].expand(2, 10, 128))
    assert e.value.status == status_codes()["ATTN_ERR_SHAPE"]
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        attn.decode_fp8(q[..., :64].contiguous(), k, v, ks, vs, lens, table)
    with pytest.raises(AttnError) as e:
        attn.decode_fp8(q[:, :3].contiguous(), k, v, ks, vs, lens, table)     # 3 heads on 2
    assert e.value.status == status_codes()["ATTN_ERR_GQA"]
    with pytest.raises(AttnError) as e:
        attn.decode_fp8(q, k, v, ks, vs, lens, table, num_splits=2000)
    assert e.value.status == status_codes()["ATTN_ERR_SPLITS"]
    with pytest.raises(AttnError) as e:
        attn.decode_fp8(q, k, v, ks, vs, lens, table, num_splits=4,
                        workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    assert e.value.status == status_codes()["ATTN_ERR_SCRATCH"]
    torch.cuda.synchronize()
    for a, b in zip((k, v), c.on(dev)[0]):
        assert torch.equal(a, b)                                # nothing was written
