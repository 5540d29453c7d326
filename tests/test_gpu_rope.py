"""Rotary positions against their formula in 64 bits."""

import pytest
import torch

import exact_io_aware_order_gb300 as attn
from drafts_util import F64, assert_bf16, turned

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def check(x, out, pos, f, name, **kw):
    """x, out (B, heads, N, d) on the GPU, pos (B, N)."""
    for b in range(x.shape[0]):
        want, err = turned(x[b].cpu(), pos[b].cpu(), f.cpu(), **kw)
        assert_bf16(out[b], want, err, name)


def make(dev, B, H, N, d, seed, tokens_first=True):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(B, N, H, d, generator=g, device=dev).to(BF16)
    return x.transpose(1, 2) if tokens_first else x.transpose(1, 2).contiguous()


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 32), (256, 256),
                                   (256, 64), (256, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,n_q,n_kv,N", [(1, 1, 1, 1), (2, 7, 1, 5), (3, 4, 2, 67), (1, 28, 4, 300)])
def test_values(dev, B, n_q, n_kv, N, interleaved, d, rot):
    f = attn.rope_inv_freq(rot, 500000.0, device=dev)
    q, k = make(dev, B, n_q, N, d, 1), make(dev, B, n_kv, N, d, 2, tokens_first=False)
    pos = torch.randint(0, 100000, (B, N), dtype=torch.int32, device=dev)
    for inverse in (False, True):
        qo, ko = attn.rope(q, k, f, pos, interleaved=interleaved, inverse=inverse, magnitude=1.25)
        kw = dict(interleaved=interleaved, sign=-1.0 if inverse else 1.0, magnitude=1.25)
        check(q, qo, pos, f, "q", **kw)
        check(k, ko, pos, f, "k", **kw)
        assert qo.stride() == q.stride() and ko.stride() == k.stride()
        for x, y in ((q, qo), (k, ko)):                      # columns past rot are copies
            assert torch.equal(x[..., rot:], y[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions(dev, interleaved):
    """None, one list for all, far and negative ones; packed tensors."""
    f = attn.rope_inv_freq(128, device=dev)
    q = make(dev, 2, 3, 9, 128, 3)
    n = torch.arange(9, dtype=torch.int32, device=dev)
    far = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 10**6, 10**9, -12345678, 2**24 + 1],
                       dtype=torch.int32, device=dev)
    kw = dict(interleaved=interleaved)
    check(q, attn.rope(q, None, f, **kw)[0], n.expand(2, 9), f, "none", **kw)
    check(q, attn.rope(q, None, f, far, **kw)[0], far.expand(2, 9), f, "far", **kw)
    both = torch.stack([far, n]).contiguous()
    check(q, attn.rope(q, None, f, both, **kw)[0], both, f, "both", **kw)
    p = q[0]
    out, none = attn.rope(p, None, f, far, **kw)
    assert none is None and out.shape == p.shape
    check(p[None], out[None], far[None], f, "packed", **kw)


def test_frequencies_are_used_modulo_a_turn(dev):
    """Any finite frequency: whole turns a position change nothing."""
    import math

    f = torch.tensor([0.0, 1.0, -0.5, 3.0, 7.0, -9.0, 1e-9, 2 * math.pi - 1e-3], dtype=F64, device=dev)
    q = make(dev, 1, 2, 40, 64, 4)
    pos = torch.arange(40, dtype=torch.int32, device=dev)[None]
    check(q, attn.rope(q, None, f)[0], pos, f, "odd frequencies")


def test_in_place_and_views(dev):
    f = attn.rope_inv_freq(64, device=dev)
    qkv = torch.randn(2, 33, 8, 128, device=dev).to(BF16)
    was = qkv.clone()
    q, k = qkv[:, :, :5].transpose(1, 2), qkv[:, :, 5:7].transpose(1, 2)
    qo, ko = attn.rope(q, k, f, q_out=q, k_out=k)
    assert qo is q and ko is k
    pos = torch.arange(33).expand(2, 33)
    check(was[:, :, :5].transpose(1, 2), q, pos, f, "q")
    check(was[:, :, 5:7].transpose(1, 2), k, pos, f, "k")
    assert torch.equal(was[:, :, 7], qkv[:, :, 7])          # what lies between stays
    out = torch.full((2, 5, 33, 256), 7.0, dtype=BF16, device=dev)
    attn.rope(was[:, :, :5].transpose(1, 2), None, f, q_out=out[..., 64:192])
    assert torch.equal(out[..., 64:192], q)
    assert bool((out[..., :64] == 7).all()) and bool((out[..., 192:] == 7).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(dev, interleaved):
    """inverse=True on dy is the gradient of sum(dy * rope(x)): of the formula (autograd in
    64 bits), and by differences."""
    f = attn.rope_inv_freq(48, device=dev)
    x, dy = make(dev, 1, 2, 11, 64, 5), make(dev, 1, 2, 11, 64, 6)
    dx = attn.rope(dy, None, f, interleaved=interleaved, inverse=True, magnitude=0.75)[0]
    leaf = x[0].cpu().to(F64).requires_grad_()
    pos = torch.arange(11)
    kw = dict(interleaved=interleaved, magnitude=0.75)
    (turned(leaf, pos, f.cpu(), **kw)[0] * dy[0].cpu().to(F64)).sum().backward()
    _, err = turned(dy[0].cpu(), pos, f.cpu(), sign=-1.0, **kw)
    assert_bf16(dx[0], leaf.grad, err, "gradient")
    step = torch.zeros_like(leaf.detach())
    step[1, 7, 3] = 0.5                                     # the map is linear: any step will do
    at = lambda s: float((turned(x[0].cpu().to(F64) + s, pos, f.cpu(), **kw)[0] * dy[0].cpu().to(F64)).sum())
    assert abs(at(step) - at(-step) - float(leaf.grad[1, 7, 3])) <= 1e-9


def test_non_finite_values_stay_in_their_pairs(dev):
    f = attn.rope_inv_freq(32, device=dev)
    q = make(dev, 1, 1, 4, 64, 7)
    q[0, 0, 1, 3], q[0, 0, 2, 50] = float("nan"), float("inf")
    out = attn.rope(q, None, f)[0]
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[0, 0, 1, 3], [0, 0, 1, 19], [0, 0, 2, 50]]
    assert out[0, 0, 2, 50] == float("inf")


def test_streams_and_graphs(dev):
    f = attn.rope_inv_freq(128, device=dev)
    q = make(dev, 1, 8, 700, 128, 8)
    want = attn.rope(q, None, f)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.rope(q, None, f, stream=side)[0]
    side.synchronize()
    assert torch.equal(want, got)
    pos = torch.arange(700, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.rope(q, None, f, pos, q_out=out)
    for add in (0, 5):
        pos.copy_(torch.arange(700, dtype=torch.int32, device=dev) + add)
        graph.replay()
        assert torch.equal(out, attn.rope(q, None, f, pos)[0])


def test_scalings(dev):
    """rope_inv_freq's rules by their definition."""
    f = attn.rope_inv_freq(64, 10000.0, device="cpu")
    assert f.dtype is F64 and float(f[0]) == 1.0 and abs(float(f[16]) - 0.01) < 1e-15
    assert torch.allclose(attn.rope_inv_freq(64, scaling="linear", factor=4, device="cpu"), f / 4, rtol=1e-15)
    b = attn.rope_inv_freq(64, scaling="base", factor=4, device="cpu")
    assert float(b[0]) == 1.0 and abs(float(b[-1] / f[-1]) - 0.25) < 1e-12
    p = attn.rope_inv_freq(64, scaling="parts", factor=8, original_len=4096, device="cpu")
    ratio = p / f
    assert float(ratio[0]) == 1.0 and abs(float(ratio[-1]) - 0.125) < 1e-15
    assert bool((ratio[1:] <= ratio[:-1] + 1e-15).all())


def test_refusals(dev):
    f = attn.rope_inv_freq(64, device=dev)
    q = make(dev, 2, 4, 8, 64, 9)
    for kw, exc in [(dict(q=q.float()), TypeError), (dict(q=q[0, 0]), ValueError), (dict(q=None), TypeError),
                    (dict(q=q[..., ::2]), ValueError), (dict(k=q[:, :, :4]), ValueError),
                    (dict(inv_freq=f.float()), TypeError), (dict(inv_freq=f.cpu()), ValueError),
                    (dict(inv_freq=f[:7].clone()), attn.AttnError), (dict(inv_freq=torch.ones(40, dtype=F64, device=dev)), attn.AttnError),
                    (dict(positions=torch.zeros(7, dtype=torch.int32, device=dev)), ValueError),
                    (dict(positions=torch.zeros(2, 8, device=dev)), TypeError),
                    (dict(q_out=torch.empty(2, 4, 9, 64, dtype=BF16, device=dev)), ValueError),
                    (dict(q_out=q[:, :1].expand(2, 4, 8, 64)), attn.AttnError),
                    (dict(k_out=q), ValueError), (dict(magnitude=float("nan")), attn.AttnError),
                    (dict(q=torch.zeros(1, 2, 8, 96, dtype=BF16, device=dev)), attn.AttnError)]:
        args = dict(q=q, k=None, inv_freq=f)
        args.update(kw)
        with pytest.raises(exc):
            attn.rope(**args)
    attn.check_device_status()
