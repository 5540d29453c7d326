"""Rotary positions, and a decode step with drafted tokens, over the C ABI in
``include/attn.h``: argument marshalling, like ``api.py``.  The calls go to
csrc/binding.cpp first, which takes the plain case, and come here otherwise.

A step of speculative decoding, for each sequence's nodes (its last token, node 0,
and the drafted tokens behind it), q, k and v tokens first as projections leave them
((total, heads, d); the cache's calls take heads first, decode_tree tokens first and
contiguous)::

    t = lambda x: x.transpose(0, 1)
    q = t(cache_append(t(k), t(v), k_cache, v_cache, kv_lens, cu, table, inv_freq, positions, q=t(q)))
    o, lse = decode_tree(q.contiguous(), k_cache, v_cache, kv_lens, cu, mask, table)
    ...                                             # the rest of the model, its probabilities
    n, path, token = verify_tree(probs, tokens, parents, cu, u, u_last, draft_probs)
"""

from __future__ import annotations

import functools
import math
from typing import Optional

import torch

from ._lib import binding, check, lib
from .api import (_BF16, _F32, _I32, _columns, _int32, _lens, _need, _need_all, _raw_stream, _rows_stride,
                  _scope)

_F64 = torch.float64
_I64 = torch.int64
TREE_OUT_BF16 = 1  # ATTN_TREE_OUT_BF16


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                  factor: float = 1.0, original_len: int = 8192, slow_turns: float = 1.0,
                  fast_turns: float = 4.0, device="cuda") -> torch.Tensor:
    """The angles a position of :func:`rope` (float64, radians): base^(-2 i /
    rotary_dim) for pair i, for contexts ``factor`` times as long

    * ``scaling="linear"``: divided by factor;
    * ``"base"``: with base * factor^(rotary_dim / (rotary_dim - 2)), which leaves the
      fastest pair as it is and divides the slowest by factor;
    * ``"parts"``: pairs that make fewer than slow_turns in original_len tokens
      divided by factor, those with more than fast_turns kept, a ramp between.
    """
    if rotary_dim < 16 or rotary_dim % 16:
        raise ValueError("rotary_dim must be a multiple of 16")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if scaling == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=_F64) / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not slow_turns < fast_turns:
            raise ValueError("slow_turns must be below fast_turns")
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def _sizes(*sizes: int) -> tuple[int, ...]:
    """Sizes as the C entry points take them."""
    return tuple(_int32(x, "a size") for x in sizes)


def _strided(t, name: str, dev, ndim: int) -> None:
    """A strided bf16 tensor on dev: contiguous rows, other strides multiples of 8."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16:
        raise TypeError(f"{name} must be a torch.bfloat16 tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    st = t.stride()
    if st[-1] != 1 or any(s % 8 for s in st[:-1]):
        raise ValueError(f"{name} must have contiguous rows and strides that are multiples of 8, "
                         f"got strides {st}")


def _frequencies(inv_freq, dev) -> tuple[int, int]:
    """inv_freq's pointer and the rotary_dim it stands for."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        _need(inv_freq, "inv_freq", _F64, 1)
    _need_all(dev, (inv_freq, "inv_freq", _F64, inv_freq.shape))
    return inv_freq.data_ptr(), 2 * inv_freq.shape[0]


def rope(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor,
         positions: Optional[torch.Tensor] = None, interleaved: bool = False,
         inverse: bool = False, magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions of queries and keys (``attn_rope``).

    q: (B, n_q, N, d) bf16, or packed (n_q, total, d); k the same with n_kv heads, or
    None.  Rows contiguous, the other strides multiples of 8 (a projection's output,
    tokens first, seen through ``transpose``).  inv_freq: (rotary_dim / 2,) float64
    (:func:`rope_inv_freq`); positions: int32 (B, N) or (N,), packed (total,), None:
    the row's index.  ``inverse`` rotates back; with gradients for q and k it gives
    the gradients of this call's inputs.  Autograd does not record this call, as none of
    this package's: outputs are detached, and a model that is trained through it wraps both
    directions in a ``torch.autograd.Function``.  Returns (q_out, k_out), allocated with
    the inputs' layout when not given; an output may be its input.
    """
    if stream is None:
        r = binding().rope(q, k, inv_freq, positions, interleaved, inverse, magnitude, q_out, k_out)
        if r is not NotImplemented:
            return r
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev, ndim = q.device, q.dim()
    if ndim not in (3, 4):
        raise ValueError(f"q must have 3 or 4 dimensions, got shape {tuple(q.shape)}")
    _strided(q, "q", dev, ndim)
    lead, n, d = q.shape[:-3], q.shape[-2], q.shape[-1]
    if k is not None:
        _strided(k, "k", dev, ndim)
        if k.shape[:-3] != lead or k.shape[-2:] != q.shape[-2:]:
            raise ValueError("k must match q in all but its heads")
    f, rot = _frequencies(inv_freq, dev)
    pos, pos_stride = None, 0
    if positions is not None:
        shape = (*lead, n) if isinstance(positions, torch.Tensor) and positions.dim() > 1 else (n,)
        _need_all(dev, (positions, "positions", _I32, shape))
        pos, pos_stride = positions.data_ptr(), n if len(shape) > 1 else 0
    with _scope(dev, stream):
        if q_out is None:
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        rows = []
        for x, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
            if x is None:
                if out is not None:
                    raise ValueError("k_out without k")
                rows += [None, 0, 0, 0, None, 0, 0, 0]
                continue
            _strided(out, name, dev, ndim)
            if out.shape != x.shape:
                raise ValueError(f"{name} must have shape {tuple(x.shape)}")
            for t in (x, out):
                rows += [t.data_ptr(), *((0,) * (4 - ndim)), *t.stride()[:-1]]
        st = lib().attn_rope(*rows, f, pos, pos_stride,
                             *_sizes(lead[0] if lead else 1, q.shape[-3],
                                     0 if k is None else k.shape[-3], n, d, rot),
                             int(bool(interleaved)),
                             int(bool(inverse)), float(magnitude), _raw_stream(dev.index))
    check("attn_rope", st)
    return q_out, k_out


def _cache_bf16(dev, k_cache, v_cache, block_table, num_seqs: int):
    """Checks a bf16 cache; returns (its two pointers and the block table's,
    (block_size, max_blocks, num_blocks, capacity))."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        _need(k_cache, "k_cache", _BF16, 4)
    shape = k_cache.shape
    _need_all(dev, (k_cache, "k_cache", _BF16, shape), (v_cache, "v_cache", _BF16, shape))
    if block_table is None:
        if shape[0] != num_seqs:
            raise ValueError("a contiguous cache must be (num_seqs, L, n_kv, d)")
        return (k_cache.data_ptr(), v_cache.data_ptr(), None), _sizes(0, 0, 0, shape[1])
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        _need(block_table, "block_table", _I32, 2)
    if block_table.shape[0] != num_seqs:
        raise ValueError("block_table must have one row per sequence")
    most = _columns(block_table)
    _need_all(dev, (block_table, "block_table", _I32, (num_seqs, most)))
    return ((k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr()),
            _sizes(shape[1], most, shape[0], shape[1] * most))


def cache_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, kv_lens: torch.Tensor,
                 cu_seqlens: Optional[torch.Tensor] = None,
                 block_table: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 interleaved: bool = False, magnitude: float = 1.0,
                 q_out: Optional[torch.Tensor] = None, stream=None):
    """New keys and values into a bf16 cache behind the kv_lens[s] tokens that each
    sequence has there, the keys rotated on the way (``attn_cache_append``).

    k_new, v_new: bf16, (n_kv, total, d) with sequence s on rows [cu_seqlens[s],
    cu_seqlens[s + 1]), or without cu_seqlens (B, n_kv, d), one token a sequence; q
    (optional): the same tokens' queries, n_q heads.  Rows contiguous, the other
    strides multiples of 8.  The cache is that of :func:`decode`, written in place;
    kv_lens is left to the caller to increment.  inv_freq as :func:`rope` (None: keys
    are written as they are); positions: (total,) int32, None: a token's slot.
    Returns the rotated queries, allocated with q's layout when ``q_out`` is not
    given (None without q); rows outside every sequence are left as they were.
    """
    if stream is None:
        r = binding().cache_append(k_new, v_new, k_cache, v_cache, kv_lens, cu_seqlens, block_table,
                                   inv_freq, positions, q, interleaved, magnitude, q_out)
        if r is not NotImplemented:
            return r
    if not isinstance(k_new, torch.Tensor) or not isinstance(v_new, torch.Tensor):
        raise TypeError("k_new and v_new must be torch.Tensors")
    dev = k_new.device
    _rows_stride(k_new, "k_new", dev)
    _rows_stride(v_new, "v_new", dev)
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    lens = _lens(kv_lens, "kv_lens", None, dev)
    B = kv_lens.shape[0]
    ptrs, geom = _cache_bf16(dev, k_cache, v_cache, block_table, B)
    tok = 0 if cu_seqlens is None else 1
    cu = None if cu_seqlens is None else _lens(cu_seqlens, "cu_seqlens", B + 1, dev)
    total, n_kv, d = k_new.shape[tok], k_new.shape[1 - tok], k_new.shape[2]
    if cu_seqlens is None and total != B:
        raise ValueError("without cu_seqlens k_new and v_new must be (B, n_kv, d)")
    if tuple(k_cache.shape[2:]) != (n_kv, d):
        raise ValueError("the cache's heads or head_dim do not match k_new")
    f, rot = (None, 0) if inv_freq is None else _frequencies(inv_freq, dev)
    pos = None
    if positions is not None:
        _need_all(dev, (positions, "positions", _I32, (total,)))
        pos = positions.data_ptr()
    if q is not None:
        if inv_freq is None:
            raise ValueError("q is rotated: inv_freq is needed")
        _rows_stride(q, "q", dev)
        if q.shape[tok] != total or q.shape[2] != d:
            raise ValueError("q must have k_new's tokens and head_dim")
    elif q_out is not None:
        raise ValueError("q_out without q")
    strides = lambda t: (t.stride(tok), t.stride(1 - tok))
    with _scope(dev, stream):
        rows, n_q = (None, 0, 0, None, 0, 0), 0
        if q is not None:
            if q_out is None:
                q_out = torch.empty_like(q)
            _rows_stride(q_out, "q_out", dev)
            if q_out.shape != q.shape:
                raise ValueError(f"q_out must have shape {tuple(q.shape)}")
            rows, n_q = (q.data_ptr(), *strides(q), q_out.data_ptr(), *strides(q_out)), q.shape[1 - tok]
        st = lib().attn_cache_append(k_new.data_ptr(), v_new.data_ptr(), *strides(k_new),
                                     *strides(v_new), *rows, *ptrs, cu, lens, f, pos,
                                     *_sizes(B, total, n_q, n_kv, d, rot), int(bool(interleaved)),
                                     float(magnitude), *geom, _raw_stream(dev.index))
    check("attn_cache_append", st)
    return q_out


def tree_mask(parents: torch.Tensor, cu_nodes: torch.Tensor) -> torch.Tensor:
    """The mask words of :func:`decode_tree` for trees: each node's ancestors and
    itself.  parents: (total,) int32, a node's parent by its index within its sequence
    (smaller than the node's, any other counts as none), the root's -1; cu_nodes: (B + 1,)
    int32.  Returns (total,) int64 on parents' device; of rows outside every sequence, 0."""
    t = torch.arange(parents.shape[0], dtype=_I64, device=parents.device)
    cu = cu_nodes.to(_I64)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = seq < cu.shape[0] - 1
    first = cu[seq.clamp(max=cu.shape[0] - 2)]
    i = (t - first).clamp(0, 63)
    one = torch.ones_like(t)
    word = torch.where(real, one << i, 0)
    # The ancestor 1, 2, 4, ... generations up, itself for none.
    up = torch.where(real & (parents >= 0) & (parents < t - first), first + parents, -1)
    for _ in range(6):
        at = up.clamp(min=0)
        word = torch.where(up >= 0, word | word[at], word)
        up = torch.where(up >= 0, up[at], -1)
    return word


@functools.lru_cache(maxsize=256)
def _tree_workspace(batch: int, total: int, n_q: int, n_kv: int, d: int, max_kv_len: int,
                    window_left: int, device: int) -> int:
    """attn_decode_tree_workspace_bytes on a device (which has to be current)."""
    return lib().attn_decode_tree_workspace_bytes(batch, total, n_q, n_kv, d, max_kv_len,
                                                  window_left)


def decode_tree(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                kv_lens: torch.Tensor, cu_nodes: torch.Tensor,
                tree_mask: Optional[torch.Tensor] = None,
                block_table: Optional[torch.Tensor] = None, max_kv_len: Optional[int] = None,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None, window_left: int = -1, softcap: float = 0.0,
                alibi_slopes: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.float32):
    """Attention of trees of drafted tokens over a bf16 cache (``attn_decode_tree``).

    q: (total, n_q, d) bf16, sequence b's nodes (its last token, then the drafted ones, 64
    at most) on rows [cu_nodes[b], cu_nodes[b + 1]).  The cache is that of
    :func:`decode`; it holds the nodes' keys and values at slots kv_lens[b],
    kv_lens[b] + 1, ... (:func:`cache_append`).  tree_mask: (total,) int64, bit j: the node
    sees node j (:func:`tree_mask` makes it from parents), None: chains.  max_kv_len: the
    most tokens and nodes of a sequence, a hint for paged caches.  Variants as
    :func:`decode_splitkv`, a node at position kv_lens[b] + depth.  ``workspace``
    (uint8, allocated when not given) holds partials.  Returns (O (total, n_q, d) fp32 or
    bf16, LSE (total, n_q) fp32); rows outside every sequence are left as they were.
    """
    if stream is None and (out_dtype is _F32 or out_dtype is _BF16):
        r = binding().decode_tree(q, k_cache, v_cache, kv_lens, cu_nodes, tree_mask, block_table,
                                  max_kv_len, scale, out, lse, workspace, window_left, softcap,
                                  alibi_slopes, out_dtype is _BF16)
        if r is not NotImplemented:
            return r
    if not isinstance(q, torch.Tensor) or q.dtype is not _BF16 or q.dim() != 3 or \
            not q.is_cuda or not q.is_contiguous():
        _need(q, "q", _BF16, 3)
    dev = q.device
    total, n_q, d = q.shape
    lens = _lens(kv_lens, "kv_lens", None, dev)
    B = kv_lens.shape[0]
    cu = _lens(cu_nodes, "cu_nodes", B + 1, dev)
    ptrs, geom = _cache_bf16(dev, k_cache, v_cache, block_table, B)
    n_kv = k_cache.shape[2]
    if k_cache.shape[3] != d:
        raise ValueError("the cache's head_dim does not match q")
    if max_kv_len is not None:
        max_kv_len = _int32(max_kv_len, "max_kv_len")
        if block_table is not None:
            geom = (*geom[:3], max_kv_len)
        elif max_kv_len > geom[3]:
            raise ValueError("max_kv_len exceeds the contiguous cache's length")
    mask = al = None
    if tree_mask is not None:
        _need_all(dev, (tree_mask, "tree_mask", _I64, (total,)))
        mask = tree_mask.data_ptr()
    if alibi_slopes is not None:
        _need_all(dev, (alibi_slopes, "alibi_slopes", _F32, (n_q,)))
        al = alibi_slopes.data_ptr()
    if out_dtype not in (_F32, _BF16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    window_left = _int32(window_left, "window_left")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _scope(dev, stream):
        if out is None:
            out = torch.empty((total, n_q, d), dtype=out_dtype, device=dev)
        else:
            _need_all(dev, (out, "out", out_dtype, (total, n_q, d)))
        if lse is None:
            lse = torch.empty((total, n_q), dtype=_F32, device=dev)
        else:
            _need_all(dev, (lse, "lse", _F32, (total, n_q)))
        if workspace is None:
            n = _tree_workspace(*_sizes(B, total, n_q, n_kv, d, geom[3]), window_left, dev.index)
            workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        else:
            _need(workspace, "workspace", torch.uint8, 1)
            _need_all(dev, (workspace, "workspace", torch.uint8, workspace.shape))
        wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
        st = lib().attn_decode_tree(q.data_ptr(), *ptrs, lens, cu, mask, wp, wn, out.data_ptr(),
                                    lse.data_ptr(), *_sizes(B, total, n_q, n_kv, d), *geom,
                                    float(scale), window_left, float(softcap), al,
                                    TREE_OUT_BF16 if out_dtype is _BF16 else 0,
                                    _raw_stream(dev.index))
    check("attn_decode_tree", st)
    return out, lse


def _probs(t, name: str, dev, total: int) -> tuple[int, int]:
    """(total, vocab) fp32 probabilities on dev, entries of a row contiguous, rows apart;
    the pointer and the rows' stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _F32:
        raise TypeError(f"{name} must be a torch.float32 tensor")
    if t.dim() != 2 or t.shape[0] != total:
        raise ValueError(f"{name} must be ({total}, vocab), got shape {tuple(t.shape)}")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), t.stride(0) if total > 1 else t.shape[1]


def verify_tree(target_probs: torch.Tensor, draft_tokens: torch.Tensor, parents: torch.Tensor,
                cu_nodes: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor,
                draft_probs: Optional[torch.Tensor] = None,
                num_accepted: Optional[torch.Tensor] = None, path: Optional[torch.Tensor] = None,
                next_token: Optional[torch.Tensor] = None, stream=None):
    """Which drafted tokens stand, and the next token (``attn_verify_tree``).

    target_probs: (total, vocab) fp32, the target's probabilities of the token after each
    node; draft_probs: those that each node's children were drawn from, None: drafts that
    are certain; draft_tokens, parents: (total,) int32; cu_nodes: (B + 1,) int32; u_accept:
    (total,) and u_sample: (B,) fp32 random numbers in [0, 1).  Children of a node are
    tried in index order; those of one node are independent draws from its draft_probs row
    (drawn without replacement, the outputs would not be distributed as the target's).
    Returns (num_accepted (B,), path (B, 64): the root and the accepted
    nodes by index within the sequence, then -1; next_token (B,)), int32.

    The accepted nodes' keys and values belong behind the cached tokens: with chains they
    already lie there; of a tree, append rows path[b, :n + 1] again.
    """
    if stream is None:
        r = binding().verify_tree(target_probs, draft_tokens, parents, cu_nodes, u_accept, u_sample,
                                  draft_probs, num_accepted, path, next_token)
        if r is not NotImplemented:
            return r
    if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 2:
        _need(target_probs, "target_probs", _F32, 2)
    dev, (total, vocab) = target_probs.device, target_probs.shape
    p, ps = _probs(target_probs, "target_probs", dev, total)
    q, qs = (None, 0) if draft_probs is None else _probs(draft_probs, "draft_probs", dev, total)
    if draft_probs is not None and draft_probs.shape[1] != vocab:
        raise ValueError("draft_probs must have target_probs' vocabulary")
    B = cu_nodes.shape[0] - 1 if isinstance(cu_nodes, torch.Tensor) and cu_nodes.dim() == 1 else 0
    cu = _lens(cu_nodes, "cu_nodes", None, dev)
    if B < 1:
        raise ValueError("cu_nodes must have at least two entries")
    _need_all(dev, (draft_tokens, "draft_tokens", _I32, (total,)), (parents, "parents", _I32, (total,)),
              (u_accept, "u_accept", _F32, (total,)), (u_sample, "u_sample", _F32, (B,)))
    with _scope(dev, stream):
        if num_accepted is None:
            num_accepted = torch.empty(B, dtype=_I32, device=dev)
        if path is None:
            path = torch.empty((B, 64), dtype=_I32, device=dev)
        if next_token is None:
            next_token = torch.empty(B, dtype=_I32, device=dev)
        _need_all(dev, (num_accepted, "num_accepted", _I32, (B,)), (path, "path", _I32, (B, 64)),
                  (next_token, "next_token", _I32, (B,)))
        st = lib().attn_verify_tree(p, ps, q, qs, draft_tokens.data_ptr(), parents.data_ptr(), cu,
                                    u_accept.data_ptr(), u_sample.data_ptr(),
                                    num_accepted.data_ptr(), path.data_ptr(),
                                    next_token.data_ptr(), *_sizes(B, total, vocab),
                                    _raw_stream(dev.index))
    check("attn_verify_tree", st)
    return num_accepted, path, next_token
