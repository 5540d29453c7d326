"""Workloads of a decode step with drafted tokens: what a serving program calls,
a plain form of each in elementary torch operations, and its value in 64 bits.

* rope:   queries and keys are rotated by their positions (or back: its gradient);
* append: new keys and values go into the bf16 cache, the keys rotated on the way,
          and the queries of the same tokens rotated with them;
* tree:   the nodes of a tree of drafted tokens attend over the cache;
* verify: which drafted tokens stand against the target's probabilities, and
          the next token, from given random numbers.

A sequence's nodes are its last token (node 0, the root) and the drafted tokens;
they lie in the cache behind the tokens cached before them.

``own`` selects the framework's calls; otherwise :func:`run` is the plain form.
"""

import math
import random

import torch

own = False

FIX = 60                        # verify: weights are whole multiples of 2^-60
MOST_NODES = 64


def _case(name, **kw):
    c = {"op": "tree", "batch": 1, "n_q": 28, "n_kv": 4, "d": 128, "block": 16, "paged": True,
         "lo": 0, "hi": 0, "new_lo": 1, "new_hi": 1, "chain": False, "rot": 0, "inter": False,
         "far": 0, "inverse": False, "packed": False, "window": -1, "softcap": 0.0, "alibi": False,
         "wide": False, "vocab": 0, "drafts": True}
    c.update(kw)
    return {"name": name, **c}


def listed():
    """lo .. hi: tokens already cached, over the sequences of the batch; new_lo .. new_hi: new
    tokens, or nodes, of each.  rot: rotated columns; far: first position; wide: O in fp32."""
    return [
        # Queries and keys of a prompt of 8192 tokens before its prefill, 28 / 4 heads.
        _case("rope_prompt_8192", op="rope", new_lo=8192, new_hi=8192, rot=128),
        # Their gradients for packed sequences far into a long context: neighbouring pairs, half
        # of the head.
        _case("rope_grad_packed_far", op="rope", packed=True, n_q=32, n_kv=8, batch=16, new_lo=256,
              new_hi=4096, rot=64, inter=True, far=900_000, inverse=True),
        # One decode step's keys, values and queries of 16 sequences: the smallest call.
        _case("append_token_b16", op="append", batch=16, n_q=32, n_kv=8, lo=1024, hi=4096, rot=128),
        # 16 prompts of 256 - 4096 tokens behind ragged cached prefixes, 64-token blocks.
        _case("append_prompts_b16", op="append", batch=16, n_q=32, n_kv=8, block=64, hi=1000,
              new_lo=256, new_hi=4096, rot=128),
        # The trees of 64 sequences, head_dim 256, a quarter of the head rotated.
        _case("append_trees_b64", op="append", batch=64, n_q=16, n_kv=8, d=256, lo=500, hi=8000,
              new_lo=9, new_hi=63, rot=64),
        # A chat's first steps: a short chain over one short sequence.
        _case("tree_short", lo=300, hi=300, new_lo=6, new_hi=6, chain=True),
        # One long sequence, contiguous cache: 7 x 32 rows a kv head.
        _case("tree_30720", paged=False, lo=30720, hi=30720, new_lo=32, new_hi=32),
        # A batch of 16 sequences of 1024 - 32768 tokens, 32 / 8 heads, trees of 5 - 64 nodes.
        _case("tree_paged_b16", batch=16, n_q=32, n_kv=8, lo=1024, hi=32768, new_lo=5, new_hi=64),
        # Head_dim 256 with soft-capping and a sliding window, odd block size, fp32 outputs.
        _case("tree_d256_window", batch=4, n_q=16, n_kv=8, d=256, block=24, lo=2000, hi=9000,
              new_lo=7, new_hi=33, window=4095, softcap=50.0, wide=True),
        # Many query heads on one kv head, head_dim 64, ALiBi, 128-token blocks: 1024 rows a kv
        # head.
        _case("tree_d64_g32_alibi", batch=8, n_q=64, n_kv=2, d=64, block=128, lo=100, hi=16000,
              new_lo=16, new_hi=32, alibi=True),
        # A chain of five drafted tokens, their tokens the draft's most likely ones.
        _case("verify_chain_b1", op="verify", new_lo=6, new_hi=6, chain=True, vocab=32000,
              drafts=False),
        # The trees of 64 sequences with the draft's probabilities, an odd vocabulary.
        _case("verify_trees_b64", op="verify", batch=64, new_lo=10, new_hi=41, vocab=128257),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("rope", "append", "tree", "tree", "tree", "verify"))
    n_kv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 4, 5, 7, 8, 16, 32))
    d = rng.choice((64, 128, 128, 256))
    batch = log(1, 64)
    c = dict(_case("", op=op, n_kv=n_kv, n_q=n_kv * g, d=d, batch=batch,
                   block=rng.choice((1, 8, 16, 16, 24, 32, 64, 100, 128, 256)),
                   paged=rng.random() < 0.7, chain=rng.random() < 0.3))
    del c["name"]
    if op in ("rope", "append"):
        c["rot"] = 16 * rng.randint(1, d // 16) if rng.random() < 0.5 else d
        c["inter"] = rng.random() < 0.4
        c["far"] = log(1, 1_000_000) if rng.random() < 0.4 else 0
        c["inverse"] = op == "rope" and rng.random() < 0.4
        c["packed"] = rng.random() < 0.5
        # Values of the whole batch, at most those of the largest listed case.
        top = max(1, 60_000_000 // (batch * d * n_kv * (g + 2)))
        c["new_hi"] = log(1, min(top, 16384)) if op == "rope" or rng.random() < 0.5 else 1
        c["new_lo"] = c["new_hi"]
        if op == "append" or c["packed"]:
            c["new_lo"] = rng.randint(min(1, c["new_hi"]), c["new_hi"])
        if op == "append":
            c["hi"] = rng.randint(0, 2000)
            c["lo"] = rng.randint(0, c["hi"])
            c["packed"] = False
    elif op == "tree":
        c["new_hi"] = log(1, MOST_NODES)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        tiles = max(1, g * c["new_hi"] // 256)
        top = max(64, 250_000_000 // (tiles * batch * n_kv * d))
        c["hi"] = log(1, min(top, 32768))
        c["lo"] = rng.randint(0, c["hi"]) if rng.random() < 0.8 else c["hi"]
        kind = rng.choice(("plain", "plain", "window", "softcap", "alibi"))
        if kind == "window":
            c["window"] = log(1, 8192)
        elif kind == "softcap":
            c["softcap"] = float(rng.choice((20, 30, 50)))
        elif kind == "alibi":
            c["alibi"] = True
        c["wide"] = rng.random() < 0.3
    else:
        c["new_hi"] = log(1, MOST_NODES)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["vocab"] = log(100, min(200_000, 200_000_000 // (batch * c["new_hi"])))
        c["drafts"] = rng.random() < 0.6
    return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, both among them where n > 1, in no order."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7919 + n // 2) % n) // (n - 1) if math.gcd(7919, n) == 1
            else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    """(cached, new) tokens of each sequence.  The new ones run the other way, so that long
    sequences meet small trees too."""
    cached = _spread(case["lo"], case["hi"], case["batch"])
    new = _spread(case["new_lo"], case["new_hi"], case["batch"])
    return cached, new[::-1]


def _far(case):
    """First position of each sequence's new tokens."""
    cached = _lens(case)[0]
    return [case["far"] + n for n in cached]


def work(case):
    cached, new = _lens(case)
    n_kv, n_q, d, t = case["n_kv"], case["n_q"], case["d"], sum(new)
    if case["op"] == "rope":
        n = t * (n_q + n_kv) * d
        return {"bytes": 4 * n + 4 * t, "flops": 3 * t * (n_q + n_kv) * case["rot"]}
    if case["op"] == "append":
        n = t * (n_q + 2 * n_kv) * d
        return {"bytes": 4 * n + 4 * t, "flops": 3 * t * (n_q + n_kv) * case["rot"]}
    if case["op"] == "verify":
        rows = case["batch"] * (2 if case["drafts"] else 1)
        return {"bytes": 4 * rows * case["vocab"], "flops": 3 * rows * case["vocab"]}
    seen = [min(a, case["window"]) if case["window"] >= 0 else a for a in cached]
    keys = sum(a + b for a, b in zip(seen, new))
    pairs = sum(b * (a + (b + 1) / 2) for a, b in zip(seen, new))
    return {"bytes": 4 * keys * n_kv * d + t * n_q * (d * (6 if case["wide"] else 4) + 4),
            "flops": 4 * pairs * n_q * d}


def _tree(case, seed):
    """Parents of each sequence's nodes, by index within the sequence (the root's is -1)."""
    rng = random.Random(seed)
    out = []
    for n in _lens(case)[1]:
        p = [-1]
        for i in range(1, n):
            p.append(i - 1 if case["chain"] or rng.random() < 0.4 else rng.randrange(i))
        out.append(p)
    return out


def _masks(trees):
    """Each node's ancestors and itself, a bit for each node of the sequence."""
    words, depths = [], []
    for p in trees:
        at = len(words)
        for i, j in enumerate(p):
            words.append((words[at + j] if j >= 0 else 0) | 1 << i)
            depths.append(depths[at + j] + 1 if j >= 0 else 0)
    return [w - (1 << 64) if w >> 63 else w for w in words], depths


def _frequencies(case, dev):
    """base^(-2 i / rot); for far positions the slow ones slowed down eightfold, the fast ones
    kept, and a ramp between them, as models for long contexts do."""
    r = case["rot"]
    f = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
    if case["far"]:
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    op, B, n_q, n_kv, d, blk = (case[k] for k in ("op", "batch", "n_q", "n_kv", "d", "block"))
    cached, new = _lens(case)
    total = sum(new)
    cu = [sum(new[:i]) for i in range(B + 1)]
    s = {"case": case, "cu": ints(cu), "total": total}
    # A few channels of the keys are larger than the rest, the same ones in every token.
    channel = 1.0 + 5.0 * (torch.rand(n_kv, 1, d, generator=gen, device=dev) < 0.03)
    if op == "rope":
        s["inv_freq"] = _frequencies(case, dev)
        s["magnitude"] = 1.1 if case["far"] else 1.0
        pos = [a + i for a, n in zip(_far(case), new) for i in range(n)]
        if case["packed"]:
            s["q"] = randn(n_q, total, d).to(torch.bfloat16)
            s["k"] = (randn(n_kv, total, d) * channel).to(torch.bfloat16)
            s["pos"] = ints(pos)
        else:
            # What a projection leaves, tokens first, seen heads first.
            n = new[0]
            s["q"] = randn(B, n, n_q, d).to(torch.bfloat16).transpose(1, 2)
            s["k"] = (randn(B, n, n_kv, d) * channel[:, 0]).to(torch.bfloat16).transpose(1, 2)
            s["pos"] = ints(pos).view(B, n)
        return s
    if op == "verify":
        V = case["vocab"]
        trees = _tree(case, seed)
        logits = 2.5 * randn(total, V)
        s["p"] = torch.softmax(logits, dim=1)
        q = torch.softmax(logits.add_(0.5 * randn(total, V)), dim=1)
        del logits
        parent = ints([p for t in trees for p in t])
        first = torch.repeat_interleave(ints(cu[:-1], torch.int64), ints(new, torch.int64))
        up = first + parent.clamp(min=0)
        rank = ints([t[:i].count(t[i]) for t in trees for i in range(len(t))], torch.int64)
        if case["drafts"]:
            picks = torch.multinomial(q, 8, replacement=True, generator=gen)
        else:
            picks = torch.topk(q, 8, dim=1).indices
        s["token"] = picks[up, rank % 8].to(torch.int32)
        s["q"] = q if case["drafts"] else None
        s["parent"] = parent
        s["u"] = torch.rand(total, generator=gen, device=dev)
        s["u_last"] = torch.rand(B, generator=gen, device=dev)
        s["most"] = max(new)
        return s
    room = [a + b for a, b in zip(cached, new)]
    most = max(room)
    if case["paged"]:
        need = [-(-n // blk) for n in room]
        blocks = sum(need) + 2
        order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
        first = ints([sum(need[:b]) for b in range(B)])
        at = first[:, None] + torch.arange(max(need), device=dev)
        inside = torch.arange(max(need), device=dev) < ints(need)[:, None]
        s["table"] = torch.where(inside, order[at.clamp(max=blocks - 1)], 0).to(torch.int32)
        shape = (blocks, blk, n_kv, d)
    else:
        s["table"], shape = None, (B, most, n_kv, d)
    s["kc"] = (randn(*shape) * channel[:, 0]).to(torch.bfloat16)
    s["vc"] = randn(*shape).to(torch.bfloat16)
    s["lens"] = ints(cached)
    s["most"] = most
    if op == "append":
        s["inv_freq"] = _frequencies(case, dev)
        # A projection's output, tokens first: one row of all heads a token.
        qkv = randn(total, n_q + 2 * n_kv, d)
        qkv[:, n_q:n_q + n_kv] *= channel[:, 0]
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = qkv.split([n_q, n_kv, n_kv], dim=1)
        s["one"] = case["new_lo"] == case["new_hi"] == 1
        s["far"] = case["far"]
        s["pos"] = None
        if case["new_hi"] <= MOST_NODES and not s["one"]:
            depth = _masks(_tree(case, seed))[1]
            start = [a for a, n in zip(_far(case), new) for _ in range(n)]
            s["pos"] = ints([a + b for a, b in zip(start, depth)])
        elif case["far"]:
            s["pos"] = ints([a + i for a, n in zip(_far(case), new) for i in range(n)])
        return s
    s["q"] = randn(total, n_q, d).to(torch.bfloat16)
    words, depth = _masks(_tree(case, seed))
    s["mask"] = None if case["chain"] else ints(words, torch.int64)
    s["words"], s["depth"] = ints(words, torch.int64), ints(depth, torch.int64)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["alibi"]:
        s["slopes"] = ints([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)], torch.float32)
    return s


def _own(s):
    import exact_io_aware_order_gb300 as attn

    case = s["case"]
    if case["op"] == "rope":
        q, k = attn.rope(s["q"], s["k"], s["inv_freq"], s["pos"], interleaved=case["inter"],
                         inverse=case["inverse"], magnitude=s["magnitude"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        rot = {"inv_freq": s["inv_freq"], "positions": s["pos"], "interleaved": case["inter"]}
        if s["one"]:
            q = attn.cache_append(s["k_new"], s["v_new"], s["kc"], s["vc"], s["lens"],
                                  block_table=s["table"], q=s["q"], **rot)
        else:
            q = attn.cache_append(s["k_new"].transpose(0, 1), s["v_new"].transpose(0, 1), s["kc"],
                                  s["vc"], s["lens"], s["cu"], s["table"],
                                  q=s["q"].transpose(0, 1), **rot).transpose(0, 1)
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if case["op"] == "tree":
        o, lse = attn.decode_tree(s["q"], s["kc"], s["vc"], s["lens"], s["cu"], s["mask"],
                                  s["table"], max_kv_len=s["most"], scale=s["scale"],
                                  window_left=case["window"], softcap=case["softcap"],
                                  alibi_slopes=s.get("slopes"),
                                  out_dtype=torch.float32 if case["wide"] else torch.bfloat16)
        return {"o": o, "lse": lse}
    n, path, token = attn.verify_tree(s["p"], s["token"], s["parent"], s["cu"], s["u"],
                                      s["u_last"], s["q"])
    return {"n": n, "path": path, "token": token}


def _rotated(x, pos, f, inter, sign=1.0, magnitude=1.0):
    """x (..., d) fp32 by positions that match its leading shape: the angles in 64 bits."""
    a = pos.double()[..., None] * f
    cos = (a.cos() * magnitude).float()
    sin = (a.sin() * (magnitude * sign)).float()
    r = 2 * f.shape[0]
    y = x.clone()
    if inter:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y


def _owner(s):
    """The sequence of each packed token, and its index there."""
    t = torch.arange(s["total"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t - s["cu"].long()[seq]


def _rows(s, seq, pos):
    """Row of the cache viewed as (rows, n_kv, d) of position pos of sequence seq."""
    blk = s["case"]["block"]
    if s["table"] is None:
        return seq * s["kc"].shape[1] + pos
    return s["table"].long()[seq, pos // blk] * blk + pos % blk


def _plain_rope(s):
    case, out = s["case"], {}
    for name in ("q", "k"):
        y = _rotated(s[name].float(), s["pos"][..., None, :].expand(s[name].shape[:-1]),
                     s["inv_freq"], case["inter"], -1.0 if case["inverse"] else 1.0,
                     s["magnitude"])
        out[name] = y.to(torch.bfloat16)
    return out


def _plain_append(s):
    case = s["case"]
    n_kv, d = case["n_kv"], case["d"]
    seq, i = _owner(s)
    slot = s["lens"].long()[seq] + i
    row = _rows(s, seq, slot)
    pos = (slot if s["pos"] is None else s["pos"])[:, None]
    rot = lambda x: _rotated(x.float(), pos.expand(x.shape[:-1]), s["inv_freq"], case["inter"])
    s["kc"].view(-1, n_kv, d)[row] = rot(s["k_new"]).to(torch.bfloat16)
    s["vc"].view(-1, n_kv, d)[row] = s["v_new"]
    return {"q": rot(s["q"]).to(torch.bfloat16), "k": s["kc"], "v": s["vc"]}


def _plain_tree(s):
    case = s["case"]
    B, n_q, n_kv, d = case["batch"], case["n_q"], case["n_kv"], case["d"]
    g, L, N, dev = n_q // n_kv, s["most"], max(_lens(case)[1]), s["cu"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    node = torch.arange(N, device=dev)
    at = (cu[:-1, None] + node).clamp(max=s["total"] - 1)                     # (B, N)
    real = node < n[:, None]
    j = torch.arange(L, device=dev)
    # Key j of a sequence: a cached token, or node j - len.
    u = j[None] - lens[:, None]                                              # (B, L)
    inside = u < n[:, None]
    word = torch.where(real, s["words"][at], 0)
    bit = (word[:, :, None] >> u.clamp(0, 63)[:, None, :]) & 1
    seen = inside[:, None, :] & ((u < 0)[:, None, :] | (bit == 1))           # (B, N, L)
    # Positions: kv_len + depth.
    depth = torch.where(real, s["depth"][at], 0)
    key_node = (cu[:-1, None] + u.clamp(min=0)).clamp(max=s["total"] - 1)
    key_pos = torch.where(u < 0, j[None], lens[:, None] + s["depth"][key_node])
    dist = (lens[:, None] + depth)[:, :, None] - key_pos[:, None, :]
    if case["window"] >= 0:
        seen = seen & (dist <= case["window"])
    row = _rows(s, torch.arange(B, device=dev)[:, None], torch.where(inside, j[None], 0))
    k = s["kc"].view(-1, n_kv, d)[row].float().permute(0, 2, 3, 1)           # (B, n_kv, d, L)
    v = s["vc"].view(-1, n_kv, d)[row].float().permute(0, 2, 1, 3)
    q = s["q"][at].float().view(B, N, n_kv, g, d).permute(0, 2, 1, 3, 4)
    x = (q.reshape(B, n_kv, N * g, d) @ k) * s["scale"]
    x = x.view(B, n_kv, N, g, L)
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if case["alibi"]:
        x = x - s["slopes"].view(n_kv, 1, g, 1) * dist[:, None, :, None, :].float()
    x = torch.where(seen[:, None, :, None, :], x, -math.inf)
    m = x.amax(dim=4, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    l = x.sum(dim=4, keepdim=True)
    o = (x.view(B, n_kv, N * g, L) @ v).view(B, n_kv, N, g, d)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 2, 1, 3, 4).reshape(B, N, n_q, d)
    lse = (m + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(B, N, n_q)
    return {"o": o[real].to(torch.float32 if case["wide"] else torch.bfloat16), "lse": lse[real]}


def _fixed(x):
    """Multiples of 2^-60 in x, rounded down."""
    return (x.double() * 2.0 ** FIX).to(torch.int64)


def _times(a, b):
    """a b / 2^60 rounded down, both below 2^62 (by halves of 30 bits)."""
    low = (1 << 30) - 1
    ah, al, bh, bl = a >> 30, a & low, b >> 30, b & low
    return ah * bh + ((ah * bl + al * bh + (al * bl >> 30)) >> 30)


def _plain_verify(s):
    B, N, V = s["case"]["batch"], s["most"], s["case"]["vocab"]
    cu, dev = s["cu"].long(), s["cu"].device
    n = cu[1:] - cu[:-1]
    b = torch.arange(B, device=dev)
    at = cu[:-1]                                                             # where each stands
    w = _fixed(s["p"][at])
    Z = torch.full((B,), 1 << FIX, dtype=torch.int64, device=dev)
    path = torch.full((B, MOST_NODES), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    count = torch.zeros(B, dtype=torch.int64, device=dev)
    # Children have larger indices than their parents: one pass over the nodes is the walk.
    for i in range(1, N):
        t = (cu[:-1] + i).clamp(max=s["total"] - 1)
        tried = (i < n) & (s["parent"][t].long() + cu[:-1] == at)
        x = s["token"][t].long()
        if s["q"] is None:
            # Without the draft's probabilities a drafted token counts as certain.
            qz, less = Z, w.clone()
            less[b, x] = 0
            rest = Z - w[b, x]
        else:
            qz = _times(_fixed(s["q"][at]), Z[:, None])
            less = (w - qz).clamp(min=0)
            rest, qz = less.sum(dim=1), qz[b, x]
        ok = tried & (_times(qz, _fixed(s["u"][t])) < w[b, x])
        no = tried & ~ok
        count += ok
        to = torch.where(ok, count, MOST_NODES - 1)
        path[b, to] = torch.where(ok, i, path[b, to]).to(torch.int32)
        at = torch.where(ok, t, at)
        w = torch.where(ok[:, None], _fixed(s["p"][at]), torch.where(no[:, None], less, w))
        Z = torch.where(ok, 1 << FIX, torch.where(no, rest.clamp(min=0), Z))
    left = w.sum(dim=1)
    w = torch.where((left > 0)[:, None], w, _fixed(s["p"][at]))
    c = w.cumsum(dim=1)
    T = _times(c[:, -1], _fixed(s["u_last"]))
    token = (c <= T[:, None]).sum(dim=1).clamp(max=V - 1)
    return {"n": count.to(torch.int32), "path": path, "token": token.to(torch.int32)}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "tree": _plain_tree,
            "verify": _plain_verify}[state["case"]["op"]](state)


def exact(case, seed):
    """The operators' values in 64 bits, sequence by sequence: rotations as products of complex
    numbers, attention over each sequence's own keys, probabilities as fractions of one."""
    s = prepare(case, seed)
    op, n_q, n_kv, d, blk = (case[k] for k in ("op", "n_q", "n_kv", "d", "block"))
    cached, new = _lens(case)
    f64 = torch.float64

    def turned(x, pos, sign=1.0, magnitude=1.0):
        """x (heads, tokens, d), pos (tokens,)."""
        f, r = s["inv_freq"], case["rot"]
        z = torch.polar(torch.full_like(f, magnitude).expand(len(pos), -1),
                        sign * pos.to(f64)[:, None] * f)
        y = x.to(f64).clone()
        if case["inter"]:
            y[..., :r] = torch.view_as_real(
                torch.view_as_complex(y[..., :r].reshape(*y.shape[:2], r // 2, 2).contiguous()) * z
            ).reshape(*y.shape[:2], r)
        else:
            c = torch.complex(y[..., :r // 2].clone(), y[..., r // 2:r].clone()) * z
            y[..., :r // 2], y[..., r // 2:r] = c.real, c.imag
        return y

    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        if case["packed"]:
            return {n: turned(s[n], s["pos"], sign, s["magnitude"]) for n in ("q", "k")}
        return {n: torch.stack([turned(x, p, sign, s["magnitude"])
                                for x, p in zip(s[n], s["pos"])]) for n in ("q", "k")}
    if op == "verify":
        out = {"n": [], "path": [], "token": []}
        at = 0
        for b, m in enumerate(new):
            p = s["p"][at:at + m].to(f64)
            q = None if s["q"] is None else s["q"][at:at + m].to(f64)
            tok, up = s["token"][at:at + m].tolist(), s["parent"][at:at + m].tolist()
            u = s["u"][at:at + m].tolist()
            cur, path = 0, [0]
            going = True
            while going:
                going, w = False, p[cur].clone()
                for k in [i for i in range(m) if up[i] == cur]:
                    x = tok[k]
                    qx = 1.0 if q is None else float(q[cur, x])
                    if u[k] * qx < float(w[x]):
                        cur, going = k, True
                        path.append(k)
                        break
                    if q is None:
                        rest = 1.0 - float(w[x])
                        w[x] = 0.0
                        w = w / rest
                    else:
                        w = (w - q[cur]).clamp(min=0)
                        w = w / w.sum()
            c = w.cumsum(0)
            out["token"].append(int((c <= float(s["u_last"][b]) * c[-1]).sum()))
            out["n"].append(len(path) - 1)
            out["path"].append(path + [-1] * (MOST_NODES - len(path)))
            at += m
        return {n: torch.tensor(x, dtype=torch.int32) for n, x in out.items()}

    def rows(b, lo, hi):
        """Where positions lo .. hi - 1 of sequence b lie, as rows of the cache."""
        j = torch.arange(lo, hi, device=s["cu"].device)
        if s["table"] is None:
            return b * s["kc"].shape[1] + j
        return s["table"][b].long()[j // blk] * blk + j % blk

    if op == "append":
        k, v = (s[n].view(-1, n_kv, d).to(f64) for n in ("kc", "vc"))
        qs, at = [], 0
        for b, m in enumerate(new):
            sl, place = slice(at, at + m), rows(b, cached[b], cached[b] + m)
            pos = (torch.arange(cached[b], cached[b] + m, device=k.device) if s["pos"] is None
                   else s["pos"][sl])
            k[place] = turned(s["k_new"][sl].transpose(0, 1), pos).transpose(0, 1)
            v[place] = s["v_new"][sl].to(f64)
            qs.append(turned(s["q"][sl].transpose(0, 1), pos).transpose(0, 1))
            at += m
        return {"q": torch.cat(qs), "k": k.view(s["kc"].shape), "v": v.view(s["vc"].shape)}

    trees, g = _tree(case, seed), n_q // n_kv
    os, ls = [], []
    for b, m in enumerate(new):
        L = cached[b] + m
        at = int(s["cu"][b])
        where = rows(b, 0, L)
        seen = torch.ones(m, L, dtype=torch.bool)
        pos, depth = list(range(cached[b])), []
        seen[:, cached[b]:] = False
        for i, p in enumerate(trees[b]):
            depth.append(depth[p] + 1 if p >= 0 else 0)
            if p >= 0:
                seen[i, cached[b]:] = seen[p, cached[b]:]
            seen[i, cached[b] + i] = True
        kp = torch.tensor(pos + [cached[b] + x for x in depth])
        dist = (kp[cached[b]:, None] - kp[None, :])
        if case["window"] >= 0:
            seen &= dist <= case["window"]
        seen, dist = seen.to(where.device), dist.to(where.device).to(f64)
        ob, lb = [], []
        for h in range(n_kv):
            q = s["q"][at:at + m, h * g:(h + 1) * g].to(f64)                  # (m, g, d)
            k = s["kc"].view(-1, n_kv, d)[where, h].to(f64)
            v = s["vc"].view(-1, n_kv, d)[where, h].to(f64)
            x = (q.reshape(m * g, d) @ k.T).view(m, g, L) / math.sqrt(d)
            if case["softcap"] > 0:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if case["alibi"]:
                x = x - s["slopes"][h * g:(h + 1) * g].to(f64)[None, :, None] * dist[:, None]
            x = x.masked_fill(~seen[:, None], -math.inf)
            lse = torch.logsumexp(x, dim=2, keepdim=True)
            ob.append((torch.exp(x - lse).view(m * g, L) @ v).view(m, g, d))
            lb.append(lse[..., 0])
        os.append(torch.cat(ob, dim=1))
        ls.append(torch.cat(lb, dim=1))
    return {"o": torch.cat(os), "lse": torch.cat(ls)}
