"""Workloads of the 8-bit key/value cache operators: what a serving program
calls, a plain form of each in elementary torch operations, and its value in
64 bits.

The cache holds e4m3 codes with one float32 scale for each block of tokens and
kv head, a power of two; a value is code * scale.  Operators:

* write:  new keys and values (bf16) are quantised into the cache;
* read:   cached tokens come back as bf16;
* decode: one query token a sequence attends over the cache;
* append: one new token a sequence is written, then attended with the rest.

``own`` selects the framework's calls; otherwise :func:`run` is the plain form.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
K_MIN, K_MAX = -60, 60          # the scale's exponents

_KEYS = ("op", "batch", "n_q", "n_kv", "d", "block", "paged", "lo", "hi", "new_lo", "new_hi",
         "window", "softcap", "alibi")


def _case(name, **kw):
    c = {"op": "decode", "batch": 1, "n_q": 28, "n_kv": 4, "d": 128, "block": 16, "paged": True,
         "lo": 0, "hi": 0, "new_lo": 0, "new_hi": 0, "window": -1, "softcap": 0.0, "alibi": False}
    c.update(kw)
    return {"name": name, **c}


def listed():
    """lo .. hi: tokens already cached, over the sequences of the batch;
    new_lo .. new_hi: tokens written, or read back, in each."""
    return [
        # One decode step's keys and values of 16 sequences: the smallest call.
        _case("write_token_b16", op="write", batch=16, n_q=32, n_kv=8, lo=1024, hi=4096, new_lo=1,
              new_hi=1),
        # A prompt of 8192 tokens after its prefill, 28 / 4 heads.
        _case("write_prompt_8192", op="write", new_lo=8192, new_hi=8192),
        # 16 prompts of 256 - 4096 tokens that continue ragged cached prefixes, 64-token blocks.
        _case("write_packed_b16", op="write", batch=16, n_q=32, n_kv=8, block=64, lo=0, hi=1000,
              new_lo=256, new_hi=4096),
        # A cached prefix of 1000 tokens handed back, 28 / 4 heads, contiguous cache.
        _case("read_prefix_1000", op="read", paged=False, lo=1000, hi=1000, new_lo=1000,
              new_hi=1000),
        # 16 sequences of 1024 - 8192 tokens read back (moved out of the cache).
        _case("read_packed_b16", op="read", batch=16, n_q=32, n_kv=8, lo=1024, hi=8192,
              new_lo=1024, new_hi=8192),
        # A chat's first steps: one short sequence.
        _case("decode_short", lo=300, hi=300),
        # One long sequence, contiguous cache: few rows, a long axis.
        _case("decode_30720", paged=False, block=64, lo=30720, hi=30720),
        # A batch of 16 sequences of 1024 - 32768 tokens, 32 / 8 heads, 16-token blocks.
        _case("decode_paged_b16", batch=16, n_q=32, n_kv=8, lo=1024, hi=32768),
        # Head_dim 256 with soft-capping and a sliding window, odd block size.
        _case("decode_d256_window", batch=4, n_q=16, n_kv=8, d=256, block=24, lo=2000, hi=9000,
              window=4095, softcap=50.0),
        # Many query heads on one kv head, head_dim 64, ALiBi, 128-token blocks.
        _case("decode_d64_g32_alibi", batch=8, n_q=64, n_kv=2, d=64, block=128, lo=100, hi=16000,
              alibi=True),
        # A decode step of one long sequence as a layer makes it: write the token, attend.
        _case("append_30720", op="append", lo=30719, hi=30719, new_lo=1, new_hi=1),
        # The same for 64 sequences.
        _case("append_b64", op="append", batch=64, n_q=32, n_kv=8, lo=500, hi=8000, new_lo=1,
              new_hi=1),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("write", "read", "decode", "decode", "append"))
    n_kv = rng.choice((1, 2, 4, 8))
    d = rng.choice((64, 128, 128, 256))
    g = rng.choice((1, 2, 4, 5, 7, 8, 16, 24, 48))
    batch = log(1, 64)
    # Tokens of the whole batch, at most those of the largest listed case.
    top = {"write": 35_000_000, "read": 70_000_000}.get(op, 250_000_000 // max(1, g // 8))
    top = max(64, top // (batch * n_kv * d))
    hi = log(1, min(top, 32768))
    lo = rng.randint(0, hi) if rng.random() < 0.8 else hi
    c = {"op": op, "batch": batch, "n_q": n_kv * g, "n_kv": n_kv, "d": d,
         "block": rng.choice((1, 8, 16, 16, 24, 32, 64, 100, 128, 256)),
         "paged": rng.random() < 0.7, "lo": lo, "hi": hi, "new_lo": 0, "new_hi": 0, "window": -1,
         "softcap": 0.0, "alibi": False}
    if op == "write":
        c["lo"], c["hi"] = 0, rng.randint(0, 300)
        c["new_lo"], c["new_hi"] = lo, hi
    elif op == "read":
        c["new_lo"], c["new_hi"] = lo, hi
    elif op == "append":
        c["new_lo"] = c["new_hi"] = 1
    if op in ("decode", "append"):
        kind = rng.choice(("plain", "plain", "window", "softcap", "alibi"))
        if kind == "window":
            c["window"] = log(1, 8192)
        elif kind == "softcap":
            c["softcap"] = float(rng.choice((20, 30, 50)))
        elif kind == "alibi":
            c["alibi"] = True
    return c


def _spread(lo, hi, n):
    """n lengths from lo to hi, both among them where n > 1, in no order."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7919 + n // 2) % n) // (n - 1) if math.gcd(7919, n) == 1
            else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    """(cached, new) tokens of each sequence.  read: a sequence's first `new`
    tokens are read, and those are what is cached."""
    cached = _spread(case["lo"], case["hi"], case["batch"])
    new = _spread(case["new_lo"], case["new_hi"], case["batch"])
    return cached, new


def _room(case):
    cached, new = _lens(case)
    if case["op"] in ("write", "append"):
        return [a + b for a, b in zip(cached, new)]
    return cached


def work(case):
    cached, new = _lens(case)
    n_kv, n_q, d, blk = case["n_kv"], case["n_q"], case["d"], case["block"]
    row = 2 * n_kv * d                                     # K and V of one token, in values
    if case["op"] == "write":
        t = sum(new)
        return {"bytes": t * row * 3 + 8 * n_kv * (t / blk + 1), "flops": 2 * t * row}
    if case["op"] == "read":
        t = sum(new)
        return {"bytes": t * row * 3 + 8 * n_kv * (t / blk + 1), "flops": t * row}
    if case["op"] == "append":
        cached = [a + 1 for a in cached]
    t = sum(min(a, case["window"] + 1) if case["window"] >= 0 else a for a in cached)
    b = t * row + 8 * n_kv * (t / blk + 1) + case["batch"] * n_q * (6 * d + 4)
    if case["op"] == "append":
        b += case["batch"] * row * 3
    return {"bytes": b, "flops": 4 * t * n_q * d}


def _pow2(k):
    """2^k as float32, k int32."""
    return ((k + 127) << 23).view(torch.float32)


def _exponent(amax):
    """Smallest k with amax <= 448 * 2^k, within the scale's range."""
    m, e = torch.frexp(amax)                               # amax = m 2^e, m in [0.5, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, k, K_MIN).clamp(K_MIN, K_MAX).to(torch.int32)


def _encode(x, scale):
    """e4m3 codes of x / scale, saturating; x float32, scale a power of two."""
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    B, n_q, n_kv, d, blk = case["batch"], case["n_q"], case["n_kv"], case["d"], case["block"]
    cached, new = _lens(case)
    room = _room(case)
    most = max(1, max(room))
    per_seq = -(-most // blk)
    # A few channels of the keys are larger than the rest, the same ones in every token.
    channel = 1.0 + 5.0 * (torch.rand(n_kv, d, generator=gen, device=dev) < 0.03)
    if case["paged"]:
        need = [-(-n // blk) for n in room]
        total = sum(need) + 2
        order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
        first = torch.tensor([sum(need[:b]) for b in range(B)], device=dev)
        at = first[:, None] + torch.arange(per_seq, device=dev)
        inside = torch.arange(per_seq, device=dev) < torch.tensor(need, device=dev)[:, None]
        table = torch.where(inside, order[at.clamp(max=total - 1)], 0).to(torch.int32)
        shape, sshape = (total, blk, n_kv, d), (total, n_kv)
    else:
        table, shape, sshape = None, (B, most, n_kv, d), (B, per_seq, n_kv)
    cache = {}
    for name, amp in (("k", channel), ("v", 1.0)):
        # What lies in the cache: written blocks of tokens, each with its scale.
        x = (randn(*shape) * amp).to(torch.bfloat16).float()
        if case["paged"]:
            scale = _pow2(_exponent(x.abs().amax(dim=(1, 3))))
            full = scale[:, None, :, None]
        else:
            pad = per_seq * blk - most
            a = torch.nn.functional.pad(x.abs().amax(dim=3), (0, 0, 0, pad))
            scale = _pow2(_exponent(a.view(B, per_seq, blk, n_kv).amax(dim=2)))
            full = scale.repeat_interleave(blk, dim=1)[:, :most, :, None]
        cache[name] = _encode(x, full).view(torch.uint8)
        cache[name + "s"] = scale.contiguous()
        del x, full
    s = {"case": case, "table": table, **cache,
         "lens": torch.tensor(cached, dtype=torch.int32, device=dev)}
    if case["op"] in ("write", "append"):
        t = sum(new)
        # A token in a hundred is larger than what its block holds so far.
        big = 1.0 + 7.0 * (torch.rand(t, generator=gen, device=dev) < 0.01)
        s["k_new"] = (randn(n_kv, t, d) * channel[:, None] * big[:, None]).to(torch.bfloat16)
        s["v_new"] = (randn(n_kv, t, d) * big[:, None]).to(torch.bfloat16)
        if case["op"] == "append":
            s["k_new"] = s["k_new"].transpose(0, 1).contiguous()
            s["v_new"] = s["v_new"].transpose(0, 1).contiguous()
    if case["op"] in ("write", "read"):
        cu = [sum(new[:i]) for i in range(B + 1)]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["total"] = cu[-1]
    if case["op"] in ("decode", "append"):
        s["q"] = randn(B, n_q, d).to(torch.bfloat16)
        s["most"] = most
        s["scale"] = 1.0 / math.sqrt(d)
        if case["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / n_q) for h in range(n_q)],
                                       dtype=torch.float32, device=dev)
    return s


def _own(s):
    import exact_io_aware_order_gb300 as attn

    case = s["case"]
    cache = (s["k"], s["v"], s["ks"], s["vs"])
    if case["op"] == "write":
        attn.cache_write_fp8(s["k_new"], s["v_new"], *cache, s["lens"], s["cu"], s["table"],
                             block_size=case["block"])
        return _cache(s)
    if case["op"] == "read":
        k, v = attn.cache_read_fp8(*cache, s["cu"], s["total"], s["table"],
                                   block_size=case["block"])
        return {"k": k, "v": v}
    variant = {"window_left": case["window"], "softcap": case["softcap"],
               "alibi_slopes": s.get("slopes")}
    if case["op"] == "decode":
        o, lse = attn.decode_fp8(s["q"], *cache, s["lens"], s["table"], block_size=case["block"],
                                 max_kv_len=s["most"], scale=s["scale"], **variant)
        return {"o": o, "lse": lse}
    o, lse = attn.decode_append_fp8(s["q"], s["k_new"], s["v_new"], *cache, s["lens"], s["table"],
                                    block_size=case["block"], max_kv_len=s["most"],
                                    scale=s["scale"], **variant)
    return {"o": o, "lse": lse, **_cache(s)}


def _cache(s):
    """The cache as the values it stands for (codes as e4m3 numbers) and its scales."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "ks": s["ks"], "vs": s["vs"]}


def _blocks(s):
    """Codes and scales by block: (blocks, block, n_kv, d) and (blocks, n_kv), and the block of
    each (sequence, index).  A contiguous cache's last blocks may be cut short: padded copies."""
    case = s["case"]
    if case["paged"]:
        return s["table"].long()
    B, per_seq = s["ks"].shape[:2]
    return torch.arange(B * per_seq, device=s["ks"].device).view(B, per_seq)


def _rows(s, seq, pos):
    """Row index into the cache viewed as (rows, n_kv, d), and into the scales as (blocks,
    n_kv), of position pos of sequence seq."""
    case = s["case"]
    block = _blocks(s)[seq, pos // case["block"]]
    if case["paged"]:
        return block * case["block"] + pos % case["block"], block
    return seq * s["k"].shape[1] + pos, block


def _plain_write(s, k_new, v_new, cu):
    """k_new, v_new: (n_kv, T, d)."""
    case = s["case"]
    blk, dev = case["block"], k_new.device
    t = torch.arange(k_new.shape[1], device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    lens = s["lens"].long()
    row, block = _rows(s, seq, lens[seq] + t - cu.long()[seq])
    # Blocks that hold earlier rows: each sequence's first, where it is not begun afresh.
    n_new = cu.long()[1:] - cu.long()[:-1]
    go = ((lens % blk > 0) & (n_new > 0)).nonzero()[:, 0]
    for x, codes, scales in ((k_new, s["k"], s["ks"]), (v_new, s["v"], s["vs"])):
        x = x.float().transpose(0, 1)                                        # (T, n_kv, d)
        flat = codes.view(-1, *codes.shape[-2:])
        sc = scales.view(-1, scales.shape[-1])
        amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(dim=2)           # (T, n_kv)
        top = torch.full_like(sc, -1.0).index_reduce_(0, block, amax, "amax")
        fresh = _pow2(_exponent(top.clamp(min=0.0)))
        first = lens[go] // blk
        old_pos = first[:, None] * blk + torch.arange(blk, device=dev)       # (n, block)
        ok = old_pos < lens[go][:, None]
        old_pos = torch.where(ok, old_pos, first[:, None] * blk)
        old_row, old_block = _rows(s, go[:, None].expand_as(old_pos), old_pos)
        was = sc[old_block[:, 0]]                                            # (n, n_kv)
        now = torch.maximum(was, fresh[old_block[:, 0]])
        fresh[old_block[:, 0]] = now
        old = flat[old_row].view(torch.float8_e4m3fn).float() * (was / now)[:, None, :, None]
        flat[old_row[ok]] = _encode(old, 1.0).view(torch.uint8)[ok]
        sc.copy_(torch.where(top >= 0, fresh, sc))
        flat[row] = _encode(x, sc[block][:, :, None]).view(torch.uint8)


def _plain_read(s):
    cu = s["cu"]
    t = torch.arange(s["total"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    row, block = _rows(s, seq, t - cu.long()[seq])
    out = {}
    for name in ("k", "v"):
        x = s[name].view(-1, *s[name].shape[-2:])[row].view(torch.float8_e4m3fn).float()
        sc = s[name + "s"].view(-1, s[name + "s"].shape[-1])[block]
        out[name] = (x * sc[:, :, None]).to(torch.bfloat16).transpose(0, 1).contiguous()
    return out


def _plain_decode(s, lens):
    case = s["case"]
    B, n_q, n_kv, d = case["batch"], case["n_q"], case["n_kv"], case["d"]
    g, L = n_q // n_kv, s["most"]
    pos = torch.arange(L, device=lens.device)
    seq = torch.arange(B, device=lens.device)
    row, block = _rows(s, seq[:, None], pos[None].expand(B, L))
    own_pos = lens.long()[:, None] - 1                                       # the query's position
    seen = pos[None] <= own_pos
    if case["window"] >= 0:
        seen = seen & (pos[None] >= own_pos - case["window"])

    def values(name):
        x = s[name].view(-1, n_kv, d)[row].view(torch.float8_e4m3fn).float()
        x = x * s[name + "s"].view(-1, n_kv)[block][..., None]
        return x.permute(0, 2, 1, 3)                                         # (B, n_kv, L, d)

    q = s["q"].float().view(B, n_kv, g, d)
    x = (q @ values("k").transpose(2, 3)) * s["scale"]                       # (B, n_kv, g, L)
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if case["alibi"]:
        x = x - s["slopes"].view(n_kv, g, 1) * (own_pos - pos[None])[:, None, None, :].float()
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    m = x.amax(dim=3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)                                  # a row that sees nothing
    p = torch.exp(x - m)
    l = p.sum(dim=3, keepdim=True)
    o = torch.where(l > 0, (p @ torch.where(seen[:, None, :, None], values("v"), 0.0)) / l, 0.0)
    return {"o": o.reshape(B, n_q, d), "lse": (m + torch.log(l)).reshape(B, n_q)}


def run(state):
    if own:
        return _own(state)
    s, op = state, state["case"]["op"]
    if op == "write":
        _plain_write(s, s["k_new"], s["v_new"], s["cu"])
        return _cache(s)
    if op == "read":
        return _plain_read(s)
    if op == "decode":
        return _plain_decode(s, s["lens"])
    one = torch.arange(s["case"]["batch"] + 1, dtype=torch.int32, device=s["lens"].device)
    _plain_write(s, s["k_new"].transpose(0, 1), s["v_new"].transpose(0, 1), one)
    return {**_plain_decode(s, s["lens"] + 1), **_cache(s)}


def exact(case, seed):
    """The operators' values in 64 bits: sequence by sequence, codes taken apart and rounded by
    their definition (sign, 4 exponent bits of bias 7, 3 mantissa bits; steps of 2^-9 below
    2^-6)."""
    s = prepare(case, seed)
    n_kv, n_q, d, blk = case["n_kv"], case["n_q"], case["d"], case["block"]
    f64 = torch.float64
    cached, new = _lens(case)

    def value(code):
        c = code.to(torch.int64)
        e, m = (c >> 3) & 15, (c & 7).to(f64)
        v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).to(f64)), m * 2.0 ** -9)
        v = torch.where((c & 127) == 127, torch.nan, v)
        return torch.where(c >= 128, -v, v)

    def rounded(x):
        a = x.abs().clamp(max=E4M3_MAX)
        e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
        e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
        step = torch.exp2(e - 3)
        return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), x)

    def place(b, lo, hi):
        """Where positions lo .. hi - 1 (of one block) of sequence b lie."""
        j = lo // blk
        if case["paged"]:
            p = int(s["table"][b, j])
            return (p, slice(lo - j * blk, hi - j * blk)), (p,)
        return (b, slice(lo, hi)), (b, j)

    vals = {n: value(s[n]) for n in ("k", "v")} if case["op"] in ("write", "append") else None
    scales = {n: s[n].to(f64) for n in ("ks", "vs")}
    if case["op"] in ("write", "append"):
        at = 0
        heads_first = case["op"] == "write"
        if sum(-(-n // blk) + 1 for n in new) > 12000:
            return None
        for b, n in enumerate(new):
            pos, end = cached[b], cached[b] + n
            while pos < end:
                stop = min(end, (pos // blk + 1) * blk)
                rows, sc = place(b, pos, stop)
                for name in ("k", "v"):
                    x = s[name + "_new"].to(f64)[:, at:at + stop - pos].transpose(0, 1) \
                        if heads_first else s[name + "_new"][at:at + stop - pos].to(f64)
                    top = x.abs().amax(dim=(0, 2))
                    k = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX))
                    k = torch.where(torch.exp2(k) * E4M3_MAX < top, k + 1, k)
                    k = torch.where(torch.exp2(k - 1) * E4M3_MAX >= top, k - 1, k)
                    now = torch.exp2(k.clamp(K_MIN, K_MAX))
                    if pos % blk:
                        was = scales[name + "s"][sc]
                        now = torch.maximum(now, was)
                        before, _ = place(b, pos // blk * blk, pos)
                        vals[name][before] = rounded(vals[name][before] * (was / now)[:, None])
                    scales[name + "s"][sc] = now
                    vals[name][rows] = rounded(x / now[:, None])
                at += stop - pos
                pos = stop
        state = {"k": vals["k"], "v": vals["v"], "ks": scales["ks"], "vs": scales["vs"]}
        if case["op"] == "write":
            return state

    def cached_values(name, b, n):
        """(n, n_kv, d) values of the first n tokens of sequence b."""
        src = vals[name] if vals is not None else s[name]
        sc = scales[name + "s"]
        if case["paged"]:
            ids = s["table"][b, :-(-n // blk)].long()
            c, f = src[ids], sc[ids][:, None, :, None]
            c = c if vals is not None else value(c)
            return (c * f).reshape(-1, n_kv, d)[:n]
        c = src[b, :n] if vals is not None else value(src[b, :n])
        return c * sc[b].repeat_interleave(blk, dim=0)[:n, :, None]

    if case["op"] == "read":
        return {name: torch.cat([cached_values(name, b, n) for b, n in enumerate(new)])
                .transpose(0, 1).contiguous() for name in ("k", "v")}
    outs, lses = [], []
    for b, n in enumerate(cached):
        n += case["op"] == "append"
        lo = max(0, n - 1 - case["window"]) if case["window"] >= 0 else 0
        if n == 0:
            outs.append(torch.zeros(n_q, d, dtype=f64, device=s["q"].device))
            lses.append(torch.full((n_q,), -math.inf, dtype=f64, device=s["q"].device))
            continue
        k = cached_values("k", b, n)[lo:].permute(1, 2, 0)                       # (n_kv, d, tokens)
        x = (s["q"][b].to(f64).view(n_kv, -1, d) @ k).reshape(n_q, -1) * s["scale"]
        del k
        if case["softcap"] > 0:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        if case["alibi"]:
            back = torch.arange(n - 1 - lo, -1, -1, dtype=f64, device=x.device)
            x = x - s["slopes"].to(f64)[:, None] * back
        lse = torch.logsumexp(x, dim=1)
        v = cached_values("v", b, n)[lo:].transpose(0, 1)                        # (n_kv, tokens, d)
        p = torch.exp(x - lse[:, None]).view(n_kv, n_q // n_kv, -1)
        outs.append((p @ v).reshape(n_q, d))
        lses.append(lse)
        del v
    out = {"o": torch.stack(outs), "lse": torch.stack(lses)}
    return {**out, **state} if case["op"] == "append" else out
