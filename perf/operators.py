"""Operators of an 8-bit paged KV cache and of the append that fills a paged cache: real work, in its plain form and
through the framework's calls.

* ``append``      norm (optional) and rotation of new queries and keys, keys and values into the 16-bit paged cache
* ``append_q8``   the same into a cache of e4m3 codes with one scale for each (block, KV head) of K and of V
* ``decode_q8``   one query per sequence over that cache
* ``prefill_q8``  several new tokens per sequence over it, causal
* ``copy_q8``     copy-on-write of its blocks

A case's lengths come from its own ``len_seed`` (so its work is known without its inputs); values come from the seed of
``prepare``.  Codes are returned as the float8 tensors that the cache holds, with the float32 scales beside them.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # one user's next token behind a short context: the smallest append there is (latency)
        dict(name="append one token", op="append", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=1, ctx_lo=333, ctx_hi=333,
             q_lo=1, q_hi=1, rot=128, layout="half", norm=False, base=500000.0, far=1.0, len_seed=1),
        # a chunked prefill step: 512-token chunks of 16 prompts of 2048 to 8192 tokens, 70B heads, with norms
        dict(name="append 16 chunks", op="append", dtype="bf16", hq=64, hkv=8, d=128, bs=16, seqs=16, ctx_lo=2048, ctx_hi=8192,
             q_lo=448, q_hi=512, rot=128, layout="half", norm=True, base=500000.0, far=8.0, len_seed=2),
        # one decode step of a batch of 256, 70B heads, 8-bit cache
        dict(name="append q8 batch 256", op="append_q8", dtype="bf16", hq=64, hkv=8, d=128, bs=16, seqs=256, ctx_lo=1, ctx_hi=700,
             q_lo=1, q_hi=1, rot=128, layout="half", norm=True, base=500000.0, far=1.0, len_seed=3),
        # whole prompts of ragged length into fresh blocks of 32, interleaved rotation of half the head, fp16
        dict(name="append q8 prompts", op="append_q8", dtype="fp16", hq=32, hkv=8, d=128, bs=32, seqs=8, ctx_lo=300, ctx_hi=4096,
             q_lo=300, q_hi=4096, rot=64, layout="interleaved", norm=False, base=10000.0, far=1.0, len_seed=4),
        # the four short sequences of the tiny workload (head_dim 64, no grouping): latency
        dict(name="decode q8 tiny", op="decode_q8", dtype="fp16", hq=8, hkv=8, d=64, bs=16, seqs=4, ctx_lo=47, ctx_hi=1900,
             q_lo=1, q_hi=1, len_seed=5),
        # the batch-256 serving mix: 70B heads, contexts spread over 1 to 8192 tokens
        dict(name="decode q8 batch 256", op="decode_q8", dtype="bf16", hq=64, hkv=8, d=128, bs=16, seqs=256, ctx_lo=120, ctx_hi=8192,
             q_lo=1, q_hi=1, len_seed=6),
        # eight long contexts, block 32, fp16: the work has to be split along the context
        dict(name="decode q8 long", op="decode_q8", dtype="fp16", hq=64, hkv=8, d=128, bs=32, seqs=8, ctx_lo=32768, ctx_hi=131072,
             q_lo=1, q_hi=1, len_seed=7),
        # speculative verification: a few draft tokens of 64 sequences over 128 to 4096 cached ones, 8B heads
        dict(name="prefill q8 drafts", op="prefill_q8", dtype="bf16", hq=32, hkv=8, d=128, bs=16, seqs=64, ctx_lo=128, ctx_hi=4096,
             q_lo=2, q_hi=5, len_seed=8),
        # chunks of 512 appended to what is cached, 70B heads
        dict(name="prefill q8 chunks", op="prefill_q8", dtype="bf16", hq=64, hkv=8, d=128, bs=16, seqs=8, ctx_lo=2048, ctx_hi=8192,
             q_lo=512, q_hi=512, len_seed=9),
        # whole prompts of odd lengths, fp16, block 32
        dict(name="prefill q8 prompts", op="prefill_q8", dtype="fp16", hq=32, hkv=8, d=128, bs=32, seqs=4, ctx_lo=1000, ctx_hi=4095,
             q_lo=4096, q_hi=4096, len_seed=10),
        # one fork's partly filled block
        dict(name="copy q8 one block", op="copy_q8", dtype="bf16", hkv=8, d=128, bs=16, pool=256, pairs=1),
        # 127 sequences fork from one prefix at once, several groups of them
        dict(name="copy q8 forks", op="copy_q8", dtype="bf16", hkv=8, d=128, bs=16, pool=8192, pairs=2540),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "append_q8", "decode_q8", "decode_q8", "prefill_q8", "prefill_q8", "copy_q8"])
    dtype, d, bs = rng.choice(["bf16", "fp16"]), rng.choice([64, 128, 128]), rng.choice([16, 32])
    hkv = rng.choice([1, 2, 4, 8, 8])
    seed = rng.randrange(1 << 30)
    if op == "copy_q8":
        n = _log(rng, 1, 2540)
        return dict(op=op, dtype=dtype, hkv=hkv, d=d, bs=bs, pool=2 * n + _log(rng, 8, 2000), pairs=n)
    c = dict(op=op, dtype=dtype, hkv=hkv, d=d, bs=bs, len_seed=seed)
    if op in ("append", "append_q8"):
        c.update(hq=hkv * rng.choice([1, 2, 4, 5, 8]), rot=rng.choice([d, d, d // 2, 32, 48]), layout=rng.choice(["half", "interleaved"]),
                 norm=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]), far=rng.choice([1.0, 1.0, 8.0]))
        if rng.random() < 0.4:  # a decode step
            c.update(seqs=_log(rng, 1, 256), ctx_lo=1, ctx_hi=_log(rng, 20, 1500), q_lo=1, q_hi=1)
        else:
            hi = _log(rng, 20, 4096)
            c.update(seqs=_log(rng, 1, 16), ctx_lo=max(1, hi // 8), ctx_hi=hi, q_lo=1, q_hi=_log(rng, 2, 1024))
    elif op == "decode_q8":
        c.update(hq=hkv * rng.choice([1, 2, 3, 4, 7, 8]), q_lo=1, q_hi=1)
        seqs = _log(rng, 1, 256)
        hi = min(131072, _log(rng, 64, 500000 // seqs + 64))
        c.update(seqs=seqs, ctx_lo=max(1, hi // 20), ctx_hi=hi)
    else:
        c.update(hq=hkv * rng.choice([1, 2, 4, 8]))
        if rng.random() < 0.4:  # draft tokens
            c.update(seqs=_log(rng, 1, 64), ctx_lo=16, ctx_hi=_log(rng, 64, 4096), q_lo=1, q_hi=rng.randrange(2, 9))
        else:
            hi = _log(rng, 100, 4096)
            c.update(seqs=_log(rng, 1, 6), ctx_lo=max(1, hi // 3), ctx_hi=hi, q_lo=1, q_hi=_log(rng, 16, 2048))
    return c


def _lengths(c):
    """Context lengths (the new tokens included) and new tokens of each sequence: both known from the case alone."""
    r = random.Random(c["len_seed"])
    ctx = [_log(r, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    new = [min(n, r.randint(c["q_lo"], c["q_hi"])) for n in ctx]
    return ctx, new


def _freqs(c):
    """Angle per position of each rotated pair, in 64 bits; `far` > 1 scales them linearly for long contexts."""
    j = torch.arange(c["rot"] // 2, dtype=torch.float64)
    return c["base"] ** (-2.0 * j / c["rot"]) / c["far"]


def _need(amax):
    """The smallest power of two s with amax <= 448 s (as a float32 tensor), from the exponent: no rounding."""
    m, x = torch.frexp(amax.float())
    e = torch.where(amax > 0, x - 9 + (m > 0.875).to(x.dtype), torch.full_like(x, -64)).clamp(-64, 120)
    return torch.ldexp(torch.ones_like(m), e)


def _codes(g, n, h, bs, d):
    """Codes and scales of a pool in use: values with channels of unlike size and tokens of unlike size."""
    dev = "cuda"
    codes, scales = torch.empty(n, h, bs, d, dtype=E4M3, device=dev), torch.empty(n, h, device=dev)
    gain = torch.exp(0.4 * torch.randn(h, 1, d, generator=g, device=dev))
    step = max(1, (1 << 26) // (h * bs * d))
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), h, bs, d, generator=g, device=dev) * gain
        x *= torch.exp(0.5 * torch.randn(x.shape[0], h, 1, 1, generator=g, device=dev))
        s = _need(x.abs().amax((2, 3)))
        codes[i:i + step] = (x / s[:, :, None, None]).to(E4M3)
        scales[i:i + step] = s
    return codes, scales


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]
    s = {"case": c, "scale": c["d"] ** -0.5}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "copy_q8":
        for x in "kv":
            s[x + "_cache"], s[x + "_scales"] = _codes(g, c["pool"], c["hkv"], c["bs"], c["d"])
        perm = torch.randperm(c["pool"], generator=g, device=dev)[:2 * c["pairs"]].to(torch.int32)
        src = perm[:c["pairs"]]
        if c["pairs"] > 127:  # many forks share a source
            src = src[:c["pairs"] // 127].repeat_interleave(127)[:c["pairs"]]
            src = torch.cat([src, perm[:c["pairs"] - src.numel()]])
        s["pairs"] = torch.stack([src, perm[c["pairs"]:]], 1).contiguous()
        return s
    ctx, new = _lengths(c)
    bs, h, d = c["bs"], c["hkv"], c["d"]
    blocks = [-(-n // bs) for n in ctx]
    pool = sum(blocks) + sum(blocks) // 8 + 1
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((len(ctx), max(blocks)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    start = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32)
    s["table"], s["ctx"], s["start"] = table.to(dev), torch.tensor(ctx, dtype=torch.int32).to(dev), start.to(dev)
    s["rows"], s["max_new"], s["max_ctx"] = sum(new), max(new), max(ctx)
    rows = s["rows"]
    if c["op"] in ("append", "append_q8"):
        # one projection's output: the rows of q, k and v lie side by side
        qkv = (randn(rows, c["hq"] + 2 * h, d) * torch.exp(0.4 * randn(1, c["hq"] + 2 * h, d))).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + h], qkv[:, c["hq"] + h:]
        s["q_norm"] = (1 + 0.2 * randn(d)).to(dt) if c["norm"] else None
        s["k_norm"] = (1 + 0.2 * randn(d)).to(dt) if c["norm"] else None
        s["freqs"] = _freqs(c).to(dev)
        s["q_out"] = torch.empty(rows, c["hq"], d, dtype=dt, device=dev)
        if c["op"] == "append":
            s["k_cache"], s["v_cache"] = randn(pool, h, bs, d).to(dt), randn(pool, h, bs, d).to(dt)
        else:
            for x in "kv":
                s[x + "_cache"], s[x + "_scales"] = _codes(g, pool, h, bs, d)
        return s
    for x in "kv":
        s[x + "_cache"], s[x + "_scales"] = _codes(g, pool, h, bs, d)
    s["q"] = randn(rows, c["hq"], d).to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---- the plain forms --------------------------------------------------------------------------------------------------

def _places(s):
    """For each row: its sequence, position, block and offset."""
    start, ctx = s["start"].long(), s["ctx"].long()
    new = start[1:] - start[:-1]
    b = torch.repeat_interleave(torch.arange(ctx.numel(), device=ctx.device), new, output_size=s["rows"])
    pos = (ctx - new)[b] + torch.arange(s["rows"], device=ctx.device) - start[b]
    bs = s["case"]["bs"]
    return pos, s["table"][b, pos // bs].long(), pos % bs


def _norm_rotate(x, weight, pos, s):
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    a = pos.double()[:, None, None] * s["freqs"]
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    r, rest = c["rot"], x[..., c["rot"]:]
    if c["layout"] == "half":
        u, w = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([u * cos - w * sin, w * cos + u * sin, rest], -1)
    u, w = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2), rest], -1)


def _append_plain(s):
    pos, blk, off = _places(s)
    q = _norm_rotate(s["q"], s["q_norm"], pos, s).to(s["q"].dtype)
    k = _norm_rotate(s["k"], s["k_norm"], pos, s)
    s["k_cache"][blk, :, off] = k.to(s["q"].dtype)
    s["v_cache"][blk, :, off] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _quantise(s, x, blk, off, cache, scales):
    """Rows x [rows, heads, dim] into cache (codes) and scales, in place."""
    n, bs = cache.shape[0], cache.shape[2]
    idx = blk[:, None].expand(-1, x.shape[1])
    amax = torch.zeros_like(scales).scatter_reduce(0, idx, x.abs().amax(-1), "amax")
    first = torch.full((n,), bs, dtype=torch.long, device=x.device).scatter_reduce(0, blk, off, "amin")
    new = torch.maximum(_need(amax), torch.where((first == 0)[:, None], torch.zeros_like(scales), scales))
    new = torch.where((first == bs)[:, None], scales, new)
    # a sequence's first new token may join a block that holds older ones: their codes follow the scale
    start, ctx = s["start"].long(), s["ctx"].long()
    p0 = ctx - (start[1:] - start[:-1])
    page = s["table"].gather(1, (p0 // bs).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    raw = cache.view(torch.uint8)
    old = raw[page].view(E4M3).float()
    moved = (old * (scales[page] / new[page])[:, :, None, None]).to(E4M3).view(torch.uint8)
    keep = torch.arange(bs, device=x.device) >= torch.where(first[page] < bs, first[page], 0)[:, None]
    raw[page] = torch.where(keep[:, None, :, None], raw[page], moved)
    raw[blk, :, off] = (x / new[blk][..., None]).to(E4M3).view(torch.uint8)
    scales.copy_(new)


def _append_q8_plain(s):
    pos, blk, off = _places(s)
    q = _norm_rotate(s["q"], s["q_norm"], pos, s).to(s["q"].dtype)
    _quantise(s, _norm_rotate(s["k"], s["k_norm"], pos, s), blk, off, s["k_cache"], s["k_scales"])
    _quantise(s, s["v"].float(), blk, off, s["v_cache"], s["v_scales"])
    return q, s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _gather(s, x):
    """The sequences' values in 32 bits: [sequence, head, padded position, dim]."""
    t = s["table"].clamp(min=0).long()
    v = s[x + "_cache"].view(torch.uint8)[t].view(E4M3).float() * s[x + "_scales"][t][..., None, None]
    return v.transpose(1, 2).flatten(2, 3)


def _attend(s, q, pos):
    """q [sequence, head, query, dim] in 32 bits at positions pos [sequence, query]."""
    c = s["case"]
    h, group, n = c["hkv"], c["hq"] // c["hkv"], q.shape[2]
    sc = torch.matmul(q.reshape(q.shape[0], h, group * n, -1) * s["scale"], _gather(s, "k").transpose(2, 3))
    seen = torch.arange(sc.shape[-1], device=q.device) <= pos[..., None]
    sc = sc.unflatten(2, (group, n)).masked_fill_(~seen[:, None, None], -math.inf)
    sc = torch.exp(sc.sub_(sc.amax(-1, keepdim=True)))
    sc = sc.div_(sc.sum(-1, keepdim=True))
    v = _gather(s, "v")
    seen = torch.arange(v.shape[2], device=q.device) < s["ctx"][:, None]  # codes that no token has written are no values
    v = torch.where(seen[:, None, :, None], v, 0.0)
    return torch.matmul(sc.flatten(2, 3), v).unflatten(2, (group, n)).flatten(1, 2)


def _decode_plain(s):
    return _attend(s, s["q"].float()[:, :, None], s["ctx"].long()[:, None] - 1)[:, :, 0].to(s["q"].dtype)


def _prefill_plain(s):
    start, ctx = s["start"].long(), s["ctx"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(s["max_new"], device=ctx.device)
    rows = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    o = _attend(s, s["q"].float()[rows].transpose(1, 2), (ctx - new)[:, None] + i)
    b = torch.repeat_interleave(torch.arange(ctx.numel(), device=ctx.device), new, output_size=s["rows"])
    return o.transpose(1, 2)[b, torch.arange(s["rows"], device=ctx.device) - start[b]].to(s["q"].dtype)


def _copy_plain(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    for x in "kv":
        raw = s[x + "_cache"].view(torch.uint8)
        raw[dst] = raw[src]
        s[x + "_scales"][dst] = s[x + "_scales"][src]
    return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


PLAIN = {"append": _append_plain, "append_q8": _append_q8_plain, "decode_q8": _decode_plain, "prefill_q8": _prefill_plain,
         "copy_q8": _copy_plain}


# ---- the framework's calls ----------------------------------------------------------------------------------------------

def _own(s):
    import paged_kv_cache_383_b200 as pkv
    op = s["case"]["op"]
    if op in ("append", "append_q8"):
        kw = dict(max_q_len=s["max_new"], q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=EPS, rope_freqs=s["freqs"],
                  rope_layout=s["case"]["layout"])
        start = s["start"] if s["max_new"] > 1 else None  # a decode step: one row for each sequence
        if op == "append":
            pkv.pa_append(s["q_out"], s["k_cache"], s["v_cache"], s["q"], s["k"], s["v"], s["table"], s["ctx"], start, **kw)
            return s["q_out"], s["k_cache"], s["v_cache"]
        pkv.pa_append_q8(s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["q"], s["k"], s["v"],
                         s["table"], s["ctx"], start, **kw)
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    cache = (s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
    if op == "decode_q8":
        return pkv.pa_decode_q8(s["out"], s["q"], *cache, s["table"], s["ctx"], s["scale"], max_context_len=s["max_ctx"])
    if op == "prefill_q8":
        return pkv.pa_prefill_q8(s["out"], s["q"], *cache, s["table"], s["ctx"], s["start"], s["scale"], max_q_len=s["max_new"],
                                 max_context_len=s["max_ctx"])
    pkv.pa_copy_blocks_q8(*cache, s["pairs"])
    return cache


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------------

def work(case):
    c = case
    h, d = c["hkv"], c["d"]
    if c["op"] == "copy_q8":
        n = c["pairs"]
        read = n if n <= 127 else max(n // 127, n % 127)  # forks of one source read it once
        return {"bytes": (read + n) * 2 * (h * c["bs"] * d + 4 * h), "flops": 0}
    ctx, new = _lengths(c)
    rows, hq, bs = sum(new), c["hq"], c["bs"]
    if c["op"] in ("append", "append_q8"):
        read = 2 * rows * d * (hq + 2 * h)
        if c["op"] == "append":
            write = read
        else:
            touched = sum((n - 1) // bs - (n - m) // bs + 1 for n, m in zip(ctx, new) if m)
            write = 2 * rows * d * hq + 2 * rows * d * h + 2 * 2 * 4 * h * touched
        return {"bytes": read + write, "flops": 10 * rows * d * (hq + h)}
    kv = sum(2 * n * h * d + 2 * -(-n // bs) * h * 4 for n in ctx)
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(ctx, new))
    return {"bytes": kv + 2 * 2 * rows * hq * d, "flops": 4 * hq * d * pairs}


# ---- in 64 bits ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    """What run returns, in 64 bits: new codes as the unrounded value in units of the block's scale, old ones as they move."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "copy_q8":
        k, v, ks, vs = (s[n].double() for n in ("k_cache", "v_cache", "k_scales", "v_scales"))
        for a, b in s["pairs"].tolist():
            for x in (k, v, ks, vs):
                x[b] = x[a]
        return k, v, ks, vs
    ctx, new = _lengths(c)
    table, bs, h = s["table"].cpu(), c["bs"], c["hkv"]
    group = c["hq"] // h
    at = 0
    if c["op"] in ("append", "append_q8"):
        q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        k, v = s["k_cache"].double(), s["v_cache"].double()
        ks = s["k_scales"].double() if c["op"] == "append_q8" else None
        vs = s["v_scales"].double() if c["op"] == "append_q8" else None
        for b, (n, m) in enumerate(zip(ctx, new)):
            p = torch.arange(n - m, n, dtype=torch.float64, device="cuda")
            z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p[:, None] * s["freqs"])[:, None]
            made = []
            for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
                y = x[at:at + m].double()
                if w is not None:
                    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
                r = c["rot"]
                pair = y[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else y[..., :r].unflatten(-1, (r // 2, 2))
                turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
                turned = turned.transpose(-1, -2) if c["layout"] == "half" else turned
                made.append(torch.cat([turned.flatten(-2), y[..., r:]], -1))
            q_out[at:at + m] = made[0]
            for x, cache, scale in ((made[1], k, ks), (s["v"][at:at + m].double(), v, vs)):
                i = 0
                while i < m:
                    pos = n - m + i
                    o, blk = pos % bs, int(table[b, pos // bs])
                    j = min(m, i + bs - o)
                    rows = x[i:j].transpose(0, 1)
                    if scale is not None:
                        top = rows.abs().amax((1, 2)).clamp(min=448 * 2.0 ** -64)
                        f = torch.exp2(torch.floor(torch.log2(top)) - 9)  # at most half of what is needed: doubled until it is enough
                        for _ in range(3):
                            f = torch.where(top > 448 * f, 2 * f, f)
                        if o:
                            f = torch.maximum(f, scale[blk])
                            cache[blk, :, :o] *= (scale[blk] / f)[:, None, None]
                        scale[blk] = f
                        rows = rows / f[:, None, None]
                    cache[blk, :, o:o + j - i] = rows
                    i = j
            at += m
        return (q_out, k, v) if ks is None else (q_out, k, v, ks, vs)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(ctx, new)):
        ids = s["table"][b, :-(-n // bs)].long()
        for kv in range(h):
            k, v = (((s[x + "_cache"].view(torch.uint8)[ids, kv].view(E4M3).double()) * s[x + "_scales"][ids, kv].double()[:, None, None])
                    .flatten(0, 1)[:n] for x in "kv")
            q = s["q"][at:at + m, kv * group:(kv + 1) * group].double()
            w = torch.einsum("mgd,nd->mgn", q, k) * s["scale"]
            last = torch.arange(n - m, n, device="cuda")[:, None, None]
            w = torch.where(torch.arange(n, device="cuda") <= last, w, -math.inf)
            out[at:at + m, kv * group:(kv + 1) * group] = torch.softmax(w, -1) @ v
        at += m
    return out
