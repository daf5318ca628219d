"""Attention over the 8-bit cache, and its block moves, against the fp64
oracle on the values that the codes and scales stand for.

Tolerance on the float32 output, per element: the weights enter the second
product in fp16, each off by at most half a step, 2^-11 of itself (the sum
that divides them is exact), or in the decode of fp16 outputs, with its
residual, by 2^-22; scores and exponentials in fp32 move a weight
by less than 2^-16 (arguments below 2^7 rounded at 2^-24, 128 products
accumulated in fp32).  Both act on sum p |v|:
  |err| <= (2^-11 or 2^-22, + 2^-15) * sum_t p_t |v_t|  + tiny.
The 16-bit output must be the float32 one's rounding.
"""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from paged_kv_cache_383_b200 import workloads as wl

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
BF, HF = torch.bfloat16, torch.float16


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Pool:
    """A random 8-bit pool and tables for given contexts; slots and blocks
    that no sequence wrote hold NaN codes, their scales NaN."""

    def __init__(self, hkv, d, bs, ctx, *, seed=0, pow2=True, spread=2.0,
                 extra=4):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx = np.array(ctx, dtype=np.int32)
        nblk = -(-self.ctx // bs)
        need = int(nblk.sum())
        self.n = need + extra
        perm = rng.permutation(self.n).astype(np.int32)
        self.table = np.full((len(ctx), max(int(nblk.max()), 1)), -1,
                             dtype=np.int32)
        at, used = 0, np.zeros((self.n, bs), dtype=bool)
        for b, c in enumerate(nblk):
            self.table[b, :c] = perm[at:at + c]
            at += c
            for i, blk in enumerate(self.table[b, :c]):
                used[blk, :min(bs, int(ctx[b]) - i * bs)] = True
        shape = (self.n, hkv, bs, d)
        u = torch.from_numpy(used).cuda()[:, None, :, None]
        self.t = []
        for _ in "kv":
            c = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(
                -448, 448)
            c = torch.where(u, c, torch.full_like(c, float("nan"))).to(E4M3)
            e = torch.randn(shape[:2], generator=g, device="cuda") * spread
            s = 2.0 ** (torch.round(e) if pow2 else e) / 100
            if pow2:
                s = 2.0 ** torch.round(torch.log2(s))
            s = torch.where(u.any(2)[..., 0].expand_as(s), s,
                            torch.full_like(s, float("nan")))
            self.t.append((c, s.contiguous()))
        (self.kc, self.ks), (self.vc, self.vs) = self.t
        self.cache = (self.kc, self.vc, self.ks, self.vs)
        self.dev = [torch.from_numpy(x).cuda() for x in (self.table,
                                                         self.ctx)]

    def values(self):
        """fp64 K and V pools (NaN where nothing was written)."""
        return [to64(c) * to64(s)[:, :, None, None] for c, s in self.t]


def reference(pool, q, qpos, scale):
    """fp64 output and sum p |v| of each query row; qpos: (sequence, last
    visible position) per row."""
    kv, vv = pool.values()
    q = to64(q)
    hq, hkv = q.shape[1], kv.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    bs = kv.shape[2]
    for r, (b, p) in enumerate(qpos):
        if p < 0:
            continue
        for h in range(hkv):
            K = oa.depage(kv, pool.table[b], p + 1, h, bs)
            V = oa.depage(vv, pool.table[b], p + 1, h, bs)
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                out[r, g] = oa.attend(q[r, g], K, V, scale)
                mag[r, g] = oa.attend(q[r, g], K, np.abs(V), scale)
    return out, mag


def check(out32, out, ref, mag, dtype, rows=None):
    got = to64(out32)
    rel = (2.0 ** -11 if dtype == BF else 2.0 ** -22) + 2.0 ** -15
    ok = np.abs(got - ref) <= rel * mag + 1e-30
    if rows is not None:
        ok = ok[rows]
        assert torch.equal(out[rows], out32.to(dtype)[rows])
    else:
        assert torch.equal(out, out32.to(dtype))
    assert ok.all(), float((np.abs(got - ref) / (mag + 1e-30)).max())


def decode(pkv, pool, q, scale, **kw):
    out32 = torch.full(q.shape, float("nan"), device="cuda")
    out = torch.empty_like(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for o in (out32, out):
        pkv.pa_decode_q8(o, q, *pool.cache, *pool.dev, scale, dev_err=err,
                         **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out32, out


DECODE = [
    # dtype, hq, hkv, d, bs, ctx, kw
    (BF, 8, 8, 64, 16, [1], {}),
    (HF, 8, 8, 64, 16, [47, 612, 130, 1900], {}),
    (BF, 16, 2, 128, 16, [0, 1, 15, 16, 17, 100, 0], {}),
    (HF, 16, 2, 128, 32, [31, 32, 33, 1, 700], {}),
    (BF, 6, 2, 64, 32, [5, 90, 64], {}),
    (HF, 7, 1, 128, 16, [333, 2], {}),
    (BF, 64, 8, 128, 16, [900, 3, 1200], {"partition_size": 64}),
    (BF, 64, 8, 128, 16, [900, 3, 1200],
     {"partition_size": 64, "reduce": "kernel"}),
    (HF, 32, 8, 128, 32, [2049, 512, 513],
     {"partition_size": 512, "reduce": "kernel"}),
    (BF, 8, 1, 128, 16, [5000], {"partition_size": 16}),
    (HF, 4, 4, 64, 16, [3000, 700], {"partition_size": 2048,
                                     "reduce": "kernel"}),
    (BF, 8, 2, 64, 32, [4100, 2050], {"max_context_len": 4100}),
]


@pytest.mark.parametrize("case", DECODE,
                         ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}")
@pytest.mark.parametrize("pow2", [True, False])
def test_decode(pkv, case, pow2):
    dtype, hq, hkv, d, bs, ctx, kw = case
    pool = Pool(hkv, d, bs, ctx, seed=len(ctx), pow2=pow2)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(len(ctx), hq, d, generator=g, device="cuda").to(dtype)
    scale = d ** -0.5
    out32, out = decode(pkv, pool, q, scale, **kw)
    ref, mag = reference(pool, q, [(b, c - 1) for b, c in enumerate(ctx)],
                         scale)
    check(out32, out, ref, mag, dtype)
    assert (to64(out)[np.array(ctx) == 0] == 0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_decode_wide_ranges(pkv, dtype):
    """Scales of V that span 60 binades block by block, blocks of zeros with
    scale 0 among them, large and tiny queries, peaked scores."""
    ctx = [300, 77]
    pool = Pool(2, 128, 16, ctx, seed=8)
    n = pool.n
    e = torch.arange(n, device="cuda") * 37 % 61 - 30
    ok = ~torch.isnan(pool.vs)
    pool.vs.copy_(torch.where(ok, torch.exp2(e.float())[:, None].expand(n, 2),
                              pool.vs))
    for b in (int(pool.table[0, 3]), int(pool.table[1, 0])):
        pool.vc[b] = torch.zeros_like(pool.vc[b].float()).to(E4M3)
        pool.vs[b] = 0.0
    b = int(pool.table[0, 5])
    pool.kc[b] = torch.zeros_like(pool.kc[b].float()).to(E4M3)
    pool.ks[b] = 0.0
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(2, 16, 128, generator=g, device="cuda")
    q[:, 3] *= 50
    q[:, 4] *= 2.0 ** -13
    q[:, 5] = 0
    q[:, 6, 7] = 300  # one large element among small ones
    q = q.to(dtype)
    out32, out = decode(pkv, pool, q, 0.05)
    ref, mag = reference(pool, q, [(0, 299), (1, 76)], 0.05)
    got = to64(out32)
    # 300 / 50 times larger scores: arguments to 2^10, so 2^-13 on a weight;
    # and a weight below 2^-24 of the largest v in reach is rounded to it
    vmax = np.array([np.nanmax(np.abs(np.stack(
        [pool.values()[1][blk] for blk in pool.table[b][:-(-c // 16)]])))
        for b, c in enumerate(ctx)])
    tol = (2.0 ** -11 + 2.0 ** -12) * mag + \
        2.0 ** -24 * vmax[:, None, None] * 300
    assert (np.abs(got - ref) <= tol).all()
    assert torch.equal(out, out32.to(dtype)) or dtype == HF


def test_decode_nan_reaches_its_own_row_only(pkv):
    ctx = [40, 40]
    pool = Pool(1, 64, 16, ctx, seed=2)
    pool.kc[int(pool.table[0, 1]), 0, 3, 5] = torch.tensor(
        float("nan"), device="cuda").to(E4M3)
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    out32, _ = decode(pkv, pool, q, 0.125)
    assert torch.isnan(out32[0]).all() and torch.isfinite(out32[1]).all()


def test_decode_device_errors(pkv):
    from paged_kv_cache_383_b200 import _lib
    ctx = [40, 90, 20]
    for parts in (16, 64):
        for edit in ("id", "len", "negative"):
            pool = Pool(2, 64, 16, ctx, seed=6)
            q = torch.randn(3, 4, 64, device="cuda").to(HF)
            ref, mag = reference(pool, q, [(b, c - 1) for b, c in
                                           enumerate(ctx)], 0.125)
            if edit == "id":
                pool.dev[0][1, 2] = pool.n
            else:
                pool.dev[1][1] = 97 if edit == "len" else -1
            out = torch.zeros(3, 4, 64, device="cuda")
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            pkv.pa_decode_q8(out, q, *pool.cache, *pool.dev, 0.125,
                             partition_size=parts, dev_err=err)
            torch.cuda.synchronize()
            assert err.item() == _lib.PA_ERR_DEVICE_OOB
            for r in (0, 2):
                assert (np.abs(to64(out)[r] - ref[r]) <=
                        2.0 ** -14 * mag[r]).all()


def test_copy_and_swap(pkv):
    """Codes and scales move exactly, within a pool and to pinned host memory
    and back; bad pairs are flagged and skipped."""
    from paged_kv_cache_383_b200 import _lib
    for hkv, d, bs in ((8, 128, 16), (1, 64, 32), (3, 64, 16)):
        pool = Pool(hkv, d, bs, [200, 300], seed=4)
        k0, v0, ks0, vs0 = (t.clone() for t in pool.cache)
        pairs = torch.tensor([[0, 5], [1, 6], [0, 7], [99999, 2], [3, -1]],
                             dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.pa_copy_blocks_q8(*pool.cache, pairs, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == _lib.PA_ERR_DEVICE_OOB
        for t, t0 in zip(pool.cache, (k0, v0, ks0, vs0)):
            want = t0.clone().view(torch.uint8)
            for s, e in ((0, 5), (1, 6), (0, 7)):
                want[e] = t0.view(torch.uint8)[s]
            assert torch.equal(t.view(torch.uint8), want)
        host = [torch.zeros((4,) + t.shape[1:], dtype=torch.uint8 if
                            t.dtype == E4M3 else t.dtype).pin_memory()
                for t in pool.cache]
        host = [h.view(E4M3) if h.dtype == torch.uint8 else h for h in host]
        out = torch.tensor([[7, 0], [2, 3]], dtype=torch.int32, device="cuda")
        pkv.pa_swap_blocks_q8(*host, *pool.cache, out)
        back = torch.tensor([[0, 8], [3, 9]], dtype=torch.int32,
                            device="cuda")
        pkv.pa_swap_blocks_q8(*pool.cache, *host, back)
        torch.cuda.synchronize()
        for t, h in zip(pool.cache, host):
            u = t.view(torch.uint8)
            assert torch.equal(u[8], u[7]) and torch.equal(u[9], u[2])
            assert torch.equal(h.view(torch.uint8)[0], u[7].cpu())
    with pytest.raises(ValueError):
        pkv.pa_copy_blocks_q8(pool.kc, pool.vc, pool.ks.cpu(), pool.vs, pairs)
    with pytest.raises(TypeError):
        pkv.pa_copy_blocks_q8(pool.kc.view(torch.uint8),
                              pool.vc.view(torch.uint8), pool.ks, pool.vs,
                              pairs)


def test_python_refusals_on_device(pkv):
    pool = Pool(2, 64, 16, [20, 30], seed=1)
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        pkv.pa_decode_q8(q.cpu(), q, *pool.cache, *pool.dev, 1.0)
    with pytest.raises(TypeError):
        pkv.pa_decode_q8(q, q, pool.kc.view(torch.uint8), *pool.cache[1:],
                         *pool.dev, 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        pkv.pa_decode_q8(q, q, *pool.cache, pool.dev[0].t().contiguous().t(),
                         pool.dev[1], 1.0)
    with pytest.raises(ValueError, match="k_scales"):
        pkv.pa_decode_q8(q, q, pool.kc, pool.vc, pool.ks[:, :1], pool.vs,
                         *pool.dev, 1.0)
    with pytest.raises(pkv.PagedKVError):
        pkv.pa_decode_q8(q, q, *pool.cache, *pool.dev, 1.0,
                         workspace=torch.empty(
                             1, dtype=torch.uint8, device="cuda"))


def test_decode_on_another_stream(pkv):
    """Without a workspace, on a stream other than the current one, while the
    current stream allocates and writes."""
    pool = Pool(8, 128, 16, [1500] * 8, seed=5)
    q = torch.randn(8, 64, 128, device="cuda").to(BF)
    want, _ = decode(pkv, pool, q, 0.09, partition_size=64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (s, s.cuda_stream):
        for _ in range(10):
            out = torch.empty(q.shape, device="cuda")
            pkv.pa_decode_q8(out, q, *pool.cache, *pool.dev, 0.09,
                             partition_size=64, stream=stream)
            outs.append(out)
            torch.full((1 << 22,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_decode_workload(pkv):
    """The batch mix's lengths at a reduced batch, default options."""
    w = wl.WORKLOADS["llama3_70b_gqa8"].scaled(num_seqs=12, cap=3000)
    ctx = wl.draw_lengths(w, np.random.default_rng(1)).tolist()
    pool = Pool(8, 128, 16, ctx, seed=7, spread=0.5)
    q = torch.randn(12, 64, 128, device="cuda").to(BF)
    out32, out = decode(pkv, pool, q, 128 ** -0.5,
                        max_context_len=int(max(ctx)))
    ref, mag = reference(pool, q, [(b, c - 1) for b, c in enumerate(ctx)],
                         128 ** -0.5)
    check(out32, out, ref, mag, BF)


def prefill(pkv, pool, q, start, scale, max_q_len, **kw):
    qs = torch.from_numpy(np.asarray(start, dtype=np.int32)).cuda()
    out32 = torch.full(q.shape, float("nan"), device="cuda")
    out = torch.zeros_like(q)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for o in (out32, out):
        pkv.pa_prefill_q8(o, q, *pool.cache, *pool.dev, qs, scale,
                          max_q_len=max_q_len, dev_err=err, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out32, out


def positions(ctx, new):
    """(sequence, last visible position) of every query row."""
    return [(b, L - n + i) for b, (L, n) in enumerate(zip(ctx, new))
            for i in range(n)]


def bound_prefill(pool, q, qpos, scale, mag):
    """The error allowed to each element.

    Relative to sum p |v|: 2^-11 for a weight's rounding (no residual here,
    fp16 outputs too), 2^-15 as above, and the scores' own error where
    products are large: a score sums D products in D / 16 steps of the tensor
    core, each of which may drop a unit in the last place (2^-23) of a partial
    sum of at most A = max_t sum_d |q_d K_td|; the weight moves by that as the
    exponential's argument does, and the weights' sum by as much again:
    2 |scale| A (D / 16) 2^-23.

    Absolute: a weight 2^8 p vs / 2^E below fp16's normal range is off by up
    to half its smallest step, 2^-25, whatever its size; times 2^(E - 8) and
    the code, with 2^E at most the largest vs and the weights' sum at least 1:
    2^-33 max vs sum_t |vcode_t|."""
    kv, _ = pool.values()
    codes, vs = np.abs(to64(pool.vc)), to64(pool.vs)
    q = np.abs(to64(q))
    hq, hkv, d, bs = q.shape[1], kv.shape[1], q.shape[2], kv.shape[2]
    amp, low = np.zeros(q.shape[:2] + (1,)), np.zeros_like(q)
    for r, (b, p) in enumerate(qpos):
        used = pool.table[b][:-(-int(pool.ctx[b]) // bs)]
        for h in range(hkv):
            K = np.abs(oa.depage(kv, pool.table[b], p + 1, h, bs))
            c = oa.depage(codes, pool.table[b], p + 1, h, bs).sum(0)
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                amp[r, g] = (K @ q[r, g]).max()
                low[r, g] = 2.0 ** -33 * vs[used, h].max() * c
    rel = 2.0 ** -11 + 2.0 ** -15 + \
        2 * abs(scale) * amp * (d / 16) * 2.0 ** -23
    return rel * mag[:len(rel)] + low + 1e-30


def check_prefill(out32, out, ref, tol, n):
    got = to64(out32)[:n]
    assert (np.abs(got - ref[:n]) <= tol).all(), \
        float((np.abs(got - ref[:n]) / tol).max())
    assert torch.equal(out[:n], out32.to(out.dtype)[:n])


PREFILL = [
    # dtype, hq, hkv, d, bs, ctx, new
    (BF, 8, 8, 64, 16, [1], [1]),
    (HF, 2, 2, 128, 16, [130, 64, 65], [130, 64, 1]),
    (BF, 16, 2, 128, 16, [17, 200, 0, 63], [17, 3, 0, 63]),
    (HF, 8, 2, 128, 32, [300, 33, 95], [33, 33, 5]),
    (BF, 4, 2, 64, 32, [257, 90], [200, 1]),
    (HF, 8, 1, 64, 16, [100, 128, 31], [40, 128, 0]),
    (BF, 64, 8, 128, 16, [400, 1000], [4, 5]),
    (BF, 32, 8, 128, 32, [640], [97]),
    (HF, 1, 1, 128, 16, [500], [500]),
]


@pytest.mark.parametrize("case", PREFILL,
                         ids=lambda c: f"{c[1]}x{c[2]}x{c[3]}-{c[4]}")
@pytest.mark.parametrize("pow2", [True, False])
def test_prefill(pkv, case, pow2):
    dtype, hq, hkv, d, bs, ctx, new = case
    pool = Pool(hkv, d, bs, ctx, seed=len(ctx) + 20, pow2=pow2)
    n = sum(new)
    start = np.concatenate([[0], np.cumsum(new)])
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(n + 2, hq, d, generator=g, device="cuda").to(dtype)
    scale = d ** -0.5
    out32, out = prefill(pkv, pool, q, start, scale, max(new))
    ref, mag = reference(pool, q, positions(ctx, new), scale)
    tol = bound_prefill(pool, q[:n], positions(ctx, new), scale, mag)
    check_prefill(out32, out, ref, tol, n)
    assert torch.isnan(out32[n:]).all()  # rows behind the last sequence
    assert (out[n:] == 0).all()


@pytest.mark.parametrize("hq,hkv,new", [(16, 2, 16), (8, 1, 17), (4, 4, 128),
                                        (4, 4, 129), (8, 4, 3)])
def test_prefill_few_new_tokens(pkv, hq, hkv, new):
    """Up to 128 rows per KV head, where a sequence's keys are split between
    the query tiles, and just past it: contexts of one key tile, of two, of
    odd and even counts, ends inside and at the edge of a tile."""
    ctx = [new, new + 1, 64, 65, 127, 128, 129, 191, 193, 256, 640, 641]
    ctx = [max(c, new) for c in ctx] + [1]
    n = [new] * (len(ctx) - 1) + [1]
    n[5], n[8] = 1, min(2, new)
    pool = Pool(hkv, 128, 16, ctx, seed=hq + new)
    start = np.concatenate([[0], np.cumsum(n)])
    q = torch.randn(int(start[-1]), hq, 128, device="cuda").to(HF)
    out32, out = prefill(pkv, pool, q, start, 0.09, new)
    pos = positions(ctx, n)
    ref, mag = reference(pool, q, pos, 0.09)
    check_prefill(out32, out, ref, bound_prefill(pool, q, pos, 0.09, mag),
                  len(q))


def test_two_calls_at_once(pkv):
    """Two streams, each call with its own workspace, give what one call
    after the other gives."""
    pools = [Pool(4, 128, 16, [900, 33, 300], seed=s) for s in (50, 51)]
    qs = [torch.randn(60, 16, 128, device="cuda").to(BF) for _ in "12"]
    start = torch.tensor([0, 40, 53, 60], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in "12"]

    def both(streams):
        outs = []
        for pool, q, s in zip(pools, qs, streams):
            a, b = torch.empty_like(q), torch.empty_like(q[:3])
            pkv.pa_prefill_q8(a, q, *pool.cache, *pool.dev, start, 0.09,
                              max_q_len=40, stream=s)
            pkv.pa_decode_q8(b, q[:3], *pool.cache, *pool.dev, 0.09, stream=s)
            outs += [a, b]
        torch.cuda.synchronize()
        return outs
    torch.cuda.synchronize()
    one = both([None, None])
    for _ in range(5):
        for x, y in zip(one, both(streams)):
            assert torch.equal(x, y)


def test_prefill_many_items(pkv):
    """More work items than CTAs, of very unlike lengths."""
    rng = np.random.default_rng(5)
    ctx = rng.integers(1, 500, size=40).tolist()
    new = [int(rng.integers(0, c + 1)) for c in ctx]
    new[3] = 0
    pool = Pool(8, 64, 16, ctx, seed=40)
    start = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(int(start[-1]), 16, 64, device="cuda").to(BF)
    out32, out = prefill(pkv, pool, q, start, 0.125, max(new))
    rows = rng.choice(len(q), 60, replace=False)
    pos = positions(ctx, new)
    some = q[torch.from_numpy(rows).cuda()], [pos[r] for r in rows], 0.125
    ref, mag = reference(pool, *some)
    got = to64(out32)[rows]
    assert (np.abs(got - ref) <= bound_prefill(pool, *some, mag)).all()
    assert torch.equal(out, out32.to(BF))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_prefill_scales_and_ranges(pkv, scale):
    """Negative, zero and steep softmax scales; block scales that span 60
    binades, zeros among them; queries of unlike size."""
    ctx, new = [300, 77], [150, 9]
    pool = Pool(2, 128, 16, ctx, seed=9)
    e = torch.arange(pool.n, device="cuda") * 37 % 61 - 30
    ok = ~torch.isnan(pool.vs)
    pool.vs.copy_(torch.where(
        ok, torch.exp2(e.float())[:, None].expand(pool.n, 2), pool.vs))
    for c, s, b in ((pool.vc, pool.vs, pool.table[0, 3]),
                    (pool.kc, pool.ks, pool.table[0, 5])):
        c[int(b)] = torch.zeros_like(c[int(b)].float()).to(E4M3)
        s[int(b)] = 0.0
    q = torch.randn(159, 16, 128, device="cuda")
    q[:, 3] *= 8
    q[:, 4] *= 2.0 ** -13
    q[:, 5] = 0
    q = q.to(BF)
    start = [0, 150, 159]
    out32, out = prefill(pkv, pool, q, start, scale, 150)
    ref, mag = reference(pool, q, positions(ctx, new), scale)
    # and arguments up to 2^10, rounded at 2^-24: 2^-13 on a weight, twice
    tol = bound_prefill(pool, q, positions(ctx, new), scale, mag) + \
        2.0 ** -12 * mag
    assert (np.abs(to64(out32) - ref) <= tol).all()


def test_prefill_nan_reaches_its_own_rows_only(pkv):
    ctx, new = [70, 70], [10, 10]
    pool = Pool(1, 64, 16, ctx, seed=2)
    nan = torch.tensor(float("nan"), device="cuda").to(E4M3)
    pool.kc[int(pool.table[0, 4]), 0, 1, 5] = nan   # position 65
    q = torch.randn(20, 4, 64, device="cuda").to(BF)
    out32, _ = prefill(pkv, pool, q, [0, 10, 20], 0.125, 10)
    assert torch.isfinite(out32[:5]).all()      # positions 60 .. 64
    assert torch.isnan(out32[5:10]).all()
    assert torch.isfinite(out32[10:]).all()


def test_prefill_device_errors(pkv):
    from paged_kv_cache_383_b200 import _lib
    ctx, new = [40, 90, 20], [4, 70, 20]
    start = [0, 4, 74, 94]
    for edit in ("id", "len", "short", "max_q_len"):
        pool = Pool(2, 64, 16, ctx, seed=6)
        q = torch.randn(94, 4, 64, device="cuda").to(HF)
        ref, mag = reference(pool, q, positions(ctx, new), 0.125)
        tol = bound_prefill(pool, q, positions(ctx, new), 0.125, mag)
        m = 70
        if edit == "id":
            pool.dev[0][1, 2] = -3
        elif edit == "max_q_len":
            m = 60
        else:
            pool.dev[1][1] = 97 if edit == "len" else 60
        out = torch.zeros(94, 4, 64, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.pa_prefill_q8(
            out, q, *pool.cache, *pool.dev,
            torch.tensor(start, dtype=torch.int32, device="cuda"), 0.125,
            max_q_len=m, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == _lib.PA_ERR_DEVICE_OOB
        for r in list(range(4)) + list(range(74, 94)):
            assert (np.abs(to64(out)[r] - ref[r]) <= tol[r]).all()


def test_attention_in_a_graph(pkv):
    """Decode and prefill captured together, replayed after the cache, the
    lengths and the queries changed."""
    pool = Pool(2, 128, 16, [100, 40], seed=3)
    q1 = torch.randn(2, 8, 128, device="cuda").to(BF)
    q2 = torch.randn(10, 8, 128, device="cuda").to(BF)
    qs = torch.tensor([0, 7, 10], dtype=torch.int32, device="cuda")
    o = [torch.zeros_like(q1), torch.zeros_like(q2)]
    ws = [torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
          for _ in "12"]

    def step(out):
        pkv.pa_decode_q8(out[0], q1, *pool.cache, *pool.dev, 0.09,
                         max_context_len=112, workspace=ws[0])
        pkv.pa_prefill_q8(out[1], q2, *pool.cache, *pool.dev, qs, 0.09,
                          max_q_len=7, workspace=ws[1])
    step(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    for n in (100, 90, 65):
        pool.dev[1][0] = n
        q1.copy_(torch.randn_like(q1))
        q2.copy_(torch.randn_like(q2))
        pool.vs *= 2
        graph.replay()
        want = [torch.zeros_like(q1), torch.zeros_like(q2)]
        step(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_prefill_of_one_token_is_decode(pkv):
    """One new token per sequence: the two kernels agree to their rounding."""
    ctx = [5, 100, 777, 64]
    pool = Pool(4, 128, 32, ctx, seed=11)
    q = torch.randn(4, 16, 128, device="cuda").to(HF)
    a, _ = decode(pkv, pool, q, 0.09)
    b, _ = prefill(pkv, pool, q, [0, 1, 2, 3, 4], 0.09, 1)
    pos = [(i, c - 1) for i, c in enumerate(ctx)]
    _, mag = reference(pool, q, pos, 0.09)
    tol = 2 * bound_prefill(pool, q, pos, 0.09, mag)  # one's, the other's
    assert (np.abs(to64(a) - to64(b)) <= tol).all()
