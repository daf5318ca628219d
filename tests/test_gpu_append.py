"""pa_append and pa_append_q8 against the fp64 oracle.

Tolerances.  Before its one rounding a value is computed in fp32: at most a
few dozen roundings of 2^-24 (the norm's sum of 128 squares as a tree of 12,
halved by the square root, rsqrt, two products; the angle's fraction of a turn
rounded once, 2 pi 2^-25 in the angle; sine, cosine, two products and a sum),
which stays below 2^-20 of the magnitudes that enter it: |u| + |w| of the
rotated pair.  Then half a step of the type: eps / 2 of the value (16 bits),
half the distance of e4m3 values (codes).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import append as oap

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -20
E4M3 = torch.float8_e4m3fn


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Batch:
    """One append call: ragged sequences (an empty one and a padding one among
    them), rows behind the last sequence, tables whose unused entries are -1,
    and inputs that are slices of one projection."""

    def __init__(self, dtype, hq, hkv, d, bs, ctx, new, *, norm, rot, layout,
                 rope_scale=1.0, seed=0, spare_rows=2, pool=None,
                 max_blocks=None, far=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.hq, self.hkv, self.d, self.bs = dtype, hq, hkv, d, bs
        self.ctx = np.array(ctx, dtype=np.int32)
        self.new = np.array(new, dtype=np.int32)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(self.start[-1]) + spare_rows
        nblk = -(-self.ctx // bs)
        width = max_blocks or max(int(nblk.max()), 1)
        self.table = np.full((len(ctx), width), -1, dtype=np.int32)
        # Blocks the call writes; others stay -1: it must not read them.
        need = [(b, i) for b in range(len(ctx)) if ctx[b] and new[b]
                for i in range((ctx[b] - new[b]) // bs, nblk[b])]
        self.pool = pool or len(need) + 3
        for (b, i), blk in zip(need, rng.permutation(self.pool)[:len(need)]):
            self.table[b, i] = blk
        wide = torch.randn(rows, hq + 2 * hkv, d, generator=g, device="cuda")
        wide = (wide * torch.exp(torch.randn(rows, 1, 1, generator=g,
                                             device="cuda"))).to(dtype)
        self.q, self.k, self.v = wide[:, :hq], wide[:, hq:hq + hkv], \
            wide[:, hq + hkv:]
        w = torch.randn(2, d, generator=g, device="cuda").to(dtype)
        self.q_norm, self.k_norm = (w[0].clone(), w[1].clone()) if norm else \
            (None, None)
        self.freqs = None if rot == 0 else torch.tensor(
            10000.0 ** (-2 * np.arange(rot // 2) / rot), device="cuda",
            dtype=torch.float64)
        self.kw = dict(q_norm=self.q_norm, k_norm=self.k_norm, norm_eps=1e-5,
                       rope_freqs=self.freqs, rope_layout=layout,
                       rope_scale=rope_scale)
        self.shape = (self.pool, hkv, bs, d)
        self.g = g

    def args(self, with_start=True):
        t = [torch.from_numpy(x).cuda() for x in (self.table, self.ctx)]
        return t + [torch.from_numpy(self.start).cuda() if with_start
                    else None]

    def places(self):
        return list(oap.placed(self.ctx, self.start, self.table, self.bs))

    def expected(self, x, norm):
        """(unrounded rows in fp64, magnitudes that entered each value)."""
        f = None if self.freqs is None else self.freqs.cpu().numpy()
        y = oap.norm_head(to64(x), None if norm is None else to64(norm), 1e-5)
        out, mag = np.zeros_like(y), np.abs(y)
        for b, row, p, _, _ in self.places():
            out[row] = oap.rotate_head(y[row], p, f, self.kw["rope_layout"],
                                       self.kw["rope_scale"])
            if f is not None:
                r = len(f)
                a = np.abs(y[row])
                if self.kw["rope_layout"] == "half":
                    m = a[:, :r] + a[:, r:2 * r]
                    mag[row, :, :2 * r] = np.concatenate([m, m], -1)
                else:
                    m = a[:, 0:2 * r:2] + a[:, 1:2 * r:2]
                    mag[row, :, :2 * r] = np.repeat(m, 2, -1)
        return out, mag * max(1.0, abs(self.kw["rope_scale"]))

    def check_q(self, q_out, before):
        want, mag = self.expected(self.q, self.q_norm)
        got = to64(q_out)
        tol = np.abs(want) * torch.finfo(self.dtype).eps / 2 + FP32 * mag \
            + torch.finfo(self.dtype).smallest_normal * 2.0 ** -8
        rows = sorted({row for _, row, *_ in self.places()})
        assert (np.abs(got - want)[rows] <= tol[rows]).all()
        rest = sorted(set(range(len(got))) - set(rows))
        assert torch.equal(q_out[rest], before[rest])


SHAPES = [
    # dtype, hq, hkv, d, bs, ctx, new, norm, rot, layout, rope_scale
    (torch.bfloat16, 8, 2, 128, 16, [1], [1], False, 128, "half", 1.0),
    (torch.float16, 4, 4, 64, 16, [40, 0, 33, 17], [5, 0, 33, 0], True, 64,
     "interleaved", 1.0),
    (torch.bfloat16, 64, 8, 128, 32, [100, 64, 31, 1], [37, 64, 1, 1], True,
     64, "half", 1.25),
    (torch.float16, 5, 1, 128, 32, [95, 33], [63, 2], False, 48,
     "interleaved", 1.0),
    (torch.bfloat16, 3, 3, 64, 16, [16, 17, 15, 48], [16, 2, 15, 33], True,
     0, "half", 1.0),
    (torch.float16, 7, 7, 64, 32, [300], [257], True, 16, "half", 0.5),
    (torch.bfloat16, 0, 2, 128, 16, [20, 3], [4, 3], True, 128, "half", 1.0),
    (torch.float16, 16, 2, 128, 16, [700] * 3, [333, 700, 1], False, 96,
     "half", 1.0),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[3]}-{c[4]}")
def test_append_16bit(pkv, case):
    dtype, hq, hkv, d, bs, ctx, new, norm, rot, layout, sc = case
    x = Batch(dtype, hq, hkv, d, bs, ctx, new, norm=norm, rot=rot,
              layout=layout, rope_scale=sc)
    kc = torch.randn(x.shape, generator=x.g, device="cuda").to(dtype)
    vc = torch.randn(x.shape, generator=x.g, device="cuda").to(dtype)
    q_out = torch.randn(x.q.shape, generator=x.g, device="cuda").to(dtype)
    k0, v0, q0 = kc.clone(), vc.clone(), q_out.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, lens, start = x.args()
    pkv.pa_append(q_out if hq else None, kc, vc, x.q if hq else None, x.k,
                  x.v, table, lens, start, dev_err=err, **x.kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    if hq:
        x.check_q(q_out, q0)
    want, mag = x.expected(x.k, x.k_norm)
    eps = torch.finfo(dtype).eps / 2
    got = to64(kc)
    for _, row, _, blk, o in x.places():
        tol = np.abs(want[row]) * eps + FP32 * mag[row] + \
            torch.finfo(dtype).smallest_normal * 2.0 ** -8
        assert (np.abs(got[blk, :, o] - want[row]) <= tol).all()
        assert torch.equal(vc[blk, :, o], x.v[row])
        k0[blk, :, o], v0[blk, :, o] = kc[blk, :, o], vc[blk, :, o]
    # every other slot as it was
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def random_q8(x, seed=1):
    """A pool in use: codes of every size, a scale per block and head."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in "kv":
        c = (torch.randn(x.shape, generator=g, device="cuda") * 150).clamp(
            -448, 448).to(E4M3)
        e = torch.randint(-9, -2, x.shape[:2], generator=g, device="cuda")
        out += [c, torch.exp2(e.float())]
    return out[0], out[2], out[1], out[3]


def near(a, b, rel):
    return abs(a - b) <= rel * abs(b)


def check_pool(x, name, rows, mag, before, scales0, codes, scales):
    """One of K and V after a call."""
    want, ws, written = oap.append_q8(to64(before), to64(scales0), rows,
                                      x.places())
    gs = to64(scales)
    if not np.array_equal(gs, ws):
        # fp32 may put a largest value on the other side of 448 s
        off = np.argwhere(gs != ws)
        for blk, h in off:
            new = [r for _, r, _, b, _ in x.places() if b == blk]
            top = max(np.abs(rows[r, h]).max() for r in new)
            s = min(gs[blk, h], ws[blk, h])
            assert near(top, 448 * s, 2.0 ** -18), (name, blk, h)
            want[blk, h] *= ws[blk, h] / gs[blk, h]
    got = to64(codes)
    tol = oap.e4m3_step(want) / 2
    first = {}
    for _, row, _, blk, o in x.places():
        tol[blk, :, o] += FP32 * mag[row] / gs[blk][:, None]
        first[blk] = min(first.get(blk, o), o)
    raw, raw0 = codes.view(torch.uint8), before.view(torch.uint8)
    for blk in range(got.shape[0]):
        for o in range(got.shape[2]):
            if written[blk, o] or o < first.get(blk, 0):
                assert (np.abs(got[blk, :, o] - want[blk, :, o]) <=
                        tol[blk, :, o] * (1 + 1e-9)).all(), (name, blk, o)
            else:
                assert torch.equal(raw[blk, :, o], raw0[blk, :, o])


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"{c[3]}-{c[4]}")
def test_append_q8(pkv, case):
    dtype, hq, hkv, d, bs, ctx, new, norm, rot, layout, sc = case
    x = Batch(dtype, hq, hkv, d, bs, ctx, new, norm=norm, rot=rot,
              layout=layout, rope_scale=sc)
    kc, vc, ks, vs = random_q8(x)
    k0, v0, ks0, vs0 = (t.clone() for t in (kc, vc, ks, vs))
    q_out = torch.randn(x.q.shape, generator=x.g, device="cuda").to(dtype)
    q0 = q_out.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, lens, start = x.args()
    pkv.pa_append_q8(q_out if hq else None, kc, vc, ks, vs,
                     x.q if hq else None, x.k, x.v, table, lens, start,
                     max_q_len=int(max(new)), dev_err=err, **x.kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    if hq:
        x.check_q(q_out, q0)
    check_pool(x, "k", *x.expected(x.k, x.k_norm), k0, ks0, kc, ks)
    check_pool(x, "v", to64(x.v), np.zeros_like(to64(x.v)), v0, vs0, vc, vs)


@pytest.mark.parametrize("q8", [False, True])
def test_decode_step_without_query_start(pkv, q8):
    """One row per sequence: the same bits with and without query_start, and
    in place (q_out is q)."""
    ctx = [1, 16, 17, 0, 32, 40, 200]
    x = Batch(torch.bfloat16, 16, 4, 128, 16, ctx, [1] * 7, norm=True,
              rot=128, layout="half", spare_rows=0)
    table, lens, start = x.args()
    outs = []
    for use_start in (True, False):
        if q8:
            pool = random_q8(x)
        else:
            g = torch.Generator(device="cuda").manual_seed(3)
            pool = [torch.randn(x.shape, generator=g, device="cuda").to(
                x.dtype) for _ in "kv"]
        q = x.q.clone()
        fn = pkv.pa_append_q8 if q8 else pkv.pa_append
        fn(q, *pool, q, x.k, x.v, table, lens, start if use_start else None,
           **x.kw)
        outs.append([q] + [p.view(torch.uint8) if p.dtype == E4M3 else p
                           for p in pool])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    q_out = torch.zeros_like(x.q)
    x.check_q(outs[0][0], x.q)
    assert torch.equal(outs[0][0][3], x.q[3])  # padding: left as it was
    assert q_out.sum() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(pkv, layout):
    """Positions past 2^20: an angle formed in fp32 would be off by radians.
    The pools' unused table entries stay -1."""
    n = (1 << 21) + 3
    x = Batch(torch.bfloat16, 2, 1, 64, 16, [n, 999_983], [3, 2], norm=False,
              rot=64, layout=layout, max_blocks=n // 16 + 1)
    pool = [torch.zeros(x.shape, device="cuda", dtype=x.dtype) for _ in "kv"]
    q_out = torch.zeros_like(x.q)
    table, lens, start = x.args()
    pkv.pa_append(q_out, *pool, x.q, x.k, x.v, table, lens, start, **x.kw)
    x.check_q(q_out, torch.zeros_like(q_out))


def test_scale_grows_token_by_token(pkv):
    """Fifty single-token steps whose values grow and shrink by powers of two
    over three blocks: scales and moved codes follow the oracle's state."""
    bs, d, hkv = 16, 64, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda")
    x = Batch(torch.float16, 2, hkv, d, bs, [1], [1], norm=False, rot=0,
              layout="half", spare_rows=0, pool=4)
    kc, vc, ks, vs = random_q8(x, seed=9)
    for n in range(1, 51):
        row = (torch.randn(2, 1, hkv, d, generator=g, device="cuda") *
               2.0 ** ((n * 7) % 11 - 5)).half()
        before = [t.clone() for t in (kc, vc, ks, vs)]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        pkv.pa_append_q8(None, kc, vc, ks, vs, None, row[0], row[1], table,
                         lens)
        p = n - 1
        places = [(0, 0, p, int(table[0, p // bs]), p % bs)]
        for new, c0, s0, c, s in ((row[0], before[0], before[2], kc, ks),
                                  (row[1], before[1], before[3], vc, vs)):
            want, ws, _ = oap.append_q8(to64(c0), to64(s0), to64(new), places)
            assert np.array_equal(to64(s), ws)
            blk, o = places[0][3], places[0][4]
            np.testing.assert_array_equal(
                to64(c)[blk, :, :o + 1], oap.e4m3_round(want[blk, :, :o + 1]))


def test_special_values(pkv):
    """Zeros, tiny and huge values, infinities and NaN."""
    bs, d = 16, 64
    for dtype in (torch.bfloat16, torch.float16):
        big = 3e38 if dtype == torch.bfloat16 else 65504.0
        rows = torch.zeros(6, 1, d, device="cuda", dtype=dtype)
        rows[1] = torch.finfo(dtype).smallest_normal
        rows[2] = big
        rows[2, 0, 1] = -big
        rows[3, 0, 0] = float("inf")
        rows[3, 0, 1] = 1.0
        rows[4, 0, 0] = float("nan")
        rows[4, 0, 1] = 2.0
        rows[5] = 448.0
        table = torch.arange(6, dtype=torch.int32, device="cuda")[:, None]
        table = table.contiguous()
        lens = torch.ones(6, dtype=torch.int32, device="cuda")
        kc = torch.zeros(6, 1, bs, d, device="cuda").to(E4M3)
        vc, ks = kc.clone(), torch.full((6, 1), 7.0, device="cuda")
        vs = ks.clone()
        pkv.pa_append_q8(None, kc, vc, ks, vs, None, rows, rows, table, lens)
        for c, s in ((kc, ks), (vc, vs)):
            s = s[:, 0].cpu().numpy().astype(np.float64)
            got = to64(c)[:, 0, 0] * s[:, None]
            assert s[0] == 2.0 ** -64 and (got[0] == 0).all()
            top = [oap.scale_for(float(np.nanmax(np.abs(to64(rows[i])))))
                   for i in range(6)]
            assert list(s) == top
            assert np.allclose(got[2], to64(rows[2])[0], rtol=2.0 ** -4)
            assert s[3] == 2.0 ** 120 and got[3, 0] == 448 * s[3]
            assert np.isnan(got[4, 0]) and got[4, 1] == 2.0
            assert (got[5] == 448).all() and s[5] == 1.0
            if dtype == torch.bfloat16:  # 2^-126 is below 2^-9 2^-64
                assert (got[1] == 0).all()
            else:
                assert np.allclose(got[1], to64(rows[1])[0], rtol=2.0 ** -4)


def test_order_does_not_matter(pkv):
    """The same sequences in another order give the same pool, bit for bit."""
    ctx, new = [50, 33, 90, 20, 64, 5], [50, 20, 31, 1, 64, 5]
    x = Batch(torch.bfloat16, 4, 2, 128, 32, ctx, new, norm=True, rot=128,
              layout="half", spare_rows=0)
    order = [3, 0, 5, 2, 4, 1]
    pools = []
    for perm in (range(6), order):
        perm = list(perm)
        pool = random_q8(x)
        rows = np.concatenate([np.arange(x.start[b], x.start[b + 1])
                               for b in perm])
        idx = torch.from_numpy(rows).cuda()
        start = np.concatenate([[0], np.cumsum(np.array(new)[perm])])
        pkv.pa_append_q8(
            None, *pool, None, x.k[idx], x.v[idx],
            torch.from_numpy(x.table[perm]).cuda(),
            torch.from_numpy(x.ctx[perm]).cuda(),
            torch.from_numpy(start.astype(np.int32)).cuda(),
            **{k: v for k, v in x.kw.items()})
        pools.append(pool)
    for a, b in zip(*pools):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
def test_device_errors(pkv, q8):
    """Bad lengths, ranges and block ids set dev_err; the other sequences are
    written, nothing else is touched."""
    from paged_kv_cache_383_b200 import _lib

    def run(edit, spoiled):
        x = Batch(torch.bfloat16, 4, 2, 64, 16, [20, 33, 8], [3, 5, 8],
                  norm=False, rot=64, layout="half", spare_rows=0)
        good = random_q8(x) if q8 else None
        table, lens, start = x.args()
        kw = dict(x.kw)
        edit(table, lens, start, kw)
        if q8:
            pool = good
        else:
            pool = [torch.zeros(x.shape, device="cuda", dtype=x.dtype)
                    for _ in "kv"]
        before = [p.clone() for p in pool]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.zeros_like(x.q)
        (pkv.pa_append_q8 if q8 else pkv.pa_append)(
            q_out, *pool, x.q, x.k, x.v, table, lens, start, dev_err=err,
            **kw)
        torch.cuda.synchronize()
        assert err.item() == _lib.PA_ERR_DEVICE_OOB
        for b in range(3):
            r0, r1 = int(x.start[b]), int(x.start[b + 1])
            blk = int(x.table[b, (x.ctx[b] - 1) // 16])
            same = torch.equal(pool[0][blk].view(torch.uint8),
                               before[0][blk].view(torch.uint8))
            assert same == (b in spoiled), b
            if b not in spoiled:
                assert q_out[r0:r1].abs().sum() > 0

    def long_ctx(table, lens, start, kw):
        lens[1] = table.shape[1] * 16 + 1

    def negative(table, lens, start, kw):
        lens[2] = -1

    def short_ctx(table, lens, start, kw):
        lens[0] = 2  # three new tokens

    def few(table, lens, start, kw):
        kw["max_q_len"] = 5  # the last one has 8

    def bad_block(table, lens, start, kw):
        table[1, 2] = 10_000
        table[1, 1] = -7

    run(long_ctx, {1})
    run(negative, {2})
    run(short_ctx, {0})
    run(few, {2})
    run(bad_block, {1})


@pytest.mark.parametrize("q8", [False, True])
def test_device_errors_without_rows(pkv, q8):
    """A sequence whose range holds no row of the call, but is no valid empty
    one, sets dev_err all the same; padding (length 0) never does."""
    from paged_kv_cache_383_b200 import _lib

    def run(lens_at, start, flagged):
        x = Batch(torch.float16, 4, 2, 64, 16, [20, 33, 8], [3, 5, 8],
                  norm=False, rot=64, layout="half", spare_rows=0)
        pool = random_q8(x) if q8 else [
            torch.zeros(x.shape, device="cuda", dtype=x.dtype) for _ in "kv"]
        table, lens, _ = x.args()
        for i, n in lens_at.items():
            lens[i] = n
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.zeros_like(x.q)
        (pkv.pa_append_q8 if q8 else pkv.pa_append)(
            q_out, *pool, x.q, x.k, x.v, table, lens,
            torch.tensor(start, dtype=torch.int32, device="cuda"),
            dev_err=err, **x.kw)
        torch.cuda.synchronize()
        assert err.item() == (_lib.PA_ERR_DEVICE_OOB if flagged else 0)
        assert q_out[:3].abs().sum() > 0

    run({}, [0, 3, 3, 3], False)
    run({}, [0, 3, 2, 2], True)             # ends before it starts
    run({}, [0, 3, 16, 20], True)           # past the rows
    run({1: -4}, [0, 3, 3, 3], True)        # no rows, a bad length
    run({2: 49}, [0, 3, 3, 3], True)        # the table has 48 tokens
    run({1: 0, 2: 0}, [0, 3, 3, 40], False)  # padding


@pytest.mark.parametrize("q8", [False, True])
def test_queries_in_place(pkv, q8):
    """q_out is q itself, a slice of the projection."""
    x = Batch(torch.bfloat16, 8, 2, 128, 16, [40, 0, 17], [5, 2, 17],
              norm=True, rot=128, layout="interleaved")
    fn = pkv.pa_append_q8 if q8 else pkv.pa_append
    outs = []
    for in_place in (False, True):
        pool = random_q8(x) if q8 else [
            torch.zeros(x.shape, device="cuda", dtype=x.dtype) for _ in "kv"]
        q_out = x.q if in_place else x.q.clone()
        fn(q_out, *pool, x.q, x.k, x.v, *x.args(), **x.kw)
        torch.cuda.synchronize()
        outs.append([q_out.contiguous()] + [p.clone() for p in pool])
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
def test_keys_and_values_only(pkv, q8):
    """No query heads: the cache gets what a call with them writes."""
    x = Batch(torch.float16, 4, 3, 64, 32, [70, 33], [40, 33], norm=True,
              rot=32, layout="half")
    fn = pkv.pa_append_q8 if q8 else pkv.pa_append
    pools = []
    for with_q in (True, False):
        pool = random_q8(x) if q8 else [
            torch.zeros(x.shape, device="cuda", dtype=x.dtype) for _ in "kv"]
        q, q_out = (x.q, torch.empty_like(x.q)) if with_q else (None, None)
        fn(q_out, *pool, q, x.k, x.v, *x.args(), **x.kw)
        torch.cuda.synchronize()
        pools.append(pool)
    for a, b in zip(*pools):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
def test_graph_and_stream(pkv, q8):
    """Captured and replayed with other lengths and values, on a stream of
    its own, equals eager calls."""
    x = Batch(torch.float16, 8, 2, 64, 16, [10, 40, 77], [1, 1, 1], norm=True,
              rot=32, layout="interleaved", spare_rows=0, pool=20)
    table = torch.arange(18, dtype=torch.int32, device="cuda").view(3, 6)
    lens = torch.tensor([10, 40, 77], dtype=torch.int32, device="cuda")
    pool_a = random_q8(x) if q8 else [
        torch.zeros(x.shape, device="cuda", dtype=x.dtype) for _ in "kv"]
    pool_b = [p.clone() for p in pool_a]
    fn = pkv.pa_append_q8 if q8 else pkv.pa_append
    k, v, q = x.k.clone(), x.v.clone(), x.q.clone()
    out_a, out_b = torch.zeros_like(q), torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    warm = [p.clone() for p in pool_a]
    fn(out_b, *warm, q, k, v, table, lens, stream=s, **x.kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(out_a, *pool_a, q, k, v, table, lens, **x.kw)
    for step in range(4):
        graph.replay()
        fn(out_b, *pool_b, q, k, v, table, lens, **x.kw)
        torch.cuda.synchronize()
        assert torch.equal(out_a, out_b)
        for a, b in zip(pool_a, pool_b):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        lens += 1
        k.copy_(torch.randn_like(k) * 2 ** step)
        v.copy_(torch.randn_like(v) * 3 ** step)


def test_offsets_past_4_gib(pkv):
    """Blocks whose codes lie past 2^32 bytes of the pool."""
    nb, hkv, bs, d = 270_000, 8, 16, 128
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device="cuda").view(
        E4M3)
    vc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device="cuda").view(
        E4M3)
    ks = torch.zeros(nb, hkv, device="cuda")
    vs = torch.zeros(nb, hkv, device="cuda")
    rows = torch.randn(2, hkv, d, device="cuda").bfloat16()
    table = torch.tensor([[nb - 1], [262_145]], dtype=torch.int32,
                         device="cuda")
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    pkv.pa_append_q8(None, kc, vc, ks, vs, None, rows, rows, table, lens)
    for i, blk in enumerate(table[:, 0].tolist()):
        got = to64(kc[blk, :, 0]) * to64(ks[blk])[:, None]
        ref = to64(rows[i])
        assert np.allclose(got, ref, rtol=2.0 ** -4, atol=2.0 ** -10)
        assert torch.equal(vc[blk].view(torch.uint8),
                           kc[blk].view(torch.uint8))
    assert int((ks != 0).sum()) == 2 * hkv


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bound", [0, 1, 9])
def test_without_query_start_the_bound_does_not_matter(pkv, q8, bound):
    """Through the C ABI, which the binding gives a bound of 1."""
    from paged_kv_cache_383_b200 import _lib
    lib = _lib.load()
    fn = lib.pa_append_q8 if q8 else lib.pa_append
    n, hkv, d, bs = 5, 2, 64, 16
    rows = torch.randn(n, hkv, d, device="cuda").half()
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    table = table.contiguous()
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    pool = [torch.zeros(n, hkv, bs, d, device="cuda").to(
        E4M3 if q8 else torch.float16) for _ in "kv"]
    if q8:
        pool += [torch.zeros(n, hkv, device="cuda") for _ in "kv"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = _lib.pa_append_desc(n, 0, hkv, d, bs, 1, n, _lib.PA_F16, n, bound,
                               0, 0, 1.0, 1e-6, 0, hkv * d, hkv * d, 0)
    st = fn(None, *[p.data_ptr() for p in pool], None, rows.data_ptr(),
            rows.data_ptr(), None, None, None, table.data_ptr(),
            lens.data_ptr(), None, ctypes.byref(desc), err.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and err.item() == 0
    for p in pool[:2]:
        assert (p[:, :, 0].float() != 0).any(-1).all()
