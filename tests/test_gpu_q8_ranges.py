"""The 8-bit cache at the ends of its scales' range, and NaN in its parts."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import (BF, E4M3, HF, Pool, bound_prefill, decode, positions,
                         prefill, reference, to64)

pytestmark = pytest.mark.gpu


def both(pkv, pool, q, start, scale, max_q_len):
    """float32 outputs of the prefill, and of the decode of each sequence's
    last row, with the fp64 reference and the error allowed to each element
    (bound_prefill's terms cover the decode: its weights are fp16 too, kept
    relative to the largest v scale)."""
    new = np.diff(start)
    pos = positions(pool.ctx.tolist(), new.tolist())
    ref, mag = reference(pool, q, pos, scale)
    tol = bound_prefill(pool, q, pos, scale, mag)
    last = torch.from_numpy(np.asarray(start[1:]) - 1).cuda()
    p32, p16 = prefill(pkv, pool, q, start, scale, max_q_len)
    d32, d16 = decode(pkv, pool, q[last].contiguous(), scale)
    assert torch.equal(p16, p32.to(q.dtype))
    assert torch.equal(d16, d32.to(q.dtype))
    last = last.cpu().numpy()
    return (p32, ref, tol), (d32, ref[last], tol[last])


@pytest.mark.parametrize("exp", [120, 113, 104, 101, 60, -60, -64, -90])
@pytest.mark.parametrize("mixed", [False, True])
def test_scales_of_any_size(pkv, exp, mixed):
    """V scales around 2^exp (one of 2^120 is what an append of the largest
    bf16 values writes), with and without much smaller ones beside them, the
    small ones first.  Codes are small enough that sums fit float32."""
    ctx, new = [1, 40, 100, 70], [1, 30, 2, 70]
    pool = Pool(2, 128, 16, ctx, seed=5)
    codes = pool.vc.float()
    pool.vc.copy_((codes / 448 if exp > 110 else codes).to(E4M3))
    ok = ~torch.isnan(pool.vs)
    e = torch.full_like(pool.vs, float(exp))
    if mixed:
        for row in pool.table:
            for i, blk in enumerate(row[row >= 0]):
                e[int(blk)] = exp - 30 + 10 * i if i < 3 else exp - i % 2
    pool.vs.copy_(torch.where(ok, torch.exp2(e.clamp_(-100, 120)), pool.vs))
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(sum(new), 8, 128, generator=g, device="cuda").to(BF)
    start = np.concatenate([[0], np.cumsum(new)])
    for out, ref, tol in both(pkv, pool, q, start, 0.09, 70):
        assert (np.abs(to64(out) - ref) <= tol).all(), \
            float((np.abs(to64(out) - ref) / tol).max())


def test_large_values_come_back(pkv):
    """bf16 values up to the largest whose code still stands for a float32,
    appended and attended to: a context of one token returns what the code
    stands for."""
    rows = torch.randn(7, 2, 64, device="cuda") * 2.0 ** torch.tensor(
        [0., 60., 100., 110., 115., 120., 125.], device="cuda")[:, None, None]
    rows = rows.to(BF)
    rows[6, :, :2] = torch.tensor([3.2e38, -3.2e38], device="cuda").to(BF)
    table = torch.arange(7, dtype=torch.int32, device="cuda")[:, None]
    table = table.contiguous()
    lens = torch.ones(7, dtype=torch.int32, device="cuda")
    z = torch.zeros(7, 2, 16, 64, device="cuda").to(E4M3)
    cache = [z, z.clone()] + [torch.zeros(7, 2, device="cuda") for _ in "kv"]
    keys = torch.randn(7, 2, 64, device="cuda").to(BF)
    pkv.pa_append_q8(None, *cache, None, keys, rows, table, lens)
    assert float(cache[3].max()) == 2.0 ** 120
    want = to64(cache[1])[:, :, 0] * to64(cache[3])[:, :, None]
    assert (np.abs(want - to64(rows)) <= np.abs(to64(rows)) * 2.0 ** -4 +
            to64(cache[3])[:, :, None] * 2.0 ** -10).all()
    q = torch.randn(7, 4, 64, device="cuda").to(BF)
    start = torch.arange(8, dtype=torch.int32, device="cuda")
    outs = [torch.empty(7, 4, 64, device="cuda") for _ in "12"]
    pkv.pa_decode_q8(outs[0], q, *cache, table, lens, 0.125)
    pkv.pa_prefill_q8(outs[1], q, *cache, table, lens, start, 0.125,
                      max_q_len=1)
    # one weight, 1, which fp16 holds: what is left is the exponential's
    # argument in fp32, 2^-15 of the sum that divides
    for out in outs:
        got = to64(out).reshape(7, 2, 2, 64)
        assert (np.abs(got - want[:, :, None]) <=
                2.0 ** -15 * np.abs(want[:, :, None])).all()


def test_zero_scales_give_zeros(pkv):
    """Blocks of scale 0 count as zeros whatever their codes, alone or beside
    blocks of the smallest scales."""
    ctx, new = [33, 48, 130], [33, 1, 4]
    for tiny in (False, True):
        pool = Pool(2, 64, 16, ctx, seed=7)
        for b, row in enumerate(pool.table):
            for i, blk in enumerate(row[row >= 0]):
                pool.vs[int(blk)] = 2.0 ** -100 if tiny and i % 2 else 0.0
        q = torch.randn(sum(new), 8, 64, device="cuda").to(HF)
        start = np.concatenate([[0], np.cumsum(new)])
        for out, ref, tol in both(pkv, pool, q, start, 0.125, 33):
            if tiny:  # values of 2^-91 and less: the bound's own floor aside
                assert (np.abs(to64(out) - ref) <= tol - 1e-30 + 1e-38).all()
            else:
                assert (out == 0).all()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("new", [70, 4])
def test_nan_scale_reaches_the_rows_that_see_its_block(pkv, which, new):
    """The scale of positions 304 .. 319 of the first context."""
    ctx = [330, 330]
    pool = Pool(2, 128, 16, ctx, seed=3)
    blk, first = int(pool.table[0, 19]), 304
    (pool.ks if which == "k" else pool.vs)[blk, 1] = float("nan")
    q = torch.randn(2 * new, 8, 128, device="cuda").to(HF)
    start = [0, new, 2 * new]
    out, _ = prefill(pkv, pool, q, start, 0.09, new)
    pos = torch.arange(330 - new, 330, device="cuda")
    hit = torch.zeros(2 * new, 8, dtype=torch.bool, device="cuda")
    hit[:new, 4:] = (pos >= first)[:, None]
    assert torch.equal(torch.isnan(out), hit[..., None].expand_as(out))
    last, _ = decode(pkv, pool, q[[new - 1, 2 * new - 1]].contiguous(), 0.09)
    assert torch.isnan(last[0, 4:]).all()
    assert torch.isfinite(last[0, :4]).all() and torch.isfinite(last[1]).all()


@pytest.mark.parametrize("group,new,bs", [
    (1, 150, 16), (8, 150, 32), (4, 70, 16), (8, 8, 16), (1, 1, 32)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_values_reach_the_rows_that_see_them(pkv, group, new, bs, d):
    """NaN V codes of new and of old tokens: each makes its dim NaN in the
    rows from its position on, whichever tile they are computed in, and
    changes nothing else."""
    ctx = [330, 200, 330]
    new = [new, min(new, 200), new]
    pool = Pool(2, d, bs, ctx, seed=3)
    g = torch.Generator(device="cuda").manual_seed(group)
    q = torch.randn(sum(new), 2 * group, d, generator=g, device="cuda").to(BF)
    start = np.concatenate([[0], np.cumsum(new)])
    clean, _ = prefill(pkv, pool, q, start, 0.09, max(new))
    bad = np.full((3, 2, d), 1 << 30)   # first NaN key by dim
    raw = pool.vc.view(torch.uint8)
    keys = {0: (0, 63, 64, 181, 200, 250, 255, 256, 300, 329, 329),
            2: (5, 187, 191, 192, 319, 320, 321, 328)}
    for b, at in keys.items():
        for i, p in enumerate(at):
            if p < ctx[b] - new[b] and i % 3:
                continue                # a few old tokens only
            h, e = i % 2, (7 * i + 3 * b) % d
            raw[int(pool.table[b, p // bs]), h, p % bs, e] = 0x7f + 0x80 * (
                i & 1)
            bad[b, h, e] = min(bad[b, h, e], p)
    out, out16 = prefill(pkv, pool, q, start, 0.09, max(new))
    pos = np.array(positions(ctx, new))
    want = np.repeat(bad[pos[:, 0]] <= pos[:, 1][:, None, None], group,
                     axis=1)
    assert want.any() and not want.all()
    got = to64(out)
    np.testing.assert_array_equal(np.isnan(got), want)
    assert torch.equal(torch.isnan(out16), torch.isnan(out))
    np.testing.assert_array_equal(got[~want], to64(clean)[~want])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_v_scales_over_60_binades(pkv, dtype):
    """Block by block, zeros among them, with large, tiny and zero queries and
    peaked scores: within the documented 2^-33 of the largest scale, and the
    16-bit output is the float32 one's rounding, infinities included."""
    ctx, new = [300, 77], [5, 77]
    pool = Pool(2, 128, 16, ctx, seed=8)
    e = torch.arange(pool.n, device="cuda") * 37 % 61 - 30
    ok = ~torch.isnan(pool.vs)
    pool.vs.copy_(torch.where(
        ok, torch.exp2(e.float())[:, None].expand(pool.n, 2), pool.vs))
    for c, s, b in ((pool.vc, pool.vs, pool.table[0, 3]),
                    (pool.vc, pool.vs, pool.table[1, 0]),
                    (pool.kc, pool.ks, pool.table[0, 5])):
        c[int(b)] = torch.zeros_like(c[int(b)].float()).to(E4M3)
        s[int(b)] = 0.0
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(82, 16, 128, generator=g, device="cuda")
    q[:, 3] *= 50
    q[:, 4] *= 2.0 ** -13
    q[:, 5] = 0
    q[:, 6, 7] = 300  # one large element among small ones
    q = q.to(dtype)
    for out, ref, tol in both(pkv, pool, q, [0, 5, 82], 0.05, 77):
        # 300 / 50 times larger scores: arguments to 2^10, so 2^-13 on a
        # weight, and as much on their sum
        _, mag = reference(pool, q, positions(ctx, new), 0.05)
        mag = mag[[4, 81]] if len(ref) == 2 else mag
        assert (np.abs(to64(out) - ref) <= tol + 2.0 ** -12 * mag).all()


@pytest.mark.parametrize("few", [False, True])
def test_nan_values_among_many_items(pkv, few):
    """Several dozen work items per CTA, NaN V codes in a few of the sequences:
    where one is found is forgotten with its item."""
    rng = np.random.default_rng(7)
    n, hkv, d, bs = 900, 8, 64, 16
    ctx = rng.integers(1, 90, n)
    new = np.minimum(rng.integers(0, 5 if few else 90, n), ctx)
    if few:   # a batch that shares keys between the query tiles
        ctx[::50] += 400
    pool = Pool(hkv, d, bs, ctx.tolist(), seed=12)
    start = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(int(start[-1]), hkv, d, device="cuda").to(BF)
    clean, _ = prefill(pkv, pool, q, start, 0.125, int(new.max()))
    bad = np.full((n, hkv, d), 1 << 30)
    raw = pool.vc.view(torch.uint8)
    for b in rng.choice(n, 90, replace=False):
        p, h, e = (int(rng.integers(0, m)) for m in (ctx[b], hkv, d))
        raw[int(pool.table[b, p // bs]), h, p % bs, e] = 0xff
        bad[b, h, e] = p
    out, _ = prefill(pkv, pool, q, start, 0.125, int(new.max()))
    pos = np.array(positions(ctx.tolist(), new.tolist()))
    want = bad[pos[:, 0]] <= pos[:, 1][:, None, None]
    assert want.any()
    got = to64(out)
    np.testing.assert_array_equal(np.isnan(got), want)
    np.testing.assert_array_equal(got[~want], to64(clean)[~want])
