"""Appends of so many rows that a CTA streams several tokens and looks after a
window of several rows (from four rows per SM on), against the fp64 oracle;
tolerances as in test_gpu_append."""
import numpy as np
import pytest
import torch

from test_gpu_append import E4M3, FP32, Batch, check_pool, random_q8, to64

pytestmark = pytest.mark.gpu

# rows (at least; sequences of 1 to 40 new rows fill them up)
LARGE = [
    # dtype, hq, hkv, d, bs, rows, norm, rot, layout
    (torch.bfloat16, 5, 8, 64, 16, 1300, True, 64, "half"),
    (torch.float16, 2, 8, 128, 32, 2403, False, 96, "interleaved"),
    (torch.bfloat16, 1, 8, 64, 32, 5003, False, 32, "half"),
    (torch.float16, 3, 1, 128, 16, 2401, True, 128, "half"),
]


def batch(case):
    dtype, hq, hkv, d, bs, rows, norm, rot, layout = case
    rng = np.random.default_rng(rows)
    ctx, new = [], []
    while sum(new) < rows:
        n = int(rng.integers(1, 41))
        kind = len(new) % 7
        # a decode row now and then, an empty sequence, one that ends at, one
        # that starts at a block's edge
        new.append(1 if kind == 1 else 0 if kind == 2 else n)
        old = int(rng.integers(0, 50))
        if kind == 3:
            old = -n % bs
        if kind == 4:
            old = bs * (old // bs)
        ctx.append(old + new[-1])
    ctx.append(0)
    new.append(7)  # padding
    return Batch(dtype, hq, hkv, d, bs, ctx, new, norm=norm, rot=rot,
                 layout=layout, seed=rows, spare_rows=3)


@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{c[3]}-{c[4]}-{c[5]}")
@pytest.mark.parametrize("q8", [False, True])
def test_many_rows(pkv, case, q8):
    x = batch(case)
    dtype = x.dtype
    pool = random_q8(x) if q8 else [
        torch.randn(x.shape, generator=x.g, device="cuda").to(dtype)
        for _ in "kv"]
    before = [p.clone() for p in pool]
    q_out = torch.randn(x.q.shape, generator=x.g, device="cuda").to(dtype)
    q0 = q_out.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    (pkv.pa_append_q8 if q8 else pkv.pa_append)(
        q_out, *pool, x.q, x.k, x.v, *x.args(), max_q_len=40, dev_err=err,
        **x.kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    x.check_q(q_out, q0)
    want, mag = x.expected(x.k, x.k_norm)
    if q8:
        check_pool(x, "k", want, mag, before[0], before[2], pool[0], pool[2])
        check_pool(x, "v", to64(x.v), np.zeros_like(to64(x.v)), before[1],
                   before[3], pool[1], pool[3])
        return
    rows, blks, offs = (np.array(c) for c in zip(
        *[(row, blk, o) for _, row, _, blk, o in x.places()]))
    got = to64(pool[0])[blks, :, offs]
    tol = np.abs(want[rows]) * torch.finfo(dtype).eps / 2 + \
        FP32 * mag[rows] + torch.finfo(dtype).smallest_normal * 2.0 ** -8
    assert (np.abs(got - want[rows]) <= tol).all()
    at = [torch.from_numpy(c).cuda() for c in (blks, offs)]
    assert torch.equal(pool[1][at[0], :, at[1]],
                       x.v[torch.from_numpy(rows).cuda()])
    for p, p0 in zip(pool, before):  # every other slot as it was
        p0[at[0], :, at[1]] = p[at[0], :, at[1]]
        assert torch.equal(p, p0)


def test_many_rows_equal_few(pkv):
    """One call of many sequences writes what calls of a few at a time write,
    bit for bit."""
    x = batch(LARGE[1])
    table, lens, start = x.args()
    n = len(x.ctx)
    for q8 in (False, True):
        fn = pkv.pa_append_q8 if q8 else pkv.pa_append
        results = []
        for step in (n, 9):
            pool = random_q8(x) if q8 else [
                torch.zeros(x.shape, device="cuda", dtype=x.dtype)
                for _ in "kv"]
            q_out = torch.zeros_like(x.q)
            for b in range(0, n, step):
                e = min(b + step, n)
                r = slice(int(x.start[b]), int(x.start[e]))
                if r.start == r.stop:
                    continue
                fn(q_out[r], *pool, x.q[r], x.k[r], x.v[r], table[b:e],
                   lens[b:e], start[b:e + 1] - start[b], **x.kw)
            results.append([q_out] + [p.view(torch.uint8) if p.dtype == E4M3
                                      else p for p in pool])
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_more_overlapping_sequences_than_a_window_holds(pkv):
    """Twenty sequences that all claim the same 16 rows (every second range
    runs backwards): flagged, and no slot outside their blocks is touched."""
    from paged_kv_cache_383_b200 import _lib
    hkv, d, bs, rows = 8, 64, 16, 1300
    n = 40
    start = torch.tensor([0, 16] * (n // 2) + [0], dtype=torch.int32,
                         device="cuda")
    lens = torch.full((n,), 16, dtype=torch.int32, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    table = table.contiguous()
    x = torch.randn(rows, hkv, d, device="cuda").bfloat16()
    for q8 in (False, True):
        pool = [torch.zeros(n + 2, hkv, bs, d, device="cuda").to(
            E4M3 if q8 else torch.bfloat16) for _ in "kv"]
        if q8:
            pool += [torch.zeros(n + 2, hkv, device="cuda") for _ in "kv"]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        (pkv.pa_append_q8 if q8 else pkv.pa_append)(
            None, *pool, None, x, x, table, lens, start, max_q_len=16,
            dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == _lib.PA_ERR_DEVICE_OOB
        for p in pool[:2]:
            p = p.float()
            assert (p[1::2] == 0).all() and (p[n:] == 0).all()
