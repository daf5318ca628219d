"""The rotating append, both attentions and the block moves over one 8-bit
pool, the way a serving loop drives them:

1. two prompts of unlike length are appended (norm and rotation) and
   prefilled in one call each;
2. decode steps for both;
3. a fork shares the first sequence's blocks; its next token copies the
   partly filled one;
4. the second verifies four draft tokens in one pass and keeps two, and goes
   on from there;
5. the first is swapped to pinned host memory and back, and decodes again.

Every attention output is checked against fp64 attention over the values that
the pool holds, and the pool against the keys and values themselves, tracked
on the host: a code is off by at most two roundings to e4m3 (its own, and one
if its block's scale grew later): 2 * 2^-4 of the value, and 2 * 2^-10 of the
scale below e4m3's normal range."""
import numpy as np
import pytest
import torch

from oracle import append as oap
from oracle import attention as oa

pytestmark = pytest.mark.gpu
HQ, HKV, D, BS, NB = 16, 4, 128, 16, 48
SCALE, EPS = D ** -0.5, 1e-6
E4M3 = torch.float8_e4m3fn


def to64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Loop:
    def __init__(self, pkv):
        self.pkv = pkv
        self.g = torch.Generator(device="cuda").manual_seed(12)
        self.bm = pkv.BlockManager(NB, BS)
        self.bm.set_host_blocks(NB)
        z = torch.full((NB, HKV, BS, D), float("nan"), device="cuda")
        self.cache = [z.to(E4M3), z.to(E4M3),
                      torch.full((NB, HKV), float("nan"), device="cuda"),
                      torch.full((NB, HKV), float("nan"), device="cuda")]
        self.freqs, sc = pkv.pa_rope_freqs(
            D, 10000.0, scaling="wavelength", factor=8.0, original_len=64)
        assert sc == 1.0
        self.fd = self.freqs.cuda()
        self.w = [(1 + 0.1 * self.rnd(D).float()).bfloat16() for _ in "qk"]
        self.K, self.V = {}, {}
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rnd(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").bfloat16()

    def step(self, seqs, new):
        """Append ``new[i]`` tokens to ``seqs[i]`` and attend; returns q_out
        and the outputs, rows in order."""
        pkv = self.pkv
        _, pairs = self.bm.append_batch(seqs, new)
        if len(pairs):
            pkv.pa_copy_blocks_q8(*self.cache, torch.from_numpy(pairs).cuda(),
                                  dev_err=self.err)
        table, lens = (torch.from_numpy(x).cuda()
                       for x in self.bm.block_table(seqs, 16))
        n = sum(new)
        qkv = self.rnd(n, HQ + 2 * HKV, D) * (0.5 + torch.rand(
            n, 1, 1, generator=self.g, device="cuda")).bfloat16()
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        one = all(m == 1 for m in new)
        start = None if one else torch.tensor(
            np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32,
            device="cuda")
        raw = to64(k), to64(v), to64(q)
        q_out = torch.empty(n, HQ, D, dtype=torch.bfloat16, device="cuda")
        pkv.pa_append_q8(q_out, *self.cache, q, k, v, table, lens, start,
                         max_q_len=max(new), q_norm=self.w[0],
                         k_norm=self.w[1], norm_eps=EPS, rope_freqs=self.fd,
                         dev_err=self.err)
        out = torch.empty(n, HQ, D, device="cuda")
        if one:
            pkv.pa_decode_q8(out, q_out, *self.cache, table, lens, SCALE,
                             dev_err=self.err)
        else:
            pkv.pa_prefill_q8(out, q_out, *self.cache, table, lens, start,
                              SCALE, max_q_len=max(new), dev_err=self.err)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        f = self.freqs.numpy()
        row = 0
        for s, m in zip(seqs, new):
            have = self.K.setdefault(s, []), self.V.setdefault(s, [])
            for i in range(row, row + m):
                p = len(have[0])
                have[0].append(oap.rotate_head(
                    oap.norm_head(raw[0][i], to64(self.w[1]), EPS), p, f,
                    "half", 1.0))
                have[1].append(raw[1][i])
                want = oap.rotate_head(
                    oap.norm_head(raw[2][i], to64(self.w[0]), EPS), p, f,
                    "half", 1.0)
                assert np.allclose(to64(q_out[i]), want, rtol=2.0 ** -8,
                                   atol=2.0 ** -16)
            row += m
        self.check(seqs, new, q_out, out)

    def held(self, s):
        """The values the pool holds for sequence s, [len, HKV, D]."""
        ids = torch.from_numpy(self.bm.seq_blocks(s).astype(np.int64)).cuda()
        n = self.bm.seq_len(s)
        res = []
        for c, sc in ((self.cache[0], self.cache[2]),
                      (self.cache[1], self.cache[3])):
            val = to64(c.view(torch.uint8)[ids].view(E4M3)) * \
                to64(sc[ids])[:, :, None, None]
            res.append(val.transpose(0, 2, 1, 3).reshape(-1, HKV, D)[:n])
            scale = np.repeat(to64(sc[ids]), BS, 0)[:n]
            res.append(scale[:, :, None])
        return res

    def check(self, seqs, new, q, out):
        row = 0
        for s, m in zip(seqs, new):
            k, ks, v, vs = self.held(s)
            for got, sc, want in ((k, ks, np.array(self.K[s])),
                                  (v, vs, np.array(self.V[s]))):
                tol = 2 * (np.abs(want) * 2.0 ** -4 + sc * 2.0 ** -10) \
                    + 2.0 ** -18
                assert (np.abs(got - want) <= tol).all(), s
            for i in range(m):
                n = len(k) - m + i + 1
                for h in range(HQ):
                    g = h // (HQ // HKV)
                    args = to64(q[row + i, h]), k[:n, g]
                    ref = oa.attend(*args, v[:n, g], SCALE)
                    mag = oa.attend(*args, np.abs(v[:n, g]), SCALE)
                    # the weights' fp16 rounding, and scores in fp32
                    assert (np.abs(to64(out[row + i, h]) - ref) <=
                            (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -20
                            ).all()
            row += m


def test_serving_flow(pkv):
    x = Loop(pkv)
    for s in (0, 1):
        x.bm.add_seq(s)
    x.step([0, 1], [75, 130])
    for _ in range(3):
        x.step([0, 1], [1, 1])
    x.bm.fork(0, 2)
    x.K[2], x.V[2] = list(x.K[0]), list(x.V[0])
    before = x.bm.seq_blocks(0).copy()
    x.step([2, 0], [1, 1])
    assert (x.bm.seq_blocks(0)[:4] == before[:4]).all()
    assert x.bm.seq_blocks(0)[4] != x.bm.seq_blocks(2)[4]
    # four draft tokens of sequence 1, two kept, then on from there
    n = x.bm.seq_len(1)
    x.step([1], [4])
    x.bm.truncate(1, n + 2)
    x.K[1], x.V[1] = x.K[1][:n + 2], x.V[1][:n + 2]
    x.step([1, 2], [1, 1])
    # out to pinned host memory; the freed blocks are taken by another prompt
    host = [torch.zeros((NB,) + t.shape[1:], dtype=torch.uint8 if
                        t.dtype == E4M3 else t.dtype).pin_memory()
            for t in x.cache]
    host = [h.view(E4M3) if h.dtype == torch.uint8 else h for h in host]
    pairs = x.bm.swap_out([1])
    pkv.pa_swap_blocks_q8(*host, *x.cache, torch.from_numpy(pairs).cuda(),
                          dev_err=x.err)
    x.bm.add_seq(3)
    x.step([3], [200])
    pairs = x.bm.swap_in([1])
    pkv.pa_swap_blocks_q8(*x.cache, *host, torch.from_numpy(pairs).cuda(),
                          dev_err=x.err)
    x.step([1, 3, 0], [1, 1, 1])
    # a chunk that starts inside a block, beside a decode token
    x.step([1, 2], [37, 1])
