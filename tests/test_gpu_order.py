"""Calls queued one behind the other on a stream give what the same calls give
with a synchronisation after each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("q8", [False, True])
def test_decode_then_append_of_the_next_step(pkv, q8):
    """A table so wide that the decode may have 32 partitions (its separate
    reduce runs) and contexts of one partition each (which leave the reduce
    nothing to do); the append behind it overwrites the queries that the
    decode reads, moves the scales of the blocks it reads and writes into
    them."""
    hq, hkv, d, bs, n, steps = 64, 8, 128, 16, 4, 8
    width = 131072 // bs
    g = torch.Generator(device="cuda").manual_seed(1)
    # the last block of each context holds 3 tokens before the first step
    first = [4000 - 13 - 64 * b for b in range(n)]
    used = [-(-(c + steps) // bs) for c in first]
    nb = sum(used)
    table = torch.full((n, width), -1, dtype=torch.int32)
    ids, at = torch.randperm(nb, generator=torch.Generator().manual_seed(2)), 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    table = table.cuda()
    lens = [torch.tensor([c + 1 + i for c in first], dtype=torch.int32,
                         device="cuda") for i in range(steps)]
    shape = (nb, hkv, bs, d)
    dt = torch.bfloat16
    pool0 = [torch.randn(shape, generator=g, device="cuda").to(
        E4M3 if q8 else dt) for _ in "kv"]
    if q8:
        pool0 += [torch.full((nb, hkv), 2.0 ** -6, device="cuda")
                  for _ in "kv"]
    rows = [(torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda") *
             2.0 ** i).to(dt) for i in range(steps)]
    append = pkv.pa_append_q8 if q8 else pkv.pa_append
    decode = pkv.pa_decode_q8 if q8 else pkv.pa_decode
    assert pkv.pa_decode_partition_size(
        pkv.make_desc(rows[0][:, :hq], pool0[0], table)) == 4096

    def run(sync):
        pool = [p.clone() for p in pool0]
        q = torch.empty(n, hq, d, dtype=dt, device="cuda")
        outs = [torch.empty(n, hq, d, dtype=dt, device="cuda")
                for _ in range(steps)]
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        if not sync:
            torch.cuda._sleep(4_000_000)  # the calls below are queued behind
        for x, length, out in zip(rows, lens, outs):
            append(q, *pool, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:],
                   table, length, dev_err=err)
            if sync:
                torch.cuda.synchronize()
            decode(out, q, *pool, table, length, d ** -0.5, workspace=ws,
                   dev_err=err)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert err.item() == 0
        return outs + [p.view(torch.uint8) for p in pool] + [q]

    want = run(True)
    assert torch.isfinite(torch.stack(want[:steps]).float()).all()
    for _ in range(10):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_calls_on_two_streams_without_a_workspace(pkv, q8, handle):
    """A long call on the current stream and, without any wait between them, a
    call on a stream of its own: neither is given a workspace, so each must
    have memory of its own."""
    hq, hkv, d, bs = 32, 8, 128, 16
    torch.manual_seed(3)
    sets = []
    for lens in ([30_000, 9_000, 500, 20_000], [700, 25_000, 16_000, 3]):
        used = [-(-n // bs) for n in lens]
        nb = sum(used)
        table = torch.zeros(4, max(used), dtype=torch.int32)
        ids, at = torch.randperm(nb), 0
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u]
            at += u
        pool = [torch.randn(nb, hkv, bs, d, device="cuda").to(
            E4M3 if q8 else torch.bfloat16) for _ in "kv"]
        if q8:
            pool += [torch.rand(nb, hkv, device="cuda") + 0.5 for _ in "kv"]
        q = torch.randn(40, hq, d, device="cuda").bfloat16()
        sets.append((q, pool, table.cuda(),
                     torch.tensor(lens, dtype=torch.int32, device="cuda")))
    start = torch.tensor([0, 20, 30, 39, 40], dtype=torch.int32,
                         device="cuda")

    def call(out, x, kind, stream):
        q, pool, table, lens = x
        if kind == "decode":
            fn = pkv.pa_decode_q8 if q8 else pkv.pa_decode
            fn(out, q[:4], *pool, table, lens, 0.09, partition_size=64,
               stream=stream)
        else:
            fn = pkv.pa_prefill_q8 if q8 else pkv.pa_prefill
            fn(out, q, *pool, table, lens, start, 0.09, max_q_len=20,
               stream=stream)

    def outs(kind, n):
        return [torch.empty(4 if kind == "decode" else 40, hq, d,
                            dtype=torch.bfloat16, device="cuda")
                for _ in range(n)]

    want = {}
    for kind in ("decode", "prefill"):
        want[kind] = outs(kind, 2)
        for out, x in zip(want[kind], sets):
            call(out, x, kind, None)
            torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        for kind in ("decode", "prefill"):
            got = outs(kind, 4)
            torch.cuda.synchronize()
            torch.cuda._sleep(1_000_000)  # both streams start together
            with torch.cuda.stream(side):
                torch.cuda._sleep(1_000_000)
            for i, out in enumerate(got):
                s = None if i % 2 == 0 else side.cuda_stream if handle \
                    else side
                call(out, sets[i % 2], kind, s)
            torch.cuda.synchronize()
            for i, out in enumerate(got):
                assert torch.equal(out, want[kind][i % 2])


@pytest.mark.parametrize("q8", [False, True])
def test_append_on_a_stream_of_its_own(pkv, q8):
    """The same bits as on the current stream."""
    hq, hkv, d, bs, n = 8, 2, 64, 16, 30
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").half()
    table = torch.randperm(n, generator=g, device="cuda").int()[:, None]
    table = table.contiguous()
    lens = torch.arange(n, device="cuda").int() % bs + 1
    freqs = pkv.pa_rope_freqs(32)[0].cuda()
    pool0 = [torch.randn(n, hkv, bs, d, generator=g, device="cuda").to(
        E4M3 if q8 else torch.float16) for _ in "kv"]
    if q8:
        pool0 += [torch.full((n, hkv), 2.0 ** -8, device="cuda") for _ in "kv"]
    fn = pkv.pa_append_q8 if q8 else pkv.pa_append
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream):
        pool = [p.clone() for p in pool0]
        q = torch.zeros(n, hq, d, device="cuda").half()
        torch.cuda.synchronize()
        fn(q, *pool, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], table,
           lens, rope_freqs=freqs, rope_layout="interleaved", stream=stream)
        torch.cuda.synchronize()
        assert (q != 0).any(-1).all()
        got.append([q] + [p.view(torch.uint8) for p in pool])
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert not torch.equal(got[0][1], pool0[0].view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("handle", [False, True])
def test_captured_on_a_stream_without_a_workspace(pkv, q8, handle):
    """Attention captured on the stream it is given, its workspaces out of the
    graph's memory: replays equal eager calls, also with eager calls between
    that take their memory where the capture's was freed."""
    hq, hkv, d, bs = 16, 4, 64, 16
    torch.manual_seed(6)
    table = torch.randperm(60).int().view(2, 30).cuda()
    lens = torch.tensor([470, 33], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 9, 12], dtype=torch.int32, device="cuda")
    pool = [torch.randn(60, hkv, bs, d, device="cuda").to(
        E4M3 if q8 else torch.bfloat16) for _ in "kv"]
    if q8:
        pool += [torch.rand(60, hkv, device="cuda") + 0.5 for _ in "kv"]
    q = torch.randn(12, hq, d, device="cuda").bfloat16()
    decode = pkv.pa_decode_q8 if q8 else pkv.pa_decode
    prefill = pkv.pa_prefill_q8 if q8 else pkv.pa_prefill

    def step(a, b, stream=None):
        decode(a, q[:2], *pool, table, lens, 0.125, partition_size=32,
               stream=stream)
        prefill(b, q, *pool, table, lens, start, 0.125, max_q_len=9,
                stream=stream)

    want, got = ([torch.zeros_like(q[:2]), torch.zeros_like(q)] for _ in "12")
    step(*want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(*got, stream=side.cuda_stream if handle else side)
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        junk = [torch.full((1 << 16,), float("nan"), device="cuda")
                for _ in range(4)]
        step(*want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
