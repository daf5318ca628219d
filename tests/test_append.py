"""pa_append / pa_append_q8 / the 8-bit cache's calls on the host: refusals
(checked before any CUDA call), the rotation frequencies, and pins of the
oracle's own pieces."""
import ctypes
import math

import numpy as np
import pytest

from oracle import append as oap

FAKE = 0x1000


def _append_desc(**kw):
    from paged_kv_cache_383_b200 import _lib
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                block_size=16, max_blocks_per_seq=4, num_blocks=16, dtype=1,
                total_q=2, max_q_len=1, rot_dim=128, rope_layout=0,
                rope_scale=1.0, norm_eps=1e-6, q_stride=1024, k_stride=256,
                v_stride=256, q_out_stride=1024)
    base.update(kw)
    return _lib.pa_append_desc(**base)


def _call(name, desc, ptrs=None):
    from paged_kv_cache_383_b200 import _lib
    n = 12 if name == "pa_append" else 14
    ptrs = [FAKE] * n if ptrs is None else ptrs
    return getattr(_lib.load(), name)(*ptrs, ctypes.byref(desc), None, None)


@pytest.mark.parametrize("name", ["pa_append", "pa_append_q8"])
@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(num_kv_heads=0), 1),
    (dict(num_q_heads=-1), 1), (dict(dtype=2), 1), (dict(head_dim=96), 2),
    (dict(block_size=8), 2), (dict(block_size=64), 2), (dict(rot_dim=24), 2),
    (dict(rot_dim=144), 1), (dict(rot_dim=-16), 1), (dict(rope_layout=2), 1),
    (dict(rope_scale=math.inf), 1), (dict(norm_eps=-1.0), 1),
    (dict(norm_eps=math.nan), 1), (dict(q_stride=1020), 1),
    (dict(k_stride=128), 1), (dict(v_stride=260), 1),
    (dict(q_out_stride=512), 1), (dict(max_blocks_per_seq=1 << 28), 1),
    (dict(num_blocks=0), 1), (dict(total_q=-1), 1), (dict(max_q_len=-1), 1),
])
def test_append_rejects_bad_descriptors(pkv, name, kw, status):
    from paged_kv_cache_383_b200 import _lib
    assert _call(name, _append_desc(**kw)) == status
    assert name.encode() + b":" in _lib.load().pa_last_error()


@pytest.mark.parametrize("name", ["pa_append", "pa_append_q8"])
def test_append_rejects_null_and_misaligned(pkv, name):
    n = 12 if name == "pa_append" else 14
    q8 = name == "pa_append_q8"
    # q_out, k_cache, v_cache, [scales], q, k, v, (norms), freqs, table, lens
    optional = {n - 1: "query_start", n - 6: "q_norm", n - 5: "k_norm"}
    for i in range(n):
        ptrs = [FAKE] * n
        ptrs[i] = None
        if i in optional:
            continue
        assert _call(name, _append_desc(), ptrs) == 1, i
    for i in (0, 1, 2, n - 9, n - 8, n - 7, n - 6, n - 5):
        ptrs = [FAKE] * n
        ptrs[i] = FAKE + 8
        assert _call(name, _append_desc(), ptrs) == 1, i
    # without query_start: one row per sequence
    ptrs = [FAKE] * n
    ptrs[n - 1] = None
    assert _call(name, _append_desc(total_q=3), ptrs) == 1
    assert q8 == (n == 14)


@pytest.mark.parametrize("name", ["pa_append", "pa_append_q8"])
def test_append_in_place_needs_one_stride(pkv, name):
    """q_out == q (here all pointers are) with another row stride."""
    from paged_kv_cache_383_b200 import _lib
    assert _call(name, _append_desc(q_out_stride=1536)) == 1
    assert b"strides" in _lib.load().pa_last_error()


@pytest.mark.parametrize("name", ["pa_append", "pa_append_q8"])
def test_append_of_nothing_is_a_noop(pkv, name):
    n = 12 if name == "pa_append" else 14
    for kw in (dict(num_seqs=0, total_q=0), dict(total_q=0),
               dict(max_q_len=0)):
        ptrs = [FAKE] * n
        assert _call(name, _append_desc(**kw), ptrs) == 0


def test_decode_q8_rejects(pkv):
    from paged_kv_cache_383_b200 import _lib, pa_decode_desc
    lib = _lib.load()

    def call(ptrs=None, scale=1.0, ws=FAKE, wsb=1 << 20, **kw):
        base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                    block_size=16, max_blocks_per_seq=4, num_blocks=16,
                    dtype=1)
        base.update(kw)
        d = pa_decode_desc(**base)
        return lib.pa_decode_q8(*(ptrs or [FAKE] * 8), scale,
                                ctypes.byref(d), ws, wsb, None, None)
    assert call(head_dim=96) == 2
    assert call(block_size=64) == 2
    assert call(num_q_heads=32) == 2
    assert call(kernel=1) == 2          # no CUDA-core kernel here
    assert call(dtype=2) == 1
    assert call(scale=math.nan) == 1
    assert call(partition_size=24) == 1
    assert call(num_blocks=0) == 1
    assert call(ws=None, wsb=0) == _lib.PA_ERR_WORKSPACE
    assert call(num_seqs=0, ws=None) == 0
    for i in range(8):
        p = [FAKE] * 8
        p[i] = None
        assert call(p) == 1, i
    for i in range(4):
        p = [FAKE] * 8
        p[i] = FAKE + 8
        assert call(p) == 1, i
    assert b"pa_decode_q8" in lib.pa_last_error()


def test_prefill_q8_rejects(pkv):
    from paged_kv_cache_383_b200 import _lib
    lib = _lib.load()

    def call(ptrs=None, scale=1.0, ws=FAKE, wsb=1 << 20, **kw):
        base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                    block_size=16, max_blocks_per_seq=4, num_blocks=16,
                    dtype=1, total_q=10, max_q_len=8)
        base.update(kw)
        d = _lib.pa_prefill_desc(**base)
        return lib.pa_prefill_q8(*(ptrs or [FAKE] * 9), scale,
                                 ctypes.byref(d), ws, wsb, None, None)
    assert call(head_dim=96) == 2
    assert call(block_size=64) == 2
    assert call(num_q_heads=6) == 2
    assert call(num_q_heads=7) == 1
    assert call(dtype=2) == 1
    assert call(kernel=2) == 1
    assert call(pv=3) == 1
    assert call(out_fp32=2) == 1
    assert call(scale=math.inf) == 1
    assert call(num_blocks=0) == 1
    assert call(ws=None) == _lib.PA_ERR_WORKSPACE
    assert call(wsb=16) == _lib.PA_ERR_WORKSPACE
    assert call(total_q=0, ws=None) == 0
    for i in range(9):
        p = [FAKE] * 9
        p[i] = None
        assert call(p) == 1, i
    for i in range(4):
        p = [FAKE] * 9
        p[i] = FAKE + 8
        assert call(p) == 1, i
    assert b"pa_prefill_q8" in lib.pa_last_error()


def test_block_moves_q8_reject(pkv):
    from paged_kv_cache_383_b200 import _lib
    lib = _lib.load()
    ok = [FAKE] * 5
    assert lib.pa_copy_blocks_q8(*ok, 0, 2, 128, 16, 4, None, None) == 0
    assert lib.pa_copy_blocks_q8(*ok, -1, 2, 128, 16, 4, None, None) == 1
    assert lib.pa_copy_blocks_q8(*ok, 1, 2, 24, 16, 4, None, None) == 2
    for i in range(5):
        p = list(ok)
        p[i] = None
        assert lib.pa_copy_blocks_q8(*p, 1, 2, 128, 16, 4, None, None) == 1
    assert lib.pa_copy_blocks_q8(FAKE + 8, FAKE, FAKE, FAKE, FAKE, 1, 2, 128,
                                 16, 4, None, None) == 1
    assert lib.pa_swap_blocks_q8(*[None] * 9, 1, 2, 128, 16, 4, 4, None,
                                 None) == 1
    assert lib.pa_swap_blocks_q8(*[None] * 9, 0, 2, 128, 16, 4, 4, None,
                                 None) == 0


def test_pool_blocks_q8(pkv):
    per = 2 * 3 * 8 * (128 * 16 + 4)
    assert pkv.pa_pool_blocks_q8(per * 7 + per - 1, 3, 8, 128, 16) == 7
    with pytest.raises(pkv.PagedKVError):
        pkv.pa_pool_blocks_q8(1 << 30, 0, 8, 128, 16)


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0)])
def test_rope_freqs(pkv, rot, base):
    j = np.arange(rot // 2)
    plain = base ** (-2.0 * j / rot)
    f, s = pkv.pa_rope_freqs(rot, base)
    np.testing.assert_allclose(f.numpy(), plain, rtol=1e-14)
    assert s == 1.0
    f, s = pkv.pa_rope_freqs(rot, base, scaling="linear", factor=4.0)
    np.testing.assert_allclose(f.numpy(), plain / 4, rtol=1e-14)
    assert s == 1.0
    # by wavelength: long waves are stretched, short ones kept
    f, s = pkv.pa_rope_freqs(rot, base, scaling="wavelength", factor=8.0,
                             original_len=8192, low=1.0, high=4.0)
    wave = 2 * np.pi / plain
    smooth = (8192 / wave - 1.0) / 3.0
    want = np.where(wave < 8192 / 4, plain,
                    np.where(wave > 8192, plain / 8,
                             (1 - smooth) * plain / 8 + smooth * plain))
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-12)
    # yarn: a ramp over the pairs
    f, s = pkv.pa_rope_freqs(rot, base, scaling="yarn", factor=4.0,
                             original_len=4096, low=1.0, high=32.0)

    def pair(turns):
        return rot * math.log(4096 / (turns * 2 * math.pi)) / (
            2 * math.log(base))
    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)),
                                                 rot - 1)
    ramp = np.clip((j - lo) / (hi - lo), 0, 1)
    np.testing.assert_allclose(f.numpy(), plain / 4 * ramp +
                               plain * (1 - ramp), rtol=1e-12)
    assert s == pytest.approx(0.1 * math.log(4.0) + 1, rel=1e-6)


def test_rope_freqs_rejects(pkv):
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0),
               dict(rot_dim=64, scaling="linear", factor=0.5),
               dict(rot_dim=64, scaling="yarn", factor=2.0),
               dict(rot_dim=64, scaling="wavelength", factor=2.0,
                    original_len=8, low=4.0, high=4.0)):
        with pytest.raises(pkv.PagedKVError):
            pkv.pa_rope_freqs(**kw)
    with pytest.raises(ValueError):
        pkv.pa_rope_freqs(64, scaling="other")


def test_python_refusals(pkv):
    """What the binding itself refuses, on CPU tensors."""
    import torch
    bf = torch.bfloat16
    kc = torch.zeros(4, 2, 16, 128, dtype=bf)
    row = torch.zeros(2, 2, 128, dtype=bf)
    t = torch.zeros(2, 3, dtype=torch.int32)
    n = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="come together"):
        pkv.pa_append(None, kc, kc, row, row, row, t, n)
    with pytest.raises(ValueError, match="one row per"):
        pkv.pa_append(None, kc, kc, None, row[:1], row[:1], t, n)
    with pytest.raises(ValueError, match="query_start"):
        pkv.pa_append(None, kc, kc, None, row, row, t, n, n)
    with pytest.raises(ValueError, match="dense"):
        wide = torch.zeros(2, 2, 256, dtype=bf)[..., :128]
        pkv.pa_append(None, kc, kc, None, wide, row, t, n)
    with pytest.raises(TypeError):
        pkv.pa_append(None, kc, kc, None, row, row.half(), t, n)
    with pytest.raises(ValueError, match="rope_layout"):
        pkv.pa_append(None, kc, kc, None, row, row, t, n, rope_layout="x")
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="k_scales"):
        pkv.pa_append_q8(None, kc, kc, s[:3], s, None, row, row, t, n)


def test_decode_q8_refuses_a_stale_descriptor(pkv):
    """A descriptor made for other shapes would send the kernel past the
    tensors' ends."""
    import torch
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    kc = torch.zeros(5, 2, 16, 64).to(torch.float8_e4m3fn)
    ks = torch.ones(5, 2)
    table = torch.zeros(2, 3, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    for dq, dkc, dt in ((q.repeat(2, 1, 1), kc, table.repeat(2, 1)),
                        (q.repeat(1, 2, 1), kc, table),
                        (q, kc.repeat(2, 1, 1, 1), table),
                        (q, kc, table.repeat(1, 2)), (q.half(), kc, table)):
        desc = pkv.make_desc(dq, dkc, dt)
        with pytest.raises(ValueError, match="desc does not describe"):
            pkv.pa_decode_q8(torch.empty_like(q), q, kc, kc, ks, ks, table,
                             lens, 0.1, desc=desc)


def test_oracle_e4m3():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(oap.e4m3_table(), want.astype(np.float64))
    x = np.random.default_rng(0).standard_normal(20000) * 60
    got = torch.from_numpy(x.astype(np.float32)).to(
        torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(oap.e4m3_round(x.astype(np.float32)), got)


def test_oracle_scale_and_rotation():
    assert oap.scale_for(448.0) == 1.0
    assert oap.scale_for(448.0001) == 2.0
    assert oap.scale_for(0.0) == 2.0 ** -64
    assert oap.scale_for(math.inf) == 2.0 ** 120
    x = np.random.default_rng(1).standard_normal(64)
    f = 10000.0 ** (-np.arange(16) / 16)
    for layout in ("half", "interleaved"):
        y = oap.rotate_head(x, 12345, f, layout, 1.0)
        # lengths of the pairs stay, the rest of the head is untouched
        assert np.allclose(np.sum(y * y), np.sum(x * x))
        np.testing.assert_array_equal(y[32:], x[32:])
        # rotations by p and q differ by the rotation of p - q
        z = oap.rotate_head(oap.rotate_head(x, 45, f, layout, 1.0), 12300, f,
                            layout, 1.0)
        np.testing.assert_allclose(y, z, atol=1e-9)


def test_workspace_belongs_to_the_stream_it_is_used_on(pkv, monkeypatch):
    """Allocated while another stream is current, it could be memory that a
    call queued there still uses."""
    import contextlib

    import torch
    current, at = ["caller's"], []

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: ("handle", handle))
    pkv._torch_refs()
    monkeypatch.setitem(pkv._tc, "empty",
                        lambda *a, **k: at.append(current[-1]))
    for stream in (None, "side", 77):
        pkv._workspace(64, "cuda:0", stream)
    assert at == ["caller's", "side", ("handle", 77)]


def test_16_bit_attention_takes_its_workspace_the_same_way(pkv, monkeypatch):
    import torch
    asked = []

    def workspace(need, device, stream):
        asked.append((need, stream))
        raise KeyboardInterrupt
    monkeypatch.setattr(pkv, "_workspace", workspace)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    kc = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    start = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(KeyboardInterrupt):
        pkv.pa_decode(q, q, kc, kc, table, lens, 0.1, stream="side")
    with pytest.raises(KeyboardInterrupt):
        pkv.pa_prefill(q, q, kc, kc, table, lens, start, 0.1, max_q_len=1,
                       stream="side")
    assert [s for _, s in asked] == ["side", "side"]
    assert all(n > 0 for n, _ in asked)


def test_rope_freqs_default_bands(pkv):
    """Without low and high, each method's own: 1 and 32 turns for yarn, 1 and
    4 by wavelength; one of them may be given alone."""
    import torch
    kw = dict(base=10000.0, factor=8.0, original_len=8192)
    for scaling, high in (("yarn", 32.0), ("wavelength", 4.0)):
        want, _ = pkv.pa_rope_freqs(128, scaling=scaling, low=1.0, high=high,
                                    **kw)
        for band in ({}, {"low": 1.0}, {"high": high}):
            got, _ = pkv.pa_rope_freqs(128, scaling=scaling, **band, **kw)
            assert torch.equal(got, want)
        other, _ = pkv.pa_rope_freqs(128, scaling=scaling, high=2 * high, **kw)
        assert not torch.equal(other, want)


@pytest.mark.parametrize("name", ["pa_append", "pa_append_q8"])
def test_append_without_query_start_needs_no_bound(pkv, name):
    """max_q_len 0 there is no call without rows: the checks behind that exit
    (here the pool's) are reached."""
    from paged_kv_cache_383_b200 import _lib
    n = 12 if name == "pa_append" else 14
    ptrs = [FAKE] * (n - 1) + [None]
    assert _call(name, _append_desc(max_q_len=0, num_blocks=0), ptrs) == 1
    assert b"empty block pool" in _lib.load().pa_last_error()


@pytest.mark.parametrize("name", ["pa_prefill", "pa_prefill_q8"])
@pytest.mark.parametrize("bs", [16, 32])
def test_prefill_refuses_a_table_past_2_31_tokens(pkv, name, bs):
    """Its token count would not fit the kernels' 32-bit lengths; the largest
    that does is let through (to the check of the workspace)."""
    from paged_kv_cache_383_b200 import _lib
    lib = _lib.load()

    def call(blocks):
        d = _lib.pa_prefill_desc(
            num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
            block_size=bs, max_blocks_per_seq=blocks, num_blocks=16, dtype=1,
            total_q=10, max_q_len=8)
        n = 7 if name == "pa_prefill" else 9
        return getattr(lib, name)(*[FAKE] * n, 1.0, ctypes.byref(d), None, 0,
                                  None, None)
    assert call(2 ** 31 // bs) == 1
    assert name.encode() + b": max_blocks_per_seq" in lib.pa_last_error()
    assert call(2 ** 32 // bs + 4) == 1
    assert call(2 ** 31 // bs - 1) == _lib.PA_ERR_WORKSPACE
