"""Paged KV-cache decode attention for NVIDIA B200 (sm_100a).

Python binding of libpagedkv.so.  The functions keep the C ABI's names
(``pa_decode``, ``pa_cache_write``, ``pa_copy_blocks``, ``pa_bm_*``) and only
marshal arguments: they take torch tensors for device memory and streams,
check dtypes / devices / contiguity, and pass raw pointers to the library.
All computation happens in the library's CUDA kernels and C++ block manager;
if the library is missing, every call raises.

Layouts (see include/pagedkv.h for the full contract):
  q, out            [num_seqs, num_q_heads, head_dim]            fp16 / bf16
                    (out may be float32: the value before the final rounding)
  k_cache, v_cache  [num_blocks, num_kv_heads, block_size, head_dim]
  block_tables      [num_seqs, max_blocks_per_seq] int32
  context_lens      [num_seqs] int32
  k, v (new tokens) [num_tokens, num_kv_heads, head_dim]
  slot_mapping      [num_tokens] int64
  pairs             [num_pairs, 2] int32
8-bit cache (the ``*_q8`` calls):
  k_cache, v_cache  as above, torch.float8_e4m3fn
  k_scales, v_scales  [num_blocks, num_kv_heads] float32
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (PA_BF16, PA_F16, PA_KERNEL_AUTO, PA_KERNEL_MMA,
                   PA_KERNEL_SIMT, PagedKVError, NoFreeBlocksError,
                   pa_decode_desc)

__all__ = [
    "pa_decode", "pa_decode_noalloc", "pa_prefill", "pa_prefill_workspace_bytes",
    "pa_cache_write",
    "pa_copy_blocks",
    "pa_append", "pa_append_q8", "pa_rope_freqs", "pa_decode_q8",
    "pa_prefill_q8",
    "pa_copy_blocks_q8", "pa_swap_blocks_q8",
    "pa_pool_blocks_q8",
    "pa_decode_workspace_bytes", "pa_decode_partition_size", "make_desc",
    "BlockManager", "PagedKVError", "NoFreeBlocksError", "library_path",
    "pa_launch_count", "pa_read_probe", "pa_wait_probe",
    "PA_KERNEL_AUTO", "PA_KERNEL_MMA", "PA_KERNEL_SIMT",
]

_KERNELS = {"auto": PA_KERNEL_AUTO, "mma": PA_KERNEL_MMA,
            "simt": PA_KERNEL_SIMT}
_REDUCES = {"auto": _lib.PA_REDUCE_AUTO, "kernel": _lib.PA_REDUCE_KERNEL}
_PREFILL_KERNELS = {"auto": _lib.PA_PREFILL_AUTO, "tile": _lib.PA_PREFILL_TILE}
_PREFILL_PV = {"auto": _lib.PA_PV_AUTO, "split": _lib.PA_PV_SPLIT,
               "single": _lib.PA_PV_SINGLE}


def library_path() -> str:
    return _lib.LIB_PATH


def pa_read_probe(buf, sink, stream=None):
    """Read the whole CUDA tensor ``buf`` once with streaming loads (a
    bandwidth measurement helper); ``sink`` is an int32 CUDA tensor."""
    import torch
    st = _lib.load().pa_read_probe(
        _dev(buf, "buf"), buf.numel() * buf.element_size(),
        _dev(sink, "sink", torch.int32), _stream(stream))
    _lib.check(st, "pa_read_probe")


def pa_wait_probe(dev_err, stream=None):
    """Make one bounded device wait run out (about 1 s of device time): the
    kernel sets ``dev_err`` (an int32 CUDA tensor) to PA_ERR_DEVICE_TIMEOUT,
    frees its tensor memory and returns, as the attention kernels do when a
    copy never lands."""
    import torch
    if dev_err is None:
        raise ValueError("pa_wait_probe needs a dev_err tensor")
    st = _lib.load().pa_wait_probe(_dev(dev_err, "dev_err", torch.int32),
                                   _stream(stream))
    _lib.check(st, "pa_wait_probe")


def pa_launch_count() -> int:
    """Kernel launches libpagedkv has issued in this process."""
    return int(_lib.load().pa_launch_count())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return PA_F16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


def _dev(t, name: str, dtype=None):
    """Pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_desc(q, k_cache, block_tables, *, partition_size: int = 0,
              max_context_len: int = 0, kernel: str = "auto",
              reduce: str = "auto") -> pa_decode_desc:
    """Decode descriptor from tensor shapes."""
    num_seqs, num_q_heads, head_dim = q.shape
    num_blocks, num_kv_heads, block_size, hd2 = k_cache.shape
    if hd2 != head_dim:
        raise ValueError("q and k_cache disagree on head_dim")
    if block_tables.shape[0] != num_seqs:
        raise ValueError("block_tables rows != num_seqs")
    return pa_decode_desc(
        num_seqs=num_seqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
        head_dim=head_dim, block_size=block_size,
        max_blocks_per_seq=block_tables.shape[1], num_blocks=num_blocks,
        dtype=_dtype_code(q), partition_size=partition_size,
        max_context_len=max_context_len, kernel=_KERNELS[kernel],
        reduce=_REDUCES[reduce])


def _out_mode(desc, out, dt):
    """``out`` in q's dtype, or float32: the value before the final rounding
    (desc.out_fp32 follows the tensor)."""
    import torch
    if out.dtype == dt:
        desc.out_fp32 = 0
    elif out.dtype == torch.float32:
        desc.out_fp32 = 1
    else:
        raise TypeError(f"out dtype {out.dtype} is neither q's dtype {dt} "
                        "nor float32")


def pa_decode_workspace_bytes(desc: pa_decode_desc) -> int:
    return int(_lib.load().pa_decode_workspace_bytes(ctypes.byref(desc)))


def pa_decode_partition_size(desc: pa_decode_desc) -> int:
    ps = _lib.load().pa_decode_partition_size(ctypes.byref(desc))
    if ps < 0:
        _lib.check(_lib.PA_ERR_INVALID_ARG, "pa_decode_partition_size")
    return ps


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens,
              scale: float, *, partition_size: int = 0,
              max_context_len: int = 0, kernel: str = "auto",
              reduce: str = "auto", workspace=None, dev_err=None,
              stream=None, desc: pa_decode_desc | None = None):
    """out[b, h] = softmax(scale * K_b q[b, h]) V_b over each sequence's
    paged K/V.  ``workspace`` (uint8 CUDA tensor) is allocated with torch when
    the call needs one and none is given.  Returns ``out``."""
    import torch
    lib = _lib.load()
    if desc is None:
        desc = make_desc(q, k_cache, block_tables,
                         partition_size=partition_size,
                         max_context_len=max_context_len, kernel=kernel,
                         reduce=reduce)
    dt = q.dtype
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != dt:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {dt}")
    _out_mode(desc, out, dt)
    need = int(lib.pa_decode_workspace_bytes(ctypes.byref(desc)))
    if need and workspace is None:
        _tc or _torch_refs()
        workspace = _workspace(need, q.device, stream)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() \
        if workspace is not None else 0
    st = lib.pa_decode(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32),
        ctypes.c_float(scale), ctypes.byref(desc), ws_ptr, ws_bytes,
        _dev(dev_err, "dev_err", torch.int32), _stream(stream))
    _lib.check(st, "pa_decode")
    return out


def pa_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                      scale: float, *, partition_size: int = 0,
                      max_context_len: int = 0, kernel: str = "auto",
                      reduce: str = "auto", dev_err=None, stream=None,
                      desc: pa_decode_desc | None = None):
    """pa_decode for callers that cannot allocate device memory: the
    workspace is the library's built-in scratch area
    (PA_NOALLOC_SCRATCH_BYTES per device), so this wrapper allocates nothing
    either.  Calls that overlap on one device race on that area.  Returns
    ``out``."""
    import torch
    lib = _lib.load()
    if desc is None:
        desc = make_desc(q, k_cache, block_tables,
                         partition_size=partition_size,
                         max_context_len=max_context_len, kernel=kernel,
                         reduce=reduce)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    _out_mode(desc, out, q.dtype)
    st = lib.pa_decode_noalloc(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32),
        ctypes.c_float(scale), ctypes.byref(desc),
        _dev(dev_err, "dev_err", torch.int32), _stream(stream))
    _lib.check(st, "pa_decode_noalloc")
    return out


def _prefill_desc(q, k_cache, block_tables, max_q_len, max_context_len,
                  kernel="auto", pv="auto"):
    total_q, num_q_heads, head_dim = q.shape
    num_blocks, num_kv_heads, block_size, hd2 = k_cache.shape
    if hd2 != head_dim:
        raise ValueError("q and the caches disagree on head_dim")
    return _lib.pa_prefill_desc(
        num_seqs=block_tables.shape[0], num_q_heads=num_q_heads,
        num_kv_heads=num_kv_heads, head_dim=head_dim, block_size=block_size,
        max_blocks_per_seq=block_tables.shape[1], num_blocks=num_blocks,
        dtype=_dtype_code(q), total_q=total_q, max_q_len=max_q_len,
        max_context_len=max_context_len, kernel=_PREFILL_KERNELS[kernel],
        pv=_PREFILL_PV[pv])


def pa_prefill_workspace_bytes(q, k_cache, block_tables, *,
                               max_q_len: int | None = None) -> int:
    """Bytes of device workspace ``pa_prefill`` needs for these tensors and
    ``max_q_len`` (default: every row of ``q``): the sequence order and the
    tile map (``pa_prefill_workspace_bytes`` of the C ABI)."""
    if max_q_len is None:
        max_q_len = q.shape[0]
    desc = _prefill_desc(q, k_cache, block_tables, max_q_len, 0)
    return int(_lib.load().pa_prefill_workspace_bytes(ctypes.byref(desc)))


def pa_prefill(out, q, k_cache, v_cache, block_tables, context_lens,
               query_start, scale: float, *, max_q_len: int,
               max_context_len: int = 0, kernel: str = "auto",
               pv: str = "auto", workspace=None, dev_err=None, stream=None):
    """Causal attention of each sequence's new tokens (rows
    query_start[b] .. query_start[b+1]-1 of ``q``) over its paged K/V, the
    new tokens being the last ones of the context.  ``max_q_len`` bounds
    every sequence's new-token count (it picks the layout; a sequence above
    it is flagged and left unwritten).  ``kernel``: "auto" or "tile" (the
    same kernel).  ``pv``: precision of P in P . V -- "auto" (P's residual
    added in the tiles that need it), "split" (in every tile) or "single"
    (one rounding of P).  ``workspace`` (a uint8 device tensor of
    ``pa_prefill_workspace_bytes`` bytes) is allocated per call when not
    given.  Returns ``out``."""
    import torch
    lib = _lib.load()
    if out.shape != q.shape:
        raise ValueError("q and out disagree on shape")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != q.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    desc = _prefill_desc(q, k_cache, block_tables, max_q_len, max_context_len,
                         kernel, pv)
    _out_mode(desc, out, q.dtype)
    need = lib.pa_prefill_workspace_bytes(ctypes.byref(desc))
    if workspace is None:
        _tc or _torch_refs()
        workspace = _workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.pa_prefill(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32),
        _dev(query_start, "query_start", torch.int32),
        ctypes.c_float(scale), ctypes.byref(desc),
        _dev(workspace, "workspace"), ctypes.c_size_t(ws_bytes),
        _dev(dev_err, "dev_err", torch.int32), _stream(stream))
    _lib.check(st, "pa_prefill")
    return out


def _reachable(t, name: str, dtype=None):
    """Pointer of a contiguous CUDA tensor or pinned (page-locked) CPU
    tensor; the library checks that the device can reach it."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned CPU memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def pa_swap_blocks(dst_k, dst_v, src_k, src_v, pairs, *, dev_err=None,
                   stream=None):
    """Copy block pairs[i, 0] of (src_k, src_v) to block pairs[i, 1] of
    (dst_k, dst_v); any of the pools (and ``pairs``) may be pinned CPU
    tensors, e.g. a host pool for swapped-out sequences."""
    import torch
    lib = _lib.load()
    ns, hkv, bs, d = src_k.shape
    nd = dst_k.shape[0]
    for name, t, n in (("dst_k", dst_k, nd), ("dst_v", dst_v, nd),
                       ("src_v", src_v, ns)):
        if t.shape != (n, hkv, bs, d):
            raise ValueError(f"{name} shape {tuple(t.shape)} does not match")
        if t.dtype != src_k.dtype:
            raise TypeError(f"{name} dtype differs from src_k")
    if pairs.ndim != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    st = lib.pa_swap_blocks(
        _reachable(dst_k, "dst_k"), _reachable(dst_v, "dst_v"),
        _reachable(src_k, "src_k"), _reachable(src_v, "src_v"),
        _reachable(pairs, "pairs", torch.int32), pairs.shape[0], hkv, d, bs,
        ns, nd, _dtype_code(src_k), _dev(dev_err, "dev_err", torch.int32),
        _stream(stream))
    _lib.check(st, "pa_swap_blocks")


def pa_pool_blocks(nbytes: int, num_layers: int, num_kv_heads: int,
                   head_dim: int, block_size: int, dtype) -> int:
    """Blocks of block_size tokens (K and V of every layer) that fit in
    ``nbytes``; ``dtype`` is torch.float16 or torch.bfloat16."""
    import torch
    code = {torch.float16: PA_F16, torch.bfloat16: PA_BF16}.get(dtype)
    if code is None:
        raise TypeError(f"expected float16 or bfloat16, got {dtype}")
    n = _lib.load().pa_pool_blocks(int(nbytes), num_layers, num_kv_heads,
                                   head_dim, block_size, code)
    if n < 0:
        _lib.check(_lib.PA_ERR_INVALID_ARG, "pa_pool_blocks")
    return n


def pa_cache_write(k_cache, v_cache, k, v, slot_mapping, *, dev_err=None,
                   stream=None):
    """Copy each new token's K and V rows into cache slot slot_mapping[t]
    (negative slots are skipped)."""
    import torch
    lib = _lib.load()
    num_blocks, num_kv_heads, block_size, head_dim = k_cache.shape
    num_tokens = k.shape[0]
    if k.shape != (num_tokens, num_kv_heads, head_dim) or v.shape != k.shape:
        raise ValueError("k, v must be [num_tokens, num_kv_heads, head_dim]")
    if slot_mapping.shape != (num_tokens,):
        raise ValueError("slot_mapping must be [num_tokens]")
    for name, t in (("v_cache", v_cache), ("k", k), ("v", v)):
        if t.dtype != k_cache.dtype:
            raise TypeError(f"{name} dtype {t.dtype} != k_cache dtype")
    st = lib.pa_cache_write(
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _dev(k, "k"),
        _dev(v, "v"), _dev(slot_mapping, "slot_mapping", torch.int64),
        num_tokens, num_kv_heads, head_dim, block_size, num_blocks,
        _dtype_code(k_cache), _dev(dev_err, "dev_err", torch.int32),
        _stream(stream))
    _lib.check(st, "pa_cache_write")


def pa_copy_blocks(k_cache, v_cache, pairs, *, dev_err=None, stream=None):
    """k_cache[dst] = k_cache[src] and v_cache[dst] = v_cache[src] for every
    (src, dst) row of ``pairs`` (int32 [n, 2] on the device)."""
    import torch
    lib = _lib.load()
    num_blocks, num_kv_heads, block_size, head_dim = k_cache.shape
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [num_pairs, 2]")
    if v_cache.dtype != k_cache.dtype:
        raise TypeError("k_cache and v_cache dtypes differ")
    st = lib.pa_copy_blocks(
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(pairs, "pairs", torch.int32), pairs.shape[0], num_kv_heads,
        head_dim, block_size, num_blocks, _dtype_code(k_cache),
        _dev(dev_err, "dev_err", torch.int32), _stream(stream))
    _lib.check(st, "pa_copy_blocks")


# -- rotating append, 8-bit cache ---------------------------------------------
_ROPE_LAYOUTS = {"half": _lib.PA_ROPE_HALF,
                 "interleaved": _lib.PA_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {None: _lib.PA_ROPE_PLAIN, "linear": _lib.PA_ROPE_LINEAR,
                  "wavelength": _lib.PA_ROPE_WAVELENGTH,
                  "yarn": _lib.PA_ROPE_YARN}


# What the calls below ask of torch on every call, looked up once: a decode
# step's device work is a few microseconds, as much as a few dozen Python
# attribute lookups.
_tc: dict = {}


def _torch_refs():
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        def raw(dev):
            return torch.cuda.current_stream(dev).cuda_stream
    _tc.update(device=torch.cuda.current_device, raw_stream=raw,
               i32=torch.int32, f32=torch.float32, f64=torch.float64,
               e4m3=torch.float8_e4m3fn,
               codes={torch.float16: PA_F16, torch.bfloat16: PA_BF16},
               empty=torch.empty, u8=torch.uint8)
    return _tc


def _ptr(t, name: str, dev: int, dtype=None):
    """Pointer of a contiguous tensor on device ``dev``, the current one: the
    library launches there, so a tensor of another device is refused.  None
    gives NULL."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current "
                         f"device (cuda:{dev}), is on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream_on(stream, dev: int) -> int:
    if stream is None:
        return _tc["raw_stream"](dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _code(dt) -> int:
    code = _tc["codes"].get(dt)
    if code is None:
        raise TypeError(f"expected float16 or bfloat16, got {dt}")
    return code


def _workspace(need: int, device, stream):
    """A workspace of the call's own, out of the memory that torch keeps for
    the stream the call runs on.  Memory of another stream's would not do:
    torch hands it out as soon as that stream's last user is queued, and that
    user may still be running when this call starts."""
    if stream is None:
        return _tc["empty"](max(need, 16), dtype=_tc["u8"], device=device)
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return _tc["empty"](max(need, 16), dtype=_tc["u8"], device=device)


def _check_q8(k_cache, v_cache, k_scales, v_scales, names=("", "")):
    """Shapes of an 8-bit pool; returns (num_blocks, heads, block, dim)."""
    a, b = names
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"{a}k_cache and {a}v_cache must be [num_blocks, "
                         "num_kv_heads, block_size, head_dim]")
    if k_scales.shape != shape[:2] or v_scales.shape != shape[:2]:
        raise ValueError(f"{a}k_scales and {a}v_scales must be [num_blocks, "
                         "num_kv_heads]")
    return shape


# Turns over original_len between which a pair is partly scaled: each method's
# published values.
_ROPE_BANDS = {"wavelength": (1.0, 4.0), "yarn": (1.0, 32.0)}


def pa_rope_freqs(rot_dim: int, base: float = 10000.0, *, scaling=None,
                  factor: float = 1.0, original_len: int = 0,
                  low: float | None = None, high: float | None = None):
    """(freqs, rope_scale) for ``pa_append``: the angular frequencies of the
    rot_dim/2 pairs as a float64 CPU tensor (move it to the device once) and
    the factor of cos and sin.  ``scaling``: None, "linear", "wavelength" or
    "yarn" (``low`` / ``high``: turns over ``original_len``, by default 1 and
    4 for "wavelength", 1 and 32 for "yarn")."""
    import torch
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is none of "
                         f"{list(_ROPE_SCALINGS)}")
    band = _ROPE_BANDS.get(scaling, (0.0, 0.0))
    low = band[0] if low is None else low
    high = band[1] if high is None else high
    d = _lib.pa_rope_desc(rot_dim=rot_dim, scaling=_ROPE_SCALINGS[scaling],
                          original_len=original_len, base=base, factor=factor,
                          low=low, high=high)
    out = (ctypes.c_double * max(rot_dim // 2, 1))()
    sc = ctypes.c_float()
    _lib.check(_lib.load().pa_rope_freqs(ctypes.byref(d), out,
                                         ctypes.byref(sc)), "pa_rope_freqs")
    return torch.tensor(list(out), dtype=torch.float64), float(sc.value)


def _rows(t, name: str, shape, dt, dev: int):
    """(pointer, row stride) of a [rows, heads, head_dim] tensor whose heads
    are dense within a row (a slice of a projection's output, say)."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, is {list(t.shape)}")
    if t.dtype != dt:
        raise TypeError(f"{name} dtype {t.dtype} != {dt}")
    s0, s1, s2 = t.stride()
    rows, heads, head_dim = shape
    if s2 != 1 or (s1 != head_dim and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be dense "
                         f"(strides {t.stride()})")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current "
                         f"device (cuda:{dev}), is on {t.device}")
    return t.data_ptr(), s0 if rows > 1 else heads * head_dim


def _append(fn, name, q_out, k_cache, v_cache, scales, q, k, v, block_tables,
            context_lens, query_start, max_q_len, q_norm, k_norm, norm_eps,
            rope_freqs, rope_layout, rope_scale, dev_err, stream):
    tc = _tc or _torch_refs()
    shape = k_cache.shape
    num_blocks, hkv, block_size, head_dim = shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache differ in shape")
    total, dt = k.shape[0], k.dtype
    num_seqs = context_lens.shape[0]
    bt = block_tables.shape
    if context_lens.dim() != 1 or len(bt) != 2 or bt[0] != num_seqs:
        raise ValueError("context_lens must be [num_seqs] and block_tables "
                         "[num_seqs, max_blocks_per_seq]")
    if query_start is None:
        if total != num_seqs:
            raise ValueError("without query_start there is one row per "
                             f"sequence: {num_seqs} sequences, {total} rows")
        max_q_len = 1
    else:
        if query_start.shape != (num_seqs + 1,):
            raise ValueError("query_start must be [num_seqs + 1]")
        if max_q_len is None:
            max_q_len = total
    layout = _ROPE_LAYOUTS.get(rope_layout)
    if layout is None:
        raise ValueError(f"rope_layout {rope_layout!r} is none of "
                         f"{list(_ROPE_LAYOUTS)}")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    dev = k_cache.get_device()
    kv_shape = (total, hkv, head_dim)
    k_ptr, ks = _rows(k, "k", kv_shape, dt, dev)
    v_ptr, vs = _rows(v, "v", kv_shape, dt, dev)
    hq = qs = os = 0
    q_ptr = out_ptr = None
    if q is not None:
        hq = q.shape[1]
        q_shape = (total, hq, head_dim)
        q_ptr, qs = _rows(q, "q", q_shape, dt, dev)
        out_ptr, os = _rows(q_out, "q_out", q_shape, dt, dev)
    if dev != tc["device"]():
        raise ValueError(f"the caches are on {k_cache.device}, which is not "
                         "the current CUDA device")
    for w, n in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if w is not None and w.shape != (head_dim,):
            raise ValueError(f"{n} must be [{head_dim}]")
    rot_dim = 0
    if rope_freqs is not None:
        if rope_freqs.dim() != 1:
            raise ValueError("rope_freqs must be [rot_dim / 2]")
        rot_dim = 2 * rope_freqs.shape[0]
    i32 = tc["i32"]
    cache_dt = tc["e4m3"] if scales else dt
    desc = _lib.pa_append_desc(
        num_seqs, hq, hkv, head_dim, block_size, bt[1], num_blocks, _code(dt),
        total, max_q_len, rot_dim, layout, rope_scale, norm_eps, qs, ks, vs,
        os)
    st = fn(out_ptr, _ptr(k_cache, "k_cache", dev, cache_dt),
            _ptr(v_cache, "v_cache", dev, cache_dt),
            *[_ptr(t, n, dev, tc["f32"]) for t, n in scales],
            q_ptr, k_ptr, v_ptr, _ptr(q_norm, "q_norm", dev, dt),
            _ptr(k_norm, "k_norm", dev, dt),
            _ptr(rope_freqs, "rope_freqs", dev, tc["f64"]),
            _ptr(block_tables, "block_tables", dev, i32),
            _ptr(context_lens, "context_lens", dev, i32),
            _ptr(query_start, "query_start", dev, i32), ctypes.byref(desc),
            _ptr(dev_err, "dev_err", dev, i32), _stream_on(stream, dev))
    if st:
        _lib.check(st, name)
    return q_out


def pa_append(q_out, k_cache, v_cache, q, k, v, block_tables, context_lens,
              query_start=None, *, max_q_len: int | None = None, q_norm=None,
              k_norm=None, norm_eps: float = 1e-6, rope_freqs=None,
              rope_layout: str = "half", rope_scale: float = 1.0,
              dev_err=None, stream=None):
    """Norm (``q_norm`` / ``k_norm``: [head_dim] weights) and position
    rotation (``rope_freqs``: float64 [rot_dim/2], see ``pa_rope_freqs``) of
    the new tokens' queries and keys, queries into ``q_out``, keys and values
    into the paged cache, in one launch.  Rows as for ``pa_prefill``: the
    last tokens of each context; without ``query_start`` one row per
    sequence (a decode step).  q, k, v and q_out may be row slices of a wider
    tensor; q_out may be q.  Returns ``q_out``."""
    return _append(_lib.load().pa_append, "pa_append", q_out, k_cache,
                   v_cache, (), q, k, v, block_tables, context_lens,
                   query_start, max_q_len, q_norm, k_norm, norm_eps,
                   rope_freqs, rope_layout, rope_scale, dev_err, stream)


def pa_append_q8(q_out, k_cache, v_cache, k_scales, v_scales, q, k, v,
                 block_tables, context_lens, query_start=None, *,
                 max_q_len: int | None = None, q_norm=None, k_norm=None,
                 norm_eps: float = 1e-6, rope_freqs=None,
                 rope_layout: str = "half", rope_scale: float = 1.0,
                 dev_err=None, stream=None):
    """``pa_append`` into the 8-bit cache: e4m3 codes and one power-of-two
    scale per (block, KV head), older codes of a block following a scale
    that grows.  Returns ``q_out``."""
    _check_q8(k_cache, v_cache, k_scales, v_scales)
    return _append(_lib.load().pa_append_q8, "pa_append_q8", q_out, k_cache,
                   v_cache, ((k_scales, "k_scales"), (v_scales, "v_scales")),
                   q, k, v, block_tables, context_lens, query_start,
                   max_q_len, q_norm, k_norm, norm_eps, rope_freqs,
                   rope_layout, rope_scale, dev_err, stream)


def _attend_q8_ptrs(out, q, k_cache, v_cache, k_scales, v_scales,
                    block_tables, context_lens, workspace, dev_err):
    """(device, the eight tensors' pointers, workspace, dev_err)."""
    tc = _tc
    _check_q8(k_cache, v_cache, k_scales, v_scales)
    if out.shape != q.shape:
        raise ValueError("q and out disagree on shape")
    if context_lens.shape != block_tables.shape[:1]:
        raise ValueError("context_lens must be [num_seqs]")
    e4m3, f32, i32 = tc["e4m3"], tc["f32"], tc["i32"]
    dev = tc["device"]()
    return (dev, _ptr(out, "out", dev), _ptr(q, "q", dev),
            _ptr(k_cache, "k_cache", dev, e4m3),
            _ptr(v_cache, "v_cache", dev, e4m3),
            _ptr(k_scales, "k_scales", dev, f32),
            _ptr(v_scales, "v_scales", dev, f32),
            _ptr(block_tables, "block_tables", dev, i32),
            _ptr(context_lens, "context_lens", dev, i32),
            _ptr(workspace, "workspace", dev), _ptr(dev_err, "dev_err", dev,
                                                    i32))


def pa_decode_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables,
                 context_lens, scale: float, *, partition_size: int = 0,
                 max_context_len: int = 0, reduce: str = "auto",
                 workspace=None, dev_err=None, stream=None,
                 desc: pa_decode_desc | None = None):
    """``pa_decode`` over the 8-bit cache.  ``workspace`` (a uint8 CUDA
    tensor of ``pa_decode_workspace_bytes`` bytes) is allocated per call when
    not given.  Returns ``out``."""
    lib = _lib.load()
    _tc or _torch_refs()
    if desc is None:
        desc = make_desc(q, k_cache, block_tables,
                         partition_size=partition_size,
                         max_context_len=max_context_len, reduce=reduce)
    elif ((desc.num_seqs, desc.num_q_heads, desc.head_dim) != q.shape or
          (desc.num_seqs, desc.max_blocks_per_seq) != block_tables.shape or
          (desc.num_blocks, desc.num_kv_heads, desc.block_size,
           desc.head_dim) != k_cache.shape or desc.dtype != _code(q.dtype)):
        raise ValueError("desc does not describe q, k_cache and block_tables")
    _out_mode(desc, out, q.dtype)
    if workspace is None:
        workspace = _workspace(
            int(lib.pa_decode_workspace_bytes(ctypes.byref(desc))), q.device,
            stream)
    dev, *p = _attend_q8_ptrs(out, q, k_cache, v_cache, k_scales, v_scales,
                              block_tables, context_lens, workspace, dev_err)
    st = lib.pa_decode_q8(*p[:8], scale, ctypes.byref(desc), p[8],
                          workspace.nbytes, p[9], _stream_on(stream, dev))
    if st:
        _lib.check(st, "pa_decode_q8")
    return out


def pa_prefill_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables,
                  context_lens, query_start, scale: float, *, max_q_len: int,
                  max_context_len: int = 0, workspace=None, dev_err=None,
                  stream=None):
    """``pa_prefill`` over the 8-bit cache.  ``workspace`` (a uint8 CUDA
    tensor of ``pa_prefill_workspace_bytes`` bytes) is allocated per call
    when not given.  Returns ``out``."""
    lib = _lib.load()
    _tc or _torch_refs()
    if query_start.shape != (block_tables.shape[0] + 1,):
        raise ValueError("query_start must be [num_seqs + 1]")
    desc = _prefill_desc(q, k_cache, block_tables, max_q_len,
                         max_context_len)
    _out_mode(desc, out, q.dtype)
    if workspace is None:
        workspace = _workspace(
            lib.pa_prefill_workspace_bytes(ctypes.byref(desc)), q.device,
            stream)
    dev, *p = _attend_q8_ptrs(out, q, k_cache, v_cache, k_scales, v_scales,
                              block_tables, context_lens, workspace, dev_err)
    st = lib.pa_prefill_q8(
        *p[:8], _ptr(query_start, "query_start", dev, _tc["i32"]), scale,
        ctypes.byref(desc), p[8], workspace.nbytes, p[9],
        _stream_on(stream, dev))
    if st:
        _lib.check(st, "pa_prefill_q8")
    return out


def pa_copy_blocks_q8(k_cache, v_cache, k_scales, v_scales, pairs, *,
                      dev_err=None, stream=None):
    """``pa_copy_blocks`` for the 8-bit cache: codes and scales of block
    pairs[i, 0] into block pairs[i, 1]."""
    tc = _tc or _torch_refs()
    nb, hkv, bs, d = _check_q8(k_cache, v_cache, k_scales, v_scales)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [num_pairs, 2]")
    e4m3, f32, i32 = tc["e4m3"], tc["f32"], tc["i32"]
    dev = tc["device"]()
    st = _lib.load().pa_copy_blocks_q8(
        _ptr(k_cache, "k_cache", dev, e4m3),
        _ptr(v_cache, "v_cache", dev, e4m3),
        _ptr(k_scales, "k_scales", dev, f32),
        _ptr(v_scales, "v_scales", dev, f32), _ptr(pairs, "pairs", dev, i32),
        pairs.shape[0], hkv, d, bs, nb, _ptr(dev_err, "dev_err", dev, i32),
        _stream_on(stream, dev))
    if st:
        _lib.check(st, "pa_copy_blocks_q8")


def pa_swap_blocks_q8(dst_k, dst_v, dst_k_scales, dst_v_scales, src_k, src_v,
                      src_k_scales, src_v_scales, pairs, *, dev_err=None,
                      stream=None):
    """``pa_swap_blocks`` for the 8-bit cache (codes and scales); any pool
    (and ``pairs``) may be pinned CPU tensors."""
    import torch
    ns, hkv, bs, d = _check_q8(src_k, src_v, src_k_scales, src_v_scales,
                               ("src ", ""))
    nd, *rest = _check_q8(dst_k, dst_v, dst_k_scales, dst_v_scales,
                          ("dst ", ""))
    if tuple(rest) != (hkv, bs, d):
        raise ValueError("the pools' blocks differ in shape")
    if pairs.ndim != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    st = _lib.load().pa_swap_blocks_q8(
        _reachable(dst_k, "dst_k", e4m3), _reachable(dst_v, "dst_v", e4m3),
        _reachable(dst_k_scales, "dst_k_scales", f32),
        _reachable(dst_v_scales, "dst_v_scales", f32),
        _reachable(src_k, "src_k", e4m3), _reachable(src_v, "src_v", e4m3),
        _reachable(src_k_scales, "src_k_scales", f32),
        _reachable(src_v_scales, "src_v_scales", f32),
        _reachable(pairs, "pairs", torch.int32), pairs.shape[0], hkv, d, bs,
        ns, nd, _dev(dev_err, "dev_err", torch.int32), _stream(stream))
    _lib.check(st, "pa_swap_blocks_q8")


def pa_pool_blocks_q8(nbytes: int, num_layers: int, num_kv_heads: int,
                      head_dim: int, block_size: int) -> int:
    """``pa_pool_blocks`` for the 8-bit cache (codes and scales)."""
    n = _lib.load().pa_pool_blocks_q8(int(nbytes), num_layers, num_kv_heads,
                                      head_dim, block_size)
    if n < 0:
        _lib.check(_lib.PA_ERR_INVALID_ARG, "pa_pool_blocks_q8")
    return n


class BlockManager:
    """Host block manager of libpagedkv (pa_bm_* calls).

    Free pool, per-sequence block tables, reference counts, fork and
    copy-on-write.  Not thread-safe.
    """

    def __init__(self, num_blocks: int, block_size: int, free_order=None):
        self._lib = _lib.load()
        self.num_blocks = num_blocks
        self.block_size = block_size
        handle = ctypes.c_void_p()
        order = None
        if free_order is not None:
            import numpy as np
            arr = np.ascontiguousarray(free_order, dtype=np.int32)
            if arr.shape != (num_blocks,):
                raise ValueError("free_order must have num_blocks entries")
            order = arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _lib.check(self._lib.pa_bm_create(num_blocks, block_size, order,
                                          ctypes.byref(handle)),
                   "pa_bm_create")
        self._h = handle

    def close(self):
        if self._h:
            self._lib.pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id: int):
        _lib.check(self._lib.pa_bm_add_seq(self._h, seq_id), "pa_bm_add_seq")

    def fork(self, parent: int, child: int):
        _lib.check(self._lib.pa_bm_fork(self._h, parent, child), "pa_bm_fork")

    def append(self, seq_id: int, n_tokens: int):
        """Returns (slots int64 ndarray [n_tokens], cow_pairs int32 [k, 2])."""
        import numpy as np
        slots = np.empty(max(n_tokens, 0), dtype=np.int64)
        pairs = np.empty(2, dtype=np.int32)
        ncow = ctypes.c_int(0)
        st = self._lib.pa_bm_append(
            self._h, seq_id, n_tokens,
            slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            pairs.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), 1,
            ctypes.byref(ncow))
        _lib.check(st, "pa_bm_append")
        return slots, pairs[: 2 * ncow.value].reshape(-1, 2).copy()

    def append_batch(self, seq_ids, n_tokens, slots_out=None):
        """One call for a whole decode step: appends n_tokens[i] tokens to
        seq_ids[i].  Returns (slots int64 [sum], cow_pairs int32 [k, 2]).
        ``slots_out`` (optional int64 ndarray, e.g. a view of pinned memory)
        receives the slots.  Raises NoFreeBlocksError (with .num_done) if the
        pool runs out."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        nt = np.ascontiguousarray(n_tokens, dtype=np.int32)
        if nt.shape != ids.shape:
            raise ValueError("seq_ids and n_tokens differ in length")
        total = int(nt.sum())
        if slots_out is not None:
            if (slots_out.dtype != np.int64 or slots_out.shape != (total,)
                    or not slots_out.flags.c_contiguous):
                raise ValueError("slots_out must be contiguous int64 [sum]")
            slots = slots_out
        else:
            slots = np.empty(total, dtype=np.int64)
        pairs = np.empty(2 * max(len(ids), 1), dtype=np.int32)
        ncow, ndone = ctypes.c_int(0), ctypes.c_int(0)
        st = self._lib.pa_bm_append_batch(
            self._h, ids.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            nt.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(ids),
            slots.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            pairs.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), len(ids),
            ctypes.byref(ncow), ctypes.byref(ndone))
        try:
            _lib.check(st, "pa_bm_append_batch")
        except PagedKVError as e:
            e.num_done = ndone.value
            raise
        return slots, pairs[: 2 * ncow.value].reshape(-1, 2).copy()

    def free_seq(self, seq_id: int):
        _lib.check(self._lib.pa_bm_free_seq(self._h, seq_id), "pa_bm_free_seq")

    def truncate(self, seq_id: int, new_len: int):
        _lib.check(self._lib.pa_bm_truncate(self._h, seq_id, new_len),
                   "pa_bm_truncate")

    def block_table(self, seq_ids, max_blocks: int, table_out=None,
                    lens_out=None):
        """Returns (table int32 [n, max_blocks] padded with -1, lens int32).
        Optional contiguous int32 ``table_out`` / ``lens_out`` arrays receive
        the result in place."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        table = table_out if table_out is not None else \
            np.empty((len(ids), max_blocks), dtype=np.int32)
        lens = lens_out if lens_out is not None else \
            np.empty(len(ids), dtype=np.int32)
        for arr, shp in ((table, (len(ids), max_blocks)), (lens, (len(ids),))):
            if (arr.dtype != np.int32 or arr.shape != shp
                    or not arr.flags.c_contiguous):
                raise ValueError("block_table outputs: wrong dtype/shape")
        st = self._lib.pa_bm_block_table(
            self._h, ids.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
            len(ids), max_blocks,
            table.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            lens.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
        _lib.check(st, "pa_bm_block_table")
        return table, lens

    def num_free(self) -> int:
        return self._lib.pa_bm_num_free(self._h)

    def num_used(self) -> int:
        return self._lib.pa_bm_num_used(self._h)

    def refcount(self, block: int) -> int:
        return self._lib.pa_bm_refcount(self._h, block)

    def seq_len(self, seq_id: int) -> int:
        return self._lib.pa_bm_seq_len(self._h, seq_id)

    def num_seq_blocks(self, seq_id: int) -> int:
        return self._lib.pa_bm_num_seq_blocks(self._h, seq_id)

    # -- prefix cache -------------------------------------------------------
    def match_prefix(self, seq_id: int, tokens) -> int:
        """Attach the longest cached run of full blocks that starts
        ``tokens`` to the new, empty ``seq_id``; returns the tokens matched
        (only the rest needs a prefill)."""
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        out = ctypes.c_int64(0)
        _lib.check(self._lib.pa_bm_match_prefix(
            self._h, seq_id, t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            len(t), ctypes.byref(out)), "pa_bm_match_prefix")
        return out.value

    def cache_insert(self, seq_id: int, tokens):
        """Cache the full blocks of the first len(tokens) tokens of
        ``seq_id`` (call once their K/V are written)."""
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        _lib.check(self._lib.pa_bm_cache_insert(
            self._h, seq_id, t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            len(t)), "pa_bm_cache_insert")

    def cache_evict(self, max_blocks: int) -> int:
        out = ctypes.c_int(0)
        _lib.check(self._lib.pa_bm_cache_evict(self._h, max_blocks,
                                               ctypes.byref(out)),
                   "pa_bm_cache_evict")
        return out.value

    def num_cached(self) -> int:
        return self._lib.pa_bm_num_cached(self._h)

    def cache_nodes(self):
        """The cached tree as (parent_index int32 [n], block int32 [n],
        tokens int32 [n, block_size]), parents before children."""
        import numpy as np
        n = max(self.num_cached(), 0)
        parent = np.empty(max(n, 1), dtype=np.int32)
        block = np.empty(max(n, 1), dtype=np.int32)
        toks = np.empty((max(n, 1), self.block_size), dtype=np.int32)
        got = ctypes.c_int(0)
        p32 = ctypes.POINTER(ctypes.c_int32)
        _lib.check(self._lib.pa_bm_cache_nodes(
            self._h, n, parent.ctypes.data_as(p32), block.ctypes.data_as(p32),
            toks.ctypes.data_as(p32), ctypes.byref(got)), "pa_bm_cache_nodes")
        k = got.value
        return parent[:k], block[:k], toks[:k]

    def cached_paths(self):
        """Every cached block as the tuple of its token keys from the root
        (the same form as the oracle model's ``cached_paths``)."""
        parent, _, toks = self.cache_nodes()
        paths = []
        for i in range(len(parent)):
            key = tuple(int(t) for t in toks[i])
            paths.append((key,) if parent[i] < 0 else paths[parent[i]] + (key,))
        return set(paths)

    # -- swapping to a host pool ------------------------------------------------
    def set_host_blocks(self, num_host_blocks: int):
        _lib.check(self._lib.pa_bm_set_host_blocks(self._h, num_host_blocks),
                   "pa_bm_set_host_blocks")
        self.num_host_blocks = num_host_blocks

    def _swap(self, fn, name, seq_ids, pairs_out):
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        cap = sum(max(self.num_seq_blocks(int(s)), 0) for s in ids)
        if pairs_out is None:
            pairs = np.empty((max(cap, 1), 2), dtype=np.int32)
        else:
            if (pairs_out.dtype != np.int32 or pairs_out.ndim != 2
                    or pairs_out.shape[1] != 2
                    or not pairs_out.flags.c_contiguous):
                raise ValueError("pairs_out must be contiguous int32 [k, 2]")
            pairs, cap = pairs_out, pairs_out.shape[0]
        n = ctypes.c_int(0)
        _lib.check(fn(self._h, ids.ctypes.data_as(ctypes.POINTER(
            ctypes.c_int64)), len(ids), pairs.ctypes.data_as(
                ctypes.POINTER(ctypes.c_int32)), cap, ctypes.byref(n)), name)
        return pairs[:n.value]

    def swap_out(self, seq_ids, pairs_out=None):
        """Swap the group out; returns (device, host) block pairs int32
        [k, 2] (a view of ``pairs_out`` if given, e.g. pinned memory)."""
        return self._swap(self._lib.pa_bm_swap_out, "pa_bm_swap_out",
                          seq_ids, pairs_out)

    def swap_in(self, seq_ids, pairs_out=None):
        """Swap the group back in; returns (host, device) block pairs."""
        return self._swap(self._lib.pa_bm_swap_in, "pa_bm_swap_in", seq_ids,
                          pairs_out)

    def num_free_host(self) -> int:
        return self._lib.pa_bm_num_free_host(self._h)

    def host_refcount(self, block: int) -> int:
        return self._lib.pa_bm_host_refcount(self._h, block)

    def is_swapped(self, seq_id: int) -> bool:
        r = self._lib.pa_bm_is_swapped(self._h, seq_id)
        if r < 0:
            raise KeyError(seq_id)
        return bool(r)

    def seq_blocks(self, seq_id: int):
        """Table entries in logical order (host ids while swapped out)."""
        import numpy as np
        n = max(self.num_seq_blocks(seq_id), 0)
        out = np.empty(max(n, 1), dtype=np.int32)
        got = ctypes.c_int(0)
        _lib.check(self._lib.pa_bm_seq_blocks(
            self._h, seq_id, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            n, ctypes.byref(got)), "pa_bm_seq_blocks")
        return out[:got.value]
