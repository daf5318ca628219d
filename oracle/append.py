"""fp64 oracle for appending tokens: norm, position rotation, the paged write,
and the 8-bit cache's quantisation.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Plain numpy, one token and one block at a time, from the formulas that
``pagedkv.h`` states for ``pa_append`` and ``pa_append_q8``.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes (4 exponent bits, bias 7; 3
    fraction bits; all ones is NaN)."""
    out = np.empty(256)
    for c in range(256):
        s = -1.0 if c & 0x80 else 1.0
        e, f = (c >> 3) & 15, c & 7
        if e == 15 and f == 7:
            out[c] = math.nan
        elif e == 0:
            out[c] = s * f * 2.0 ** -9
        else:
            out[c] = s * (1 + f / 8) * 2.0 ** (e - 7)
    return out


def e4m3_step(x) -> np.ndarray:
    """The distance between e4m3 values around |x|."""
    _, e = np.frexp(np.abs(np.asarray(x, dtype=np.float64)))
    return 2.0 ** (np.maximum(e - 1, -6) - 3)


def e4m3_round(x) -> np.ndarray:
    """Nearest e4m3 value, ties to even, magnitudes past 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    s = e4m3_step(np.clip(x, -E4M3_MAX, E4M3_MAX))
    return np.clip(np.round(np.clip(x, -1e300, 1e300) / s) * s, -E4M3_MAX,
                   E4M3_MAX)


def norm_head(x, weight, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    ms = np.mean(x * x, axis=-1, keepdims=True)
    return np.asarray(weight, dtype=np.float64) * x / np.sqrt(ms + eps)


def rotate_head(x, pos: int, freqs, layout: str, scale: float) -> np.ndarray:
    """x [..., head_dim] at position pos; freqs [rot_dim / 2]."""
    x = np.array(x, dtype=np.float64)
    if freqs is None:
        return x
    r = 2 * len(freqs)
    for j, f in enumerate(freqs):
        a, b = (j, j + r // 2) if layout == "half" else (2 * j, 2 * j + 1)
        # reduced to one turn (the float64 product is off by pos f 2^-53)
        ang = math.fmod(pos * float(f), 2 * math.pi)
        c, s = scale * math.cos(ang), scale * math.sin(ang)
        u, w = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


def scale_for(amax: float) -> float:
    """The smallest power of two s in [2^-64, 2^120] with amax <= 448 s."""
    e = -64
    while e < 120 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def placed(context_lens, query_start, block_tables, block_size: int):
    """(sequence, row, position, block, slot) of every new token."""
    for b, L in enumerate(context_lens):
        q0, q1 = ((int(query_start[b]), int(query_start[b + 1]))
                  if query_start is not None else (b, b + 1))
        if L == 0:
            continue
        for row in range(q0, q1):
            p = int(L) - (q1 - q0) + row - q0
            yield (b, row, p, int(block_tables[b][p // block_size]),
                   p % block_size)


def append_q8(codes, scales, new, places):
    """codes [num_blocks, H, bs, D] (values), scales [num_blocks, H]; new
    [rows, H, D]; places as from ``placed``.  Returns (codes as unrounded
    values in units of the new scale, new scales, written [num_blocks, bs])."""
    codes = np.array(codes, dtype=np.float64)
    scales = np.array(scales, dtype=np.float64)
    written = np.zeros((codes.shape[0], codes.shape[2]), dtype=bool)
    runs: dict = {}
    for _, row, _, blk, o in places:
        runs.setdefault(blk, []).append((o, row))
    for blk, items in runs.items():
        items.sort()
        first = items[0][0]
        for h in range(codes.shape[1]):
            x = np.stack([new[row, h] for _, row in items])
            finite = np.abs(x[~np.isnan(x)])
            need = scale_for(float(finite.max()) if finite.size else 0.0)
            s = max(scales[blk, h], need) if first > 0 else need
            if first > 0:
                codes[blk, h, :first] *= scales[blk, h] / s
            scales[blk, h] = s
            for (o, _), row in zip(items, x):
                codes[blk, h, o] = row / s
        for o, _ in items:
            written[blk, o] = True
    return codes, scales, written
