"""Oracle for the fused rotary embedding + paged write of GQA caches, and for reading an
FP8 cache back.

TEST INFRASTRUCTURE. Only tests/, ``__graft_entry__.smoke()`` and bench.py's
cpu_baseline / reference leg may import this module; the product library never
does. float64 numpy, written from the pages:

* "KV Cache 笔记", the Llama attention forward: q and k take
  ``x * cos + rotate_half(x) * sin`` before the cache write.
* "KVCache 优化技能" 模式二 and §3.1: the write through slot_mapping.

Readings (the pages do not fix them):

* Pair i of a head turns by the angle of the position on its own axis, pair_axis[i]; the
  cosine and sine of position p are table[p][i] and table[p][rope_dim / 2 + i].
* A pair is the elements i and i + rope_dim / 2 (rotate_half) or 2i and 2i + 1
  (interleaved); elements from rope_dim on pass through.
"""
from __future__ import annotations

import numpy as np

from .fp8_ref import e4m3_decode


def rotate_rows(x, table, positions, pair_axis=None, interleaved=False) -> np.ndarray:
    """Rotary embedding of x [T, heads, d] in float64.

    table [max_pos, rope_dim]; positions [axes, T]; pair_axis [rope_dim / 2]."""
    y = np.array(x, dtype=np.float64)
    table = np.asarray(table, dtype=np.float64)
    pairs = table.shape[1] // 2
    axis = np.zeros(pairs, dtype=np.int64) if pair_axis is None else np.asarray(pair_axis)
    for i in range(pairs):
        p = np.asarray(positions)[axis[i]]
        c, s = table[p, i][:, None], table[p, pairs + i][:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        xa, xb = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a] = xa * c - xb * s
        y[:, :, b] = xb * c + xa * s
    return y


def rotate_magnitude(x, table, positions, pair_axis=None, interleaved=False) -> np.ndarray:
    """|x1 c| + |x2 s| (and |x2 c| + |x1 s|) of every rotated element, |x| of the others: what
    the rounding errors of a rotation in a shorter format are relative to."""
    y = np.abs(np.array(x, dtype=np.float64))
    table = np.abs(np.asarray(table, dtype=np.float64))
    pairs = table.shape[1] // 2
    axis = np.zeros(pairs, dtype=np.int64) if pair_axis is None else np.asarray(pair_axis)
    for i in range(pairs):
        p = np.asarray(positions)[axis[i]]
        c, s = table[p, i][:, None], table[p, pairs + i][:, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        xa, xb = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a] = xa * c + xb * s
        y[:, :, b] = xb * c + xa * s
    return y


def read_fp8(codes, scales, slots) -> np.ndarray:
    """code * scale of the rows at `slots` in float64, [T, H_kv, d]; zeros where negative.

    codes [nb, bs, H_kv, d] uint8, scales [nb, H_kv, bs] float32."""
    nb, bs, hkv, d = codes.shape
    slots = np.asarray(slots)
    out = np.zeros((len(slots), hkv, d))
    for t, slot in enumerate(slots):
        if slot >= 0:
            blk, off = divmod(int(slot), bs)
            out[t] = e4m3_decode(codes[blk, off]) * scales[blk, :, off].astype(np.float64)[:, None]
    return out
