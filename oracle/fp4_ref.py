"""Oracle for the 4-bit KV cache: E2M1 codes with one scale byte per 16 values.

TEST INFRASTRUCTURE. Only tests/ and ``__graft_entry__.smoke()`` may import this module; the
product library never does. numpy, written from the format's definition:

* "KV Cache 笔记" (Quantized: KIVI-style 4-bit grouped quantisation, the warning that a
  separate dequantisation per layer and step can eat the bandwidth it saves).
* E2M1 (OCP 4-bit floating point): 1 sign bit, 2 exponent bits with bias 1, 1 fraction bit:
  magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
* A scale byte holds 5 bits of exponent (bias 15) and 3 of fraction, exponent 0 subnormal: the
  upper 8 of an fp16's 15 magnitude bits. 0xE2 = 10240 is the largest used, 0xFF marks NaN.

Readings (the pages fix no format):

* scale = the scale value nearest to amax / 6 of the 16 values, ties to the even byte, at most
  10240; code = the E2M1 value nearest to x / scale, ties to the even code, saturating at 6.
  Every comparison is between exactly represented float64 numbers: amax and x are bf16, a
  border between scales times 6 has 7 bits, a border between codes times a scale 7 bits.
* 16 values with an infinity or a NaN: scale byte 0xFF, codes 0; they read back as NaN.
"""
from __future__ import annotations

import numpy as np

CODE_VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
MAX_SCALE, NAN_SCALE = 0xE2, 0xFF


def scale_values(u) -> np.ndarray:
    """float64 values of scale bytes (0xF8 and above: NaN, as fp16 has it, 0xF8 infinite)."""
    u = np.asarray(u, dtype=np.int64)
    e, f = u >> 3, u & 7
    val = np.where(e == 0, f * 2.0 ** -17, (1 + f / 8.0) * np.exp2(e - 15.0))
    return np.where(e == 31, np.where(f == 0, np.inf, np.nan), val)


_SCALES = scale_values(np.arange(MAX_SCALE + 1))


def _nearest_even(x, grid):
    """Index of the entry of ascending `grid` nearest to each x >= 0, ties to the even index,
    past the last entry the last."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    twice = 2 * x - (grid[hi - 1] + grid[hi])  # exact: few bits on either side
    return np.where((twice > 0) | ((twice == 0) & (hi % 2 == 0)), hi, hi - 1)


def quantise(rows):
    """(codes [..., 64], scales [..., 8]) uint8 of float64 rows [..., 128] holding bf16 values."""
    g = np.asarray(rows, dtype=np.float64)
    g = g.reshape(g.shape[:-1] + (8, 16))
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    amax = np.abs(g).max(-1)
    # Borders of amax itself, 6 times those of the scales: no quotient is formed.
    u = _nearest_even(amax, 6 * _SCALES)
    s = _SCALES[u][..., None]
    code = np.zeros(g.shape, dtype=np.int64)
    mag = np.abs(g)
    for i in range(1, 8):
        border = (CODE_VALUES[i - 1] + CODE_VALUES[i]) / 2 * s
        code += np.where(s > 0, (mag > border) | ((mag == border) & (i % 2 == 0)), False)
    code |= np.where(np.signbit(g) & (s > 0), 8, 0)
    code = code.reshape(code.shape[:-2] + (128,))
    packed = code[..., 0::2] | code[..., 1::2] << 4
    return packed.astype(np.uint8), np.where(finite, u, NAN_SCALE).astype(np.uint8)


def dequantise(codes, scales) -> np.ndarray:
    """float64 [..., 128] of codes [..., 64] and scales [..., 8]."""
    c = np.asarray(codes, dtype=np.int64)
    nib = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (128,))
    val = np.where(nib & 8, -1.0, 1.0) * CODE_VALUES[nib & 7]
    s = np.repeat(scale_values(scales), 16, -1)
    with np.errstate(invalid="ignore"):
        return val * s


def cache_write(codes, scales, rows, slots):
    """The caches (codes [nb, H_kv, bs, 64], scales [.., 8]) after rows [T, H_kv, 128] went to
    `slots`; negative slots and those past the cache are skipped."""
    codes, scales = codes.copy(), scales.copy()
    nb, _, bs, _ = codes.shape
    q, s = quantise(rows)
    for t, slot in enumerate(slots):
        if 0 <= slot < nb * bs:
            codes[slot // bs, :, slot % bs], scales[slot // bs, :, slot % bs] = q[t], s[t]
    return codes, scales


def dequantise_cache(codes, scales) -> np.ndarray:
    """float64 [nb, bs, H_kv, 128], the layout of the bf16 caches."""
    return np.ascontiguousarray(dequantise(codes, scales).transpose(0, 2, 1, 3))
