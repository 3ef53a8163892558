"""Pins of the 4-bit cache oracle: by hand, by exhaustive search over codes and scales, and
against fractions (no floating point at all)."""
from fractions import Fraction

import numpy as np
import torch

from oracle import fp4_ref as f4


def bf16(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy()


def test_scale_bytes_are_the_upper_bits_of_fp16():
    u = np.arange(256, dtype=np.uint16)
    want = (u << 7).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(f4.scale_values(u), want)
    assert f4.scale_values(f4.MAX_SCALE) == 10240
    assert 6 * 10240 <= float(np.finfo(np.float16).max) < 6 * 11264


def test_a_row_by_hand():
    x = np.zeros((1, 128))
    x[0, :16] = [6, -4, 3, 2, 1.5, 1, 0.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.2, 0]
    x[0, 16:32] = 12.0
    codes, scales = f4.quantise(x)
    assert scales[0, 0] == 15 << 3 and scales[0, 1] == 16 << 3 and not scales[0, 2:].any()
    nib = np.stack([codes[0] & 15, codes[0] >> 4], -1).reshape(-1)
    # Ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4.
    assert nib[:16].tolist() == [7, 8 | 6, 5, 4, 3, 2, 1, 0, 2, 2, 4, 4, 6, 6, 8, 0]
    assert nib[16:32].tolist() == [7] * 16 and not nib[32:].any()
    back = f4.dequantise(codes, scales)[0]
    assert back[:14].tolist() == [6, -4, 3, 2, 1.5, 1, 0.5, 0, 1, 1, 2, 2, 4, 4] and back[16] == 12


def test_nearest_scale_and_code_by_search():
    """Every group against a search over all scales and codes in exact fractions."""
    rng = np.random.default_rng(4)
    rows = bf16(rng.standard_normal((40, 128)) * np.exp2(rng.integers(-22, 20, (40, 1))))
    rows[3, :16] = bf16(np.exp2(-20) * np.arange(16))
    codes, scales = f4.quantise(rows)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(40, 8, 16)
    grid = [Fraction(float(v)) for v in f4.scale_values(np.arange(f4.MAX_SCALE + 1))]
    for r in range(40):
        for g in range(8):
            x = [Fraction(float(v)) for v in rows[r, 16 * g:16 * g + 16]]
            want = min(range(len(grid)), key=lambda u: (abs(grid[u] - max(map(abs, x)) / 6), u % 2))
            assert scales[r, g] == want
            if not want:
                assert not nib[r, g].any()
                continue
            for v, c in zip(x, nib[r, g]):
                d = [abs(abs(v) - Fraction(float(m)) * grid[want]) for m in f4.CODE_VALUES]
                assert (c & 7) == min(range(8), key=lambda i: (d[i], i % 2))
                assert bool(c & 8) == (v < 0)


def test_values_survive_a_second_rounding():
    rng = np.random.default_rng(5)
    rows = bf16(rng.standard_normal((50, 128)))
    codes, scales = f4.quantise(rows)
    back = f4.dequantise(codes, scales)
    np.testing.assert_array_equal(bf16(back), back)                          # exact in bf16
    np.testing.assert_array_equal(back.astype(np.float16).astype(float), back)  # and in fp16
    again = f4.dequantise(*f4.quantise(back))
    amax = np.abs(rows.reshape(50, 8, 16)).max(-1).repeat(16, -1)
    # Half a step of the widest interval is 1/6 of 6 scales, the scale itself is off by 2^-4.
    assert (np.abs(back - rows) <= amax / 6 * (1 + 2.0 ** -4)).all()
    assert (np.abs(again - back) <= amax / 6 * (1 + 2.0 ** -4)).all()


def test_infinities_nan_and_the_ends_of_the_range():
    x = np.ones((1, 128))
    x[0, 5], x[0, 20], x[0, 33] = np.inf, np.nan, -np.inf
    x[0, 48:64] = bf16(3e38)
    x[0, 64:80] = 6 * 2.0 ** -18       # rounds to even: scale 0
    x[0, 80:96] = bf16(6.1 * 2.0 ** -18)
    codes, scales = f4.quantise(x)
    assert (scales[0, :3] == 0xFF).all() and not codes[0, :24].any()
    back = f4.dequantise(codes, scales)[0]
    assert np.isnan(back[:48]).all()
    assert (back[48:64] == 61440).all() and (back[64:80] == 0).all()
    assert scales[0, 5] == 1 and (back[80:96] == 3 * 2.0 ** -17).all()


def test_cache_write_layout():
    rng = np.random.default_rng(6)
    rows = bf16(rng.standard_normal((4, 3, 128)))
    codes, scales = np.full((2, 3, 8, 64), 7, np.uint8), np.full((2, 3, 8, 8), 9, np.uint8)
    c, s = f4.cache_write(codes, scales, rows, [9, -1, 0, 16])
    q, qs = f4.quantise(rows)
    np.testing.assert_array_equal(c[1, :, 1], q[0])
    np.testing.assert_array_equal(s[0, :, 0], qs[2])
    c[1, :, 1], c[0, :, 0] = 7, 7
    assert (c == 7).all()
    np.testing.assert_array_equal(f4.dequantise_cache(*f4.cache_write(codes, scales, rows, [9] * 1))[1, 1],
                                  f4.dequantise(q, qs)[0])
