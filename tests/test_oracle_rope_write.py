"""Pins of the rotary-write oracle (oracle/rope_write_ref.py) against closed forms,
invariants and the RoPE of the MLA oracle."""
import numpy as np
import pytest

from oracle import fp8_ref, mla_write_ref as mw
from oracle import rope_write_ref as rw


def _table(max_pos, rope_dim, base=10000.0):
    freq = base ** (-np.arange(rope_dim // 2) * 2.0 / rope_dim)
    angle = np.arange(max_pos)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1)


def test_one_axis_equals_the_rotate_half_formula():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((9, 3, 64))
    table = _table(50, 64)
    pos = rng.integers(0, 50, (1, 9))
    cos = np.concatenate([table[pos[0], :32]] * 2, axis=1)
    sin = np.concatenate([table[pos[0], 32:]] * 2, axis=1)
    for h in range(3):
        np.testing.assert_allclose(rw.rotate_rows(x, table, pos)[:, h],
                                   mw.rope_rotate_half(x[:, h], cos, sin), rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_pair_norms_and_composes(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 48))
    table = _table(40, 32)
    pos = rng.integers(0, 20, (1, 5))
    y = rw.rotate_rows(x, table, pos, interleaved=interleaved)
    assert np.array_equal(y[..., 32:], x[..., 32:])  # elements past rope_dim pass through
    pair = (lambda z: (z[..., 0:32:2], z[..., 1:32:2])) if interleaved else \
        (lambda z: (z[..., :16], z[..., 16:32]))
    np.testing.assert_allclose(np.hypot(*pair(y)), np.hypot(*pair(x)), rtol=1e-13)
    # Position p, then position r, is position p + r.
    again = rw.rotate_rows(y, table, np.full((1, 5), 3), interleaved=interleaved)
    np.testing.assert_allclose(again, rw.rotate_rows(x, table, pos + 3, interleaved=interleaved),
                               rtol=1e-12, atol=1e-13)


def test_interleaved_is_a_permutation_of_rotate_half():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 32))
    table, pos = _table(30, 32), rng.integers(0, 30, (1, 4))
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    a = rw.rotate_rows(x, table, pos, interleaved=True)[..., perm]
    b = rw.rotate_rows(x[..., perm], table, pos)
    assert np.array_equal(a, b)


def test_each_pair_follows_its_own_axis():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 1, 16))
    table = _table(30, 16)
    axis = np.array([0, 1, 2, 0, 1, 2, 2, 1])
    pos = rng.integers(0, 30, (3, 6))
    y = rw.rotate_rows(x, table, pos, axis)
    for i, a in enumerate(axis):
        one = rw.rotate_rows(x, table, pos[a:a + 1])
        assert np.array_equal(y[..., [i, i + 8]], one[..., [i, i + 8]])
    same = np.repeat(pos[:1], 3, axis=0)  # equal positions on every axis: the one-axis form
    assert np.array_equal(rw.rotate_rows(x, table, same, axis), rw.rotate_rows(x, table, pos[:1]))


def test_magnitude_bounds_the_rotation():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 16))
    table, pos = _table(9, 16), rng.integers(0, 9, (1, 3))
    m = rw.rotate_magnitude(x, table, pos)
    assert (np.abs(rw.rotate_rows(x, table, pos)) <= m * (1 + 1e-15)).all()
    assert (m <= np.sqrt(2) * np.hypot(x[..., :8], x[..., 8:]).repeat(2, axis=0).max()).all()


def test_read_fp8_inverts_the_quantising_layout():
    rng = np.random.default_rng(6)
    codes = rng.integers(0, 256, (3, 4, 2, 128), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = rng.random((3, 2, 4)).astype(np.float32)
    out = rw.read_fp8(codes, scales, np.array([5, -1, 0, 11]))
    assert (out[1] == 0).all()
    for t, (b, o) in ((0, (1, 1)), (2, (0, 0)), (3, (2, 3))):
        for h in range(2):
            want = fp8_ref.e4m3_decode(codes[b, o, h]) * float(scales[b, h, o])
            assert np.array_equal(out[t, h], want)
