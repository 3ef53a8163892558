"""The rotary writes and the FP8 read refuse bad arguments before anything is launched
(through the C ABI, no GPU: the pointers are never read)."""
import numpy as np
import pytest

from paged_kv_cache_77_gb300._lib import load

P = 1 << 20  # a 16-byte aligned address that nothing reads


def _args(**kw):
    a = dict(k_cache=P, v_cache=2 * P, q_out=3 * P, q_out_stride=512, q=4 * P, q_stride=512, k=5 * P,
             k_stride=256, v=6 * P, v_stride=256, table=7 * P, max_pos=100, rope_dim=128,
             positions=8 * P, num_axes=1, pair_axis=None, interleaved=0, slots=9 * P, num_tokens=5,
             num_blocks=10, block_size=128, H=4, H_kv=2, head_dim=128, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


BAD_AXIS = np.array([0, 1, 2, 3] * 16, dtype=np.int32)


@pytest.mark.parametrize("kw,code,word", [
    (dict(head_dim=120, q_stride=480), -2, b"head_dim"),
    (dict(head_dim=272), -2, b"head_dim"),
    (dict(rope_dim=144), -2, b"rope_dim"),
    (dict(rope_dim=24), -2, b"rope_dim"),
    (dict(num_axes=5), -2, b"axes"),
    (dict(num_axes=0), -2, b"axes"),
    (dict(max_pos=0), -1, b"size"),
    (dict(H=0), -1, b"size"),
    (dict(num_tokens=-1), -1, b"size"),
    (dict(num_blocks=1 << 26), -2, b"int32"),
    (dict(H=1 << 21), -2, b"heads"),
    (dict(q=None), -1, b"null"),
    (dict(table=None), -1, b"null"),
    (dict(slots=None), -1, b"null"),
    (dict(k=5 * P + 2), -1, b"aligned"),
    (dict(table=7 * P + 4), -1, b"aligned"),
    (dict(q_stride=516), -1, b"stride"),
    (dict(k_stride=-256), -1, b"stride"),
    (dict(q_out_stride=256), -1, b"stride"),
    (dict(q_out=4 * P + 16), -1, b"overlaps"),
    (dict(q_out=4 * P, q_out_stride=1024), -1, b"overlaps"),
    (dict(q_out=5 * P), -1, b"overlaps"),
    (dict(q_out=6 * P - 16), -1, b"overlaps"),
    (dict(pair_axis=BAD_AXIS.ctypes.data, num_axes=3), -1, b"pair_axis[3]"),
])
def test_rope_write_refusals(kw, code, word):
    lib = load()
    assert lib.pkv_rope_kv_cache_write(*_args(**kw)) == code
    assert word in lib.pkv_last_error()
    fp8 = _args(**kw)
    fp8[2:2] = [10 * P, 11 * P]
    assert lib.pkv_rope_kv_cache_write_fp8(*fp8) == code
    assert word in lib.pkv_last_error()


def test_rope_write_fp8_needs_its_scales_and_128_dims():
    lib = load()
    for scales, code in (((None, P), -1), ((P, P + 2), -1)):
        a = _args(num_tokens=0)
        a[2:2] = list(scales)
        assert lib.pkv_rope_kv_cache_write_fp8(*a) == code and b"scale" in lib.pkv_last_error()
    a = _args(head_dim=64, rope_dim=64, q_stride=256, q_out_stride=256)
    a[2:2] = [10 * P, 11 * P]
    assert lib.pkv_rope_kv_cache_write_fp8(*a) == -2 and b"head_dim" in lib.pkv_last_error()


def test_rows_of_one_projection_buffer_are_told_apart():
    """q_out in columns of the buffer that q, k and v do not use is accepted as far as the
    overlap check goes (the next check, pair_axis, is what refuses here)."""
    lib = load()
    bad = np.full(64, 7, dtype=np.int32)
    width = (4 + 2 + 2 + 4) * 128  # q | k | v | q_out
    same = dict(q=P, k=P + 1024, v=P + 1536, q_stride=width, k_stride=width, v_stride=width,
                pair_axis=bad.ctypes.data)
    for q_out, word in ((P + 2048, b"pair_axis"), (P, b"pair_axis"), (P + 2032, b"overlaps"),
                        (P + 512, b"overlaps")):
        rc = lib.pkv_rope_kv_cache_write(*_args(q_out=q_out, q_out_stride=width, **same))
        assert rc == -1 and word in lib.pkv_last_error(), q_out


def test_read_fp8_refusals():
    lib = load()

    def call(k=P, v=P, kc=P, vc=P, ks=P, vs=P, slots=P, T=4, nb=2, bs=128, hkv=2, d=128):
        return lib.pkv_kv_cache_read_fp8(k, v, kc, vc, ks, vs, slots, T, nb, bs, hkv, d, None, None)

    assert call(d=64) == -2 and b"head_dim" in lib.pkv_last_error()
    assert call(T=-1) == -1 and call(nb=0) == -1 and call(hkv=0) == -1
    assert call(k=None) == -1 and call(slots=None) == -1 and call(ks=None) == -1
    assert call(k=P + 8) == -1 and call(vs=P + 2) == -1 and b"aligned" in lib.pkv_last_error()


@pytest.mark.parametrize("kw", [
    dict(v=P),                                # k and v the same rows
    dict(v=P + 2032), dict(k=21 * P - 2032),  # or sharing 16 bytes
    dict(k=30 * P + 16), dict(k=40 * P + 16), dict(v=50 * P + 16), dict(v=60 * P + 16), dict(v=70 * P),
    dict(k=30 * P - 2048 + 16), dict(k=30 * P + 2 * 128 * 2 * 128 - 16),
    dict(k=70 * P - 2048 + 16), dict(v=60 * P + 2 * 128 * 2 * 4 - 16),
])
def test_read_fp8_refuses_outputs_that_overlap(kw):
    """4 rows of 2 heads are 2,048 bytes; 2 blocks are 65,536 bytes of codes and 2,048 of scales."""
    lib = load()
    a = dict(k=P, v=21 * P, kc=30 * P, vc=40 * P, ks=50 * P, vs=60 * P, slots=70 * P)
    a.update(kw)
    assert lib.pkv_kv_cache_read_fp8(*a.values(), 4, 2, 128, 2, 128, None, None) == -1
    assert b"overlaps" in lib.pkv_last_error()


def test_the_binding_refuses_host_tensors():
    import torch

    from paged_kv_cache_77_gb300 import api

    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    rows = bf(3, 4, 128), bf(3, 2, 128), bf(3, 2, 128), torch.zeros((9, 128)), i32(3), i32(3)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_kv_cache_write(bf(2, 128, 2, 128), bf(2, 128, 2, 128), *rows)
    fp8 = u8(2, 128, 2, 128), u8(2, 128, 2, 128), torch.zeros((2, 2, 128)), torch.zeros((2, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_kv_cache_write_fp8(*fp8, *rows)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv_cache_read_fp8(*fp8, i32(3))


def test_pair_axis_takes_any_sequence_of_the_right_length():
    from paged_kv_cache_77_gb300 import api

    for axis in ([0, 1, 2, 1], (0, 1, 2, 1), np.array([0, 1, 2, 1]), np.array([0, 1, 2, 1], dtype=np.uint8)):
        arr, address = api._axis_array(axis, 8)
        assert list(arr) == [0, 1, 2, 1] and address == (
            arr.ctypes.data if isinstance(arr, np.ndarray) else arr.buffer_info()[0])
    assert api._axis_array(None, 8) == (None, None)
    for axis in ([0, 1, 2], np.zeros((2, 2)), np.zeros(5)):
        with pytest.raises(ValueError, match="pair_axis"):
            api._axis_array(axis, 8)
