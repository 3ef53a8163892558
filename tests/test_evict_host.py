"""The eviction calls refuse bad arguments before anything is launched (through the C ABI and the
binding, no GPU: the device pointers are never read)."""
import ctypes as C

import numpy as np
import pytest
import torch

from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import load

P = 1 << 24  # a 16-byte aligned address that nothing reads


@pytest.mark.parametrize("kw,code,word", [
    (dict(B=-1), -1, b"sizes"),
    (dict(q_len=0), -1, b"sizes"),
    (dict(H=6, H_kv=4), -1, b"multiple"),
    (dict(fmt=3), -1, b"key_format"),
    (dict(head_dim=64), -2, b"head_dim"),
    (dict(block_size=16), -2, b"block_size"),
    (dict(H=34, H_kv=2), -2, b"exceeds 16"),
    (dict(q_len=1 << 21), -2, b"q_len"),
    (dict(max_blocks=1 << 25), -2, b"int32"),
    (dict(num_blocks=1 << 25), -2, b"int32"),
    (dict(scale=float("nan")), -1, b"scale"),
    (dict(decay=1.5), -1, b"decay"),
    (dict(decay=float("nan")), -1, b"decay"),
    (dict(lse=None), -1, b"null"),
    (dict(k_scale=5 * P), -1, b"k_scale"),
    (dict(fmt=1), -1, b"k_scale"),
    (dict(fmt=2), -1, b"k_scale"),
    (dict(weights=P + 4), -1, b"aligned"),
    (dict(q=2 * P + 2), -1, b"aligned"),
    (dict(weights=2 * P), -1, b"overlaps"),
    (dict(weights=4 * P + 16), -1, b"overlaps"),
    (dict(weights=8 * P), -1, b"overlaps"),
    (dict(fmt=2, k_scale=P + 64), -1, b"overlaps"),
])
def test_accumulate_refusals(kw, code, word):
    a = dict(weights=P, q=2 * P, lse=3 * P, k_cache=4 * P, k_scale=None, fmt=0, table=6 * P,
             max_blocks=4, lens=7 * P, fresh=8 * P, B=2, q_len=1, H=4, H_kv=2, head_dim=128,
             block_size=128, num_blocks=10, scale=0.1, decay=1.0, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    lib = load()
    assert lib.pkv_accumulate_attention_weights(*a.values()) == code
    assert word in lib.pkv_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(keep=0), -1, b"sizes"),
    (dict(sink=-1), -1, b"sizes"),
    (dict(block_size=64), -2, b"block_size"),
    (dict(sink=5, recent=6), -1, b"num_keep"),
    (dict(sink=2**31 - 1, recent=2**31 - 1, keep=2**31 - 1), -1, b"num_keep"),
    (dict(max_blocks=32769), -2, b"max_blocks"),
    (dict(num_blocks=1 << 24), -2, b"int32"),
    (dict(B=1 << 27), -2, b"int32"),
    (dict(weights=None), -1, b"null"),
    (dict(kept=P + 4), -1, b"aligned"),
    (dict(kept=2 * P + 512), -1, b"overlaps"),
    (dict(kept=4 * P - 16), -1, b"overlaps"),
])
def test_select_rows_refusals(kw, code, word):
    a = dict(kept=P, weights=2 * P, table=3 * P, max_blocks=4, lens=4 * P, B=2, H_kv=2, block_size=128,
             num_blocks=10, keep=10, sink=1, recent=2, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    lib = load()
    assert lib.pkv_select_rows(*a.values()) == code
    assert word in lib.pkv_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(keep=0), -1, b"sizes"),
    (dict(n=0), -1, b"sizes"),
    (dict(n=17), -2, b"16 caches"),
    (dict(num_blocks=1 << 25), -2, b"int32"),
    (dict(new=5 * P, new_max=1, keep=129), -1, b"fit"),
    (dict(new=5 * P, new_max=0), -1, b"fit"),
    (dict(kept=None), -1, b"null"),
    (dict(ptrs=[P, None]), -1, b"null"),
    (dict(ptrs=[P, 2 * P + 8]), -1, b"aligned"),
    (dict(sizes=[256, 6]), -2, b"rows of 6"),
    (dict(sizes=[256, 0]), -2, b"rows of 0"),
    (dict(ptrs=[P, P]), -1, b"caches 0 and 1 overlap"),
    (dict(ptrs=[P, P + 4096]), -1, b"caches 0 and 1 overlap"),
    (dict(ptrs=[P, 3 * P]), -1, b"cache 1 overlaps"),
    (dict(ptrs=[4 * P, 2 * P]), -1, b"cache 0 overlaps"),
    (dict(ptrs=[P, 5 * P], new=5 * P, new_max=4), -1, b"cache 1 overlaps"),
])
def test_compact_rows_refusals(kw, code, word):
    a = dict(ptrs=[P, 2 * P], sizes=[256, 4], n=2, kept=3 * P, keep=10, table=4 * P, max_blocks=4,
             new=None, new_max=0, B=2, H_kv=2, block_size=128, num_blocks=10, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    ptrs = (C.c_void_p * 2)(*a.pop("ptrs"))
    sizes = np.array(a.pop("sizes"), dtype=np.int32)
    major = np.zeros(2, dtype=np.int32)
    lib = load()
    assert lib.pkv_compact_rows(ptrs, sizes.ctypes.data, major.ctypes.data, *a.values()) == code
    assert word in lib.pkv_last_error()


def test_nothing_to_do():
    lib = load()
    assert lib.pkv_select_rows(None, None, None, 4, None, 0, 2, 128, 10, 5, 0, 0, None, None) == 0
    assert lib.pkv_compact_rows(None, None, None, 1, None, 5, None, 4, None, 0, 0, 2, 128, 10, None, None) == 0


def test_binding_refuses_host_tensors():
    f32, i32 = torch.zeros((2, 3, 128)), torch.zeros((1, 3, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="weights must be a contiguous fp32 CUDA"):
        api.select_rows(f32, i32[0], i32[0, 0, :1], 4)
    with pytest.raises(ValueError, match="kept must be a contiguous int32 CUDA"):
        api.compact_rows(i32, i32[0], row_caches=[f32])
    with pytest.raises(ValueError, match="at least one cache"):
        api.compact_rows(i32, i32[0])
    with pytest.raises(ValueError, match="q must be a contiguous bf16 CUDA"):
        api.accumulate_attention_weights(f32, f32, f32, f32, i32, i32, i32, 1.0)
