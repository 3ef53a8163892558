"""The 4-bit cache's calls refuse bad arguments before anything is launched (through the C ABI
and the binding, no GPU: the pointers are never read)."""
import pytest
import torch

from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import load

P = 1 << 24  # a 16-byte aligned address that nothing reads


def _write(**kw):
    a = dict(k_cache=P, v_cache=2 * P, k_scale=3 * P, v_scale=4 * P, k=5 * P, k_stride=256, v=6 * P,
             v_stride=256, slots=7 * P, num_tokens=5, num_blocks=10, block_size=128, H_kv=2,
             head_dim=128, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return a


SHARED = [
    (dict(head_dim=64), -2, b"head_dim"),
    (dict(num_blocks=0), -1, b"sizes"),
    (dict(H_kv=0), -1, b"sizes"),
    (dict(num_tokens=-1), -1, b"sizes"),
    (dict(num_blocks=1 << 25), -2, b"int32"),
    (dict(num_tokens=1 << 31), -2, b"rows"),
    (dict(k_cache=None), -1, b"null"),
    (dict(v_scale=None), -1, b"null"),
    (dict(k=None), -1, b"null"),
    (dict(slots=None), -1, b"null"),
    (dict(k_scale=3 * P + 8), -1, b"aligned"),
    (dict(v=6 * P + 8), -1, b"aligned"),
    (dict(slots=7 * P + 2), -1, b"aligned"),
    (dict(k=P + 1024), -1, b"overlaps"),
    (dict(v=4 * P + 64), -1, b"overlaps"),
]


@pytest.mark.parametrize("kw,code,word", SHARED + [
    (dict(k_stride=252), -1, b"stride"),
    (dict(v_stride=-256), -1, b"stride"),
    (dict(slots=2 * P + 16), -1, b"overlaps"),
    # Rows that start before the caches and run into them.
    (dict(k=P - 4096, k_stride=1024), -1, b"overlaps"),
])
def test_write_refusals(kw, code, word):
    lib = load()
    assert lib.pkv_kv_cache_write_fp4(*_write(**kw).values()) == code
    assert word in lib.pkv_last_error()


@pytest.mark.parametrize("kw,code,word", SHARED + [
    (dict(k=6 * P + 16), -1, b"overlaps"),
    (dict(k=7 * P), -1, b"overlaps"),
])
def test_read_refusals(kw, code, word):
    lib = load()
    a = _write(**kw)
    args = [a["k"], a["v"], a["k_cache"], a["v_cache"], a["k_scale"], a["v_scale"], a["slots"],
            a["num_tokens"], a["num_blocks"], a["block_size"], a["H_kv"], a["head_dim"], None, None]
    assert lib.pkv_kv_cache_read_fp4(*args) == code
    assert word in lib.pkv_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(out_dtype=7), -1, b"out_dtype"),
    (dict(H=6, H_kv=4), -1, b"multiple"),
    (dict(H=6, H_kv=2), -2, b"unsupported"),
    (dict(head_dim=64), -2, b"head_dim"),
    (dict(block_size=64), -2, b"block_size"),
    (dict(q_len=5), -2, b"q_len"),
    (dict(q_len=0), -2, b"q_len"),
    (dict(H=32, q_len=3), -2, b"rows"),
    (dict(scale=0.0), -1, b"scale"),
    (dict(window=-1), -1, b"window"),
    (dict(max_blocks=1 << 25), -2, b"int32"),
    (dict(B=1 << 30, H=4), -2, b"int32"),
    (dict(k_cache=None), -1, b"null"),
    (dict(v_cache=2 * P + 8), -1, b"aligned"),
])
def test_decode_refusals(kw, code, word):
    a = dict(out=P, out_dtype=1, lse=None, q=8 * P, k_cache=P, v_cache=2 * P, k_scale=3 * P,
             v_scale=4 * P, table=5 * P, max_blocks=4, lens=6 * P, B=2, q_len=1, H=4, H_kv=2,
             head_dim=128, block_size=128, num_blocks=10, scale=0.1, window=0, ws=7 * P,
             ws_bytes=1 << 30, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    lib = load()
    assert lib.pkv_paged_attention_decode_fp4(*a.values()) == code
    assert word in lib.pkv_last_error()


def test_binding_refuses_host_tensors_and_wrong_layouts():
    codes = torch.zeros((2, 3, 128, 64), dtype=torch.uint8)
    scales = torch.zeros((2, 3, 128, 8), dtype=torch.uint8)
    rows = torch.zeros((1, 3, 128), dtype=torch.bfloat16)
    slots = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_cache must be a contiguous uint8 CUDA"):
        api.kv_cache_write_fp4(codes, codes, scales, scales, rows, rows, slots)
    with pytest.raises(ValueError, match="k_cache must be a contiguous uint8 CUDA"):
        api.kv_cache_read_fp4(codes, codes, scales, scales, slots)
    with pytest.raises(ValueError, match="q must be a contiguous bf16 CUDA"):
        api.paged_attention_decode_fp4(rows, codes, codes, scales, scales, slots, slots, 1.0)
