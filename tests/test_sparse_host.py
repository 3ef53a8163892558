"""The sparse-decode calls refuse bad arguments before anything is launched (through the C
ABI, no GPU: the pointers are never read)."""
import pytest

from paged_kv_cache_77_gb300._lib import load

P = 1 << 20  # a 16-byte aligned address that nothing reads
BIG = 2 ** 31 - 1


def _call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return getattr(load(), fn)(*{**defaults, **kw}.values())


SUMMARIES = dict(summaries=P, k_cache=P, table=P, max_blocks=4, lens=P, num_new=P, max_new=5, B=2, Hkv=2,
                 d=128, bs=128, nb=9, st=None, stream=None)
SELECT = dict(out=P, q=P, summaries=P, table=P, max_blocks=4, lens=P, B=2, q_len=1, H=8, Hkv=2, d=128,
              bs=128, nb=9, K=4, sink=0, recent=1, st=None, stream=None)
SPARSE = dict(out=P, dtype=1, lse=None, q=P, k=P, v=P, table=P, max_blocks=4, lens=P, idx=P, K=4, B=2, q_len=1,
              H=8, Hkv=2, d=128, bs=128, nb=9, scale=0.1, ws=None, ws_bytes=0, st=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(Hkv=0), -1), (dict(max_blocks=0), -1), (dict(nb=0), -1), (dict(max_new=-1), -1),
    (dict(d=64), -2), (dict(bs=64), -2), (dict(summaries=None), -1), (dict(k_cache=P + 8), -1),
    (dict(num_new=None), -1), (dict(B=1 << 20, Hkv=1 << 12), -2),
    (dict(B=0, table=None, lens=None, num_new=None), 0), (dict(max_new=0), 0),
])
def test_summaries_refusals(kw, code):
    assert _call("pkv_update_block_summaries", SUMMARIES, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(q_len=0), -1), (dict(H=9), -1), (dict(H=34), -2), (dict(d=64), -2),
    (dict(bs=16), -2), (dict(K=0), -1), (dict(sink=-1), -1), (dict(sink=4), -1), (dict(sink=BIG, recent=BIG), -1),
    (dict(max_blocks=8193), -2), (dict(B=1 << 28), -2), (dict(q=None), -1), (dict(out=None), -1),
    (dict(q=P + 2), -1), (dict(B=0, q=None, out=None, lens=None, table=None, summaries=None), 0),
])
def test_select_refusals(kw, code):
    assert _call("pkv_select_blocks", SELECT, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(q_len=0), -1), (dict(K=0), -1), (dict(H=9), -1), (dict(H=6), -2), (dict(H=64), -2),
    (dict(d=64), -2), (dict(bs=64), -2), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(dtype=7), -1), (dict(B=1 << 16, q_len=1 << 16), -2), (dict(B=1 << 30, Hkv=8), -2),
    (dict(max_blocks=BIG), -2), (dict(q=None), -1), (dict(k=P + 2), -1),
    (dict(B=0, q=None, out=None), 0),
])
def test_sparse_decode_refusals(kw, code):
    assert _call("pkv_paged_attention_decode_sparse", SPARSE, kw) == code


@pytest.mark.parametrize("fn,defaults,out,size,inputs", [
    # 9 blocks of 2 heads: summaries of 512 bytes each, keys of 32,768.
    ("pkv_update_block_summaries", SUMMARIES, "summaries", 9216,
     dict(k_cache=9 * 2 * 32768, table=32, lens=8, num_new=8)),
    # 2 rows, 8 query heads, 4 of 4 blocks for 2 kv heads.
    ("pkv_select_blocks", SELECT, "out", 64, dict(q=4096, summaries=9216, table=32, lens=8)),
])
def test_outputs_that_overlap_what_the_call_reads_are_refused(fn, defaults, out, size, inputs):
    lib = load()
    apart = {name: (i + 2) * P for i, name in enumerate(inputs)}
    for name, nbytes in inputs.items():
        for at in (apart[name], apart[name] - size + 16, apart[name] + max(nbytes - 16, 0)):
            assert _call(fn, defaults, {**apart, out: at}) == -1
            assert b"overlaps" in lib.pkv_last_error(), (name, at)


def test_workspace_is_that_of_a_batch_of_rows():
    lib = load()
    for B, Q in ((4, 1), (4, 3), (0, 2)):
        assert lib.pkv_decode_sparse_workspace_size(B, Q, 64, 8, 128) == \
            lib.pkv_decode_workspace_size(B * Q, 64, 8, 128)
    assert lib.pkv_decode_sparse_workspace_size(4, 0, 64, 8, 128) == 0
    assert lib.pkv_decode_sparse_workspace_size(1 << 20, 1 << 20, 64, 8, 128) == 0


def test_selftest_of_the_products_refuses_bad_arguments():
    lib = load()
    for args in ((P, P, P, -1), (None, P, P, 2), (P, P, None, 2), (P, P + 8, P, 2)):
        assert lib.pkv_selftest_bf16_products(*args, None) == -1


def test_the_binding_refuses_host_tensors():
    import torch

    from paged_kv_cache_77_gb300 import api

    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache, summaries, q, table, lens = bf(3, 128, 2, 128), bf(3, 2, 2, 128), bf(1, 4, 128), i32(1, 2), i32(1)
    with pytest.raises(ValueError, match="CUDA"):
        api.update_block_summaries(summaries, cache, table, lens, i32(1), 1)
    with pytest.raises(ValueError, match="CUDA"):
        api.select_blocks(q, summaries, table, lens, 2)
    with pytest.raises(ValueError, match="CUDA"):
        api.paged_attention_decode_sparse(q, cache, cache, table, lens, i32(1, 2, 2), 0.1)
