"""GB300-native paged KV cache: slot_mapping writes and paged attention on sm_103a.

The compute lives in libpaged_kv.so (C ABI, include/paged_kv.h); this package is
the build step and a thin ctypes binding over it.
"""
from . import api
from .api import (BlockPool, accumulate_attention_weights, block_num_fixed, block_num_full_offline,
                  block_num_full_online, build_block_table_arange, build_slot_mapping, compact_rows,
                  decode_sparse_workspace_size, decode_workspace_size, kv_cache_read_fp4,
                  kv_cache_read_fp8, kv_cache_write, kv_cache_write_fp4, mla_paged_decode,
                  num_skipped_tokens, paged_attention_decode, paged_attention_decode_fp4,
                  paged_attention_decode_sparse, paged_attention_decode_static,
                  paged_attention_prefill, rope_kv_cache_write, rope_kv_cache_write_fp8,
                  select_blocks, select_rows, update_block_summaries)

__all__ = ["api", "BlockPool", "accumulate_attention_weights", "block_num_fixed",
           "block_num_full_offline", "block_num_full_online", "build_block_table_arange",
           "build_slot_mapping", "compact_rows", "decode_sparse_workspace_size",
           "decode_workspace_size", "kv_cache_read_fp4", "kv_cache_read_fp8", "kv_cache_write",
           "kv_cache_write_fp4", "mla_paged_decode", "num_skipped_tokens", "paged_attention_decode",
           "paged_attention_decode_fp4", "paged_attention_decode_sparse",
           "paged_attention_decode_static", "paged_attention_prefill", "rope_kv_cache_write",
           "rope_kv_cache_write_fp8", "select_blocks", "select_rows", "update_block_summaries"]
