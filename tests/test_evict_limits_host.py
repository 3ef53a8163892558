"""Lists of kept rows are refused where the kernels' 32-bit indexes would pass 2^31 (no GPU: the device
pointers are never read)."""
import ctypes as C

import numpy as np
import pytest

from paged_kv_cache_77_gb300._lib import load

P = 1 << 24  # a 16-byte aligned address that nothing reads


@pytest.mark.parametrize("keep", [(1 << 30) + 1, 2**31 - 1])
@pytest.mark.parametrize("B", [0, 1])
def test_select_rows_refuses_lists_past_its_indexes(keep, B):
    lib = load()
    assert lib.pkv_select_rows(1 << 40, 2 * P, 3 * P, 4, 4 * P, B, 1, 128, 10, keep, 0, 0, None, None) == -2
    assert b"num_keep" in lib.pkv_last_error()


@pytest.mark.parametrize("keep", [(1 << 30) + 1, 2**31 - 1])
@pytest.mark.parametrize("new", [None, 5 * P])
def test_compact_rows_refuses_lists_past_its_indexes(keep, new):
    ptrs, sizes, major = (C.c_void_p * 1)(P), np.array([256], dtype=np.int32), np.zeros(1, dtype=np.int32)
    lib = load()
    assert lib.pkv_compact_rows(ptrs, sizes.ctypes.data, major.ctypes.data, 1, 1 << 40, keep, 4 * P, 4, new,
                                1 << 24 if new else 0, 1, 1, 128, 10, None, None) == -2
    assert b"num_keep" in lib.pkv_last_error()
