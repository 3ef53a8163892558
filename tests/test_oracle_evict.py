"""Pins of the eviction oracle: by hand, by enumeration, and against the attention oracle."""
import itertools

import numpy as np

from oracle import evict_ref as ev
from oracle import paged_ref as ref


def _case(seed, lens, H, hkv, Q, bs=4, d=8):
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 2
    order = rng.permutation(nb)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    keys = rng.standard_normal((nb, bs, hkv, d))
    vals = rng.standard_normal((nb, bs, hkv, d))
    q = rng.standard_normal((len(lens), Q, H, d))
    return rng, table, nb, keys, vals, q


def test_the_added_weights_are_the_softmax_of_the_attention():
    lens = [9, 1, 4, 13]
    _, table, nb, keys, vals, q = _case(1, lens, 6, 3, 2)
    _, lse = ref.paged_spec_decode(q, keys, vals, table, lens, 4, 0.3)
    out, _ = ev.accumulate(np.zeros((nb, 3, 4)), q, lse, keys, table, lens, [0] * 4, 0.3)
    for b, n in enumerate(lens):
        rows = min(n, 2)
        got = np.array([out[table[b, p // 4], :, p % 4] for p in range(n)])
        # A row's weights sum to 1 for each of the two heads of a kv head.
        np.testing.assert_allclose(got.sum(0), 2.0 * rows)
    # Position by position for one sequence and head group, from the scores.
    n, g = 13, 1
    want = np.zeros(n)
    for i in range(2):
        for h in (2, 3):
            end = n - 2 + 1 + i
            s = np.array([0.3 * q[3, i, h] @ keys[table[3, p // 4], p % 4, g] for p in range(end)])
            e = np.exp(s - s.max())
            want[:end] += e / e.sum()
    np.testing.assert_allclose([out[table[3, p // 4], g, p % 4] for p in range(n)], want)


def test_fresh_rows_start_over_and_the_others_decay():
    _, table, nb, keys, _, q = _case(2, [6], 1, 1, 1)
    old = np.full((nb, 1, 4), 5.0)
    lse = np.full((1, 1, 1), 1e9)  # nothing is added
    out, _ = ev.accumulate(old, q, lse, keys, table, [6], [2], 0.3, decay=0.5)
    at = [out[table[0, p // 4], 0, p % 4] for p in range(8)]
    assert at == [2.5] * 4 + [0, 0] + [5, 5]
    for fresh, want in ((-3, 2.5), (99, 0.0)):
        out, _ = ev.accumulate(old, q, lse, keys, table, [6], [fresh], 0.3, decay=0.5)
        assert out[table[0, 0], 0, 0] == want


def test_selection_is_the_best_subset():
    rng, table, nb, _, _, _ = _case(3, [7, 3], 1, 2, 1)
    w = rng.random((nb, 2, 4))
    out = ev.select_rows(w, table, [7, 3], 4, 1, 1)
    for g in range(2):
        row = np.array([w[table[0, p // 4], g, p % 4] for p in range(7)])
        best = max((c for c in itertools.combinations(range(7), 4) if 0 in c and 6 in c),
                   key=lambda c: row[list(c)].sum())
        assert out[0, g].tolist() == list(best)
        assert out[1, g].tolist() == [0, 1, 2, -1]


def test_ties_nan_and_bad_blocks_by_hand():
    table = np.array([[0, 1]], dtype=np.int32)
    w = np.array([[[1, 2, 2, 0]], [[2, -0.0, np.nan, 2]]])
    assert ev.select_rows(w, table, [8], 3)[0, 0].tolist() == [1, 2, 6]
    assert ev.select_rows(w, table, [8], 1)[0, 0].tolist() == [6]
    assert ev.select_rows(w, table, [8], 7)[0, 0].tolist() == [0, 1, 2, 3, 4, 6, 7]
    assert ev.select_rows(w, np.array([[9, 1]]), [8], 4, 1, 0)[0, 0].tolist() == [0, 4, 6, 7]


def test_compaction_keeps_the_attention_over_the_kept_rows():
    lens = [11]
    _, table, nb, keys, vals, q = _case(4, lens, 4, 2, 1)
    kept = np.array([[[0, 2, 3, 5, 10], [1, 2, 6, 9, 10]]], dtype=np.int32)
    k2 = ev.compact(keys, kept, table, table, False)
    v2 = ev.compact(vals, kept, table, table, False)
    o, lse = ref.paged_spec_decode(q, k2, v2, table, [5], 4, 0.3)
    for h in range(4):
        g = h // 2
        K = np.array([keys[table[0, p // 4], p % 4, g] for p in kept[0, g]])
        V = np.array([vals[table[0, p // 4], p % 4, g] for p in kept[0, g]])
        s = 0.3 * K @ q[0, 0, h]
        p = np.exp(s) / np.exp(s).sum()
        np.testing.assert_allclose(o[0, 0, h], p @ V)
    # Head-major caches, a table of its own, an empty tail.
    w = np.arange(nb * 2 * 4.0).reshape(nb, 2, 4)
    new = np.array([[nb - 1, nb - 2]], dtype=np.int32)
    free = [b for b in range(nb) if b not in table]
    new = np.array([free], dtype=np.int32)
    kept[0, 1, 4] = -1
    out = ev.compact(w, kept, table, new, True)
    assert out[new[0, 1], 0, 0] == w[table[0, 2], 0, 2]
    assert out[new[0, 1], 1, 0] == w[new[0, 1], 1, 0]
    assert np.array_equal(out[table[0]], w[table[0]])
