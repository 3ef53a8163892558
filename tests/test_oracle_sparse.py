"""Pins of the block-sparse oracle (oracle/sparse_ref.py): the score bounds every key, the
selection against enumeration, and the attention against the dense oracle."""
import itertools

import numpy as np

from oracle import paged_ref as ref
from oracle import sparse_ref as sp

BS = 4


def _cache(rng, nb, hkv, d):
    return rng.standard_normal((nb, BS, hkv, d))


def test_summaries_are_the_minima_and_maxima_of_the_rows():
    rng = np.random.default_rng(1)
    k = _cache(rng, 9, 2, 3)
    table = np.array([[5, 1, 7], [2, 8, 0]])
    s = np.full((9, 2, 2, 3), 99.0)
    lens = np.zeros(2, dtype=int)
    for step in ([3, 0], [1, 5], [1, 0], [6, 2]):  # within, to the edge, over it, nothing
        lens = lens + step
        s = sp.update_summaries(s, k, table, lens, step, BS)
    for b, n in enumerate(lens):
        for j in range(-(-n // BS)):
            rows = k[table[b, j], :min(BS, n - j * BS)]
            assert np.array_equal(s[table[b, j], :, 0], rows.min(0))
            assert np.array_equal(s[table[b, j], :, 1], rows.max(0))
    assert (s[[3, 4, 6, 0]] == 99.0).all()


def test_score_bounds_the_groups_products_with_every_key():
    rng = np.random.default_rng(2)
    for _ in range(20):
        q = rng.standard_normal((3, 8))
        keys = rng.standard_normal((BS, 8))
        bound = sp.block_score(q, keys.min(0), keys.max(0))
        assert ((q @ keys.T).sum(0) <= bound + 1e-12).all()
    key = rng.standard_normal((1, 8))  # one key: the bound is the product
    np.testing.assert_allclose(sp.block_score(q, key[0], key[0]), (q @ key.T).sum(), rtol=1e-12)


def test_selection_equals_the_best_subset_by_enumeration():
    rng = np.random.default_rng(3)
    nb, n, K = 12, 7, 4
    s = np.sort(rng.standard_normal((nb, 1, 2, 5)), axis=2)
    table = rng.permutation(nb)[:n][None]
    q = rng.standard_normal((1, 1, 2, 5))
    got = sp.select_blocks(q, s, table, [n * BS], K, 1, 1, BS)[0, 0, 0]
    score = [sp.block_score(q[0, 0], *s[table[0, j], 0]) for j in range(n)]
    best = max((c for c in itertools.combinations(range(n), K) if 0 in c and n - 1 in c),
               key=lambda c: sum(score[j] for j in c))
    assert tuple(got) == best


def test_selection_edges():
    s = np.zeros((6, 1, 2, 2))
    table = np.arange(6)[None]
    q = np.ones((1, 2, 1, 2))
    pick = lambda lens, K, sink=0, recent=0, q=q, s=s, t=table: sp.select_blocks(
        q, s, t, lens, K, sink, recent, BS)[0].reshape(2, K).tolist()
    assert pick([0], 2) == [[-1, -1], [-1, -1]]
    assert pick([1], 2) == [[-1, -1], [0, -1]]            # the first of two rows sees nothing
    assert pick([9], 3) == [[0, 1, -1], [0, 1, 2]]        # the second row opens a block
    assert pick([24], 3) == [[0, 1, 2]] * 2               # all equal: the lowest
    assert pick([24], 3, 1, 1) == [[0, 1, 5]] * 2
    assert pick([24], 2, 1, 1) == [[0, 5]] * 2
    s2 = s.copy()
    s2[3, 0, 1] = np.nan
    s2[4] = np.inf
    assert pick([24], 2, s=s2) == [[3, 4]] * 2            # NaN, then infinity
    assert pick([24], 5, t=np.array([[9, 1, 2, 3, 4, 5]])) == [[1, 2, 3, 4, 5]] * 2


def test_sparse_decode_over_all_blocks_is_the_dense_attention():
    rng = np.random.default_rng(4)
    k, v = _cache(rng, 10, 2, 8), _cache(rng, 10, 2, 8)
    table = np.array([[1, 4, 2], [7, 8, 3]])
    lens = [11, 2]
    q = rng.standard_normal((2, 3, 4, 8))
    idx = np.tile(np.array([2, 0, 1]), (2, 3, 2, 1))
    idx[1] = [0, -1, -1]
    o, lse, spread = sp.sparse_decode(q, k, v, table, lens, idx, BS, 0.3)
    want, want_lse = ref.paged_spec_decode(q, k, v, table, lens, BS, 0.3)
    # The second block of the first row is its third entry, beyond the two blocks it sees.
    np.testing.assert_allclose(o, want, atol=1e-13)
    np.testing.assert_allclose(lse[np.isfinite(want_lse)], want_lse[np.isfinite(want_lse)], atol=1e-13)
    assert np.array_equal(np.isfinite(lse), np.isfinite(want_lse))
    assert (spread >= 0).all() and (spread[1, 0] == 0).all()


def test_sparse_decode_masks_to_the_listed_blocks():
    rng = np.random.default_rng(5)
    k, v = _cache(rng, 10, 1, 8), _cache(rng, 10, 1, 8)
    table, n = np.array([[1, 4, 2, 9, 0]]), 18
    q = rng.standard_normal((1, 1, 2, 8))
    o, lse, _ = sp.sparse_decode(q, k, v, table, [n], np.array([[[[3, -1, 4, 0, 7]]]]), BS, 0.5)
    K = ref.gather_sequence(k, table[0], n, BS)[:, 0]
    V = ref.gather_sequence(v, table[0], n, BS)[:, 0]
    seen = np.isin(np.arange(n) // BS, [0, 3, 4])
    for h in range(2):
        w, wl, _ = ref.attend(q[0, 0, h], K, V, seen, 0.5)
        np.testing.assert_allclose(o[0, 0, h], w, atol=1e-14)
        np.testing.assert_allclose(lse[0, 0, h], wl, atol=1e-14)
