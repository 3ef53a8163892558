"""GPU parity of eviction by accumulated attention weight against the float64 oracle.

Selections are whole numbers and moves are copies: equal. A weight is exp(scale q . k - lse): the
products are exact and their fp32 sums off by at most 512 2^-24 of the sum of their magnitudes
(`reach`, scaled), the scaled score and the log-sum-exp (rounded to fp32 and multiplied by log2 e)
by 4 2^-24 of themselves each, the exponential by 2^-21 of itself; a position's sum over n terms
and its product with the decay add (n + 2) 2^-24 of the sum."""
import numpy as np
import pytest
import torch

import synth
from oracle import evict_ref as ev
from oracle import fp4_ref as f4
from oracle import fp8_ref as f8
from oracle import paged_ref as ref
from oracle.paged_ref import bf16_bits_to_f64
from paged_kv_cache_77_gb300 import api

pytestmark = pytest.mark.gpu

BS, D = 128, 128


def f64(t):
    return bf16_bits_to_f64(synth.bf16_bits(t.contiguous()))


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make_table(rng, lens, nb_more=2, width=None, bs=BS):
    need = [-(-int(n) // bs) for n in lens]
    nb = sum(need) + nb_more
    order = rng.permutation(nb)
    table = np.full((len(need), width or max(1, max(need))), -5, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, nb


def keys_of(fmt, rng, nb, hkv):
    """(k_cache, k_scale, float64 keys [nb, bs, H_kv, d]) of random rows."""
    rows = torch.as_tensor(rng.standard_normal((nb * BS, hkv, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    every = ints(np.arange(nb * BS))
    if fmt == "bf16":
        cache = rows.view(nb, BS, hkv, D)
        return cache, None, f64(cache)
    if fmt == "fp8":
        c = [torch.zeros((nb, BS, hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.zeros((nb, hkv, BS), device="cuda") for _ in range(2)]
        api.kv_cache_write_fp8(*c, *s, rows, rows, every)
        return c[0], s[0], f8.dequantize_cache(c[0].cpu().numpy(), s[0].cpu().numpy())
    c = [torch.zeros((nb, hkv, BS, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.zeros((nb, hkv, BS, 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    api.kv_cache_write_fp4(*c, *s, rows, rows, every)
    return c[0], s[0], f4.dequantise_cache(c[0].cpu().numpy(), s[0].cpu().numpy())


def check_weights(got, want, reach, lse, count, old=0.0):
    """`count`: terms of a position's sum at most; `old`: magnitude of what was there before."""
    got = got.double().cpu().numpy()
    top = np.abs(lse[np.isfinite(lse)]).max(initial=0.0)
    rel = reach * 512 * 2.0 ** -24 + (2 * reach + top) * 4 * 2.0 ** -24 + 2.0 ** -21 + (count + 2) * 2.0 ** -24
    err = np.abs(got - want)
    assert (err <= 1.01 * rel * np.abs(want) + 1e-30).all(), (err / (rel * np.abs(want) + 1e-30)).max()


# ------------------------------------------------------------------ accumulate
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("H,hkv,Q", [(8, 8, 1), (16, 2, 1), (6, 2, 3), (16, 1, 4), (5, 1, 2), (4, 4, 40)])
def test_weights(fmt, H, hkv, Q):
    rng = np.random.default_rng(H + Q)
    lens = [1, 0, 130, 300, 128, 15, 3, 257]
    table, nb = make_table(rng, lens)
    cache, k_scale, keys = keys_of(fmt, rng, nb, hkv)
    q = torch.as_tensor(rng.standard_normal((len(lens), Q, H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    _, lse = ref.paged_spec_decode(f64(q), keys, keys, np.maximum(table, 0), lens, BS, 0.09)
    lse_d = torch.as_tensor(lse, dtype=torch.float32).cuda()
    w0 = rng.random((nb, hkv, BS)).astype(np.float32)
    w = torch.as_tensor(w0).cuda()
    fresh = [1, 3, 0, -2, 500, 7, Q, 100]
    st = status()
    qq = q[:, 0].contiguous() if Q == 1 else q
    ll = lse_d[:, 0].contiguous() if Q == 1 else lse_d
    api.accumulate_attention_weights(w, qq, ll, cache, ints(table), ints(lens), ints(fresh), 0.09,
                                     k_scale=k_scale, decay=0.75, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    want, reach = ev.accumulate(w0, f64(q), lse_d.double().cpu().numpy(), keys, table, lens, fresh, 0.09, 0.75)
    check_weights(w, want, reach, lse, Q * H // hkv)
    # Rows behind the sequences' ends, and blocks of no sequence, are as they were.
    same = want == w0
    assert same.any() and np.array_equal(w.cpu().numpy()[same], w0[same])


def test_weights_of_many_query_rows_in_pieces():
    """An observation window: the last 37 rows of each prompt, 16 heads per kv head."""
    rng = np.random.default_rng(7)
    lens, Q, H = [200, 20], 37, 16
    table, nb = make_table(rng, lens)
    cache, _, keys = keys_of("bf16", rng, nb, 1)
    q = torch.as_tensor(rng.standard_normal((2, Q, H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    _, lse = ref.paged_spec_decode(f64(q), keys, keys, np.maximum(table, 0), lens, BS, 0.09)
    lse_d = torch.as_tensor(lse, dtype=torch.float32).cuda()
    w0 = rng.random((nb, 1, BS)).astype(np.float32)
    got = []
    for _ in range(2):
        w = torch.as_tensor(w0).cuda()
        api.accumulate_attention_weights(w, q, lse_d, cache, ints(table), ints(lens), ints([50, 20]), 0.09,
                                         decay=0.5)
        torch.cuda.synchronize()
        got.append(w.clone())
    assert torch.equal(*got)
    want, reach = ev.accumulate(w0, f64(q), lse_d.double().cpu().numpy(), keys, table, lens, [50, 20], 0.09, 0.5)
    check_weights(got[0], want, reach, lse, Q * H)
    # Each row's weights sum to one per head.
    total = sum(float(got[0][table[b, p // BS], 0, p % BS].double()) for b in (1,) for p in range(20))
    assert abs(total - 20 * H) < 1e-3 * 20 * H


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_weights_skip_what_no_row_sees_and_bad_entries(fmt):
    """NaN keys behind the end and in later rows stay out; a NaN key that a row sees shows."""
    rng = np.random.default_rng(9)
    lens, hkv, Q = [140, 260], 2, 2
    table, nb = make_table(rng, lens)
    cache, k_scale, keys = keys_of(fmt, rng, nb, hkv)

    def poison(seq, pos):
        blk, off = int(table[seq, pos // BS]), pos % BS
        if fmt == "bf16":
            cache[blk, off] = float("nan")
        elif fmt == "fp8":
            k_scale[blk, :, off] = float("nan")
        else:
            k_scale[blk, :, off, 3] = 0xFF

    q = torch.as_tensor(rng.standard_normal((2, Q, 4, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    _, lse = ref.paged_spec_decode(f64(q), keys, keys, np.maximum(table, 0), lens, BS, 0.09)
    lse_d = torch.as_tensor(lse, dtype=torch.float32).cuda()
    for p in range(141, 256):
        poison(0, p)
    poison(1, 77)
    w0 = rng.random((nb, hkv, BS)).astype(np.float32)
    w = torch.as_tensor(w0).cuda()
    bad = table.copy()
    bad[1, 1] = nb + 3
    st = status()
    api.accumulate_attention_weights(w, q, lse_d, cache, ints(bad), ints(lens), ints([0, 0]), 0.09,
                                     k_scale=k_scale, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    want, reach = ev.accumulate(w0, f64(q), lse_d.double().cpu().numpy(), keys, bad, lens, [0, 0], 0.09)
    got = w.cpu().numpy()
    at = (int(table[1, 0]), slice(None), 77)
    assert np.isnan(got[at]).all()
    got[at] = want[at]
    assert np.isfinite(got).all()
    check_weights(torch.as_tensor(got), want, reach, lse, 4)
    st.zero_()
    api.accumulate_attention_weights(w, q, lse_d, cache, ints(table), ints([999999, -1]), ints([0, 0]), 0.09,
                                     k_scale=k_scale, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) & 4


def test_weights_over_many_sequences_and_a_long_one():
    rng = np.random.default_rng(10)
    lens = [int(n) for n in rng.integers(0, 300, 90)] + [9000]
    table, nb = make_table(rng, lens)
    cache, _, keys = keys_of("bf16", rng, nb, 4)
    q = torch.as_tensor(rng.standard_normal((91, 8, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    w = torch.zeros((nb, 4, BS), device="cuda")
    lse = torch.zeros((91, 8), device="cuda")
    out = api.paged_attention_decode(q, cache, cache, ints(table), ints(lens), 0.09, lse=lse)
    assert out is not None
    fresh = ints(lens)
    w.fill_(float("nan"))
    api.accumulate_attention_weights(w, q, lse, cache, ints(table), ints(lens), fresh, 0.09)
    torch.cuda.synchronize()
    got = w.double().cpu().numpy()
    l64 = lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        if not n:
            continue
        p = np.arange(n)
        rows = keys[table[b, p // BS], p % BS]                      # [n, 4, d]
        z = 0.09 * np.einsum("ghd,ngd->ngh", f64(q)[b].reshape(4, 2, D), rows)
        want = np.exp(z - l64[b].reshape(4, 2)).sum(-1)
        here = got[table[b, p // BS], :, p % BS]
        assert np.abs(here - want).max() <= 1e-4 * want.max()
        np.testing.assert_allclose(here, want, rtol=1e-4)


# ------------------------------------------------------------------ select
def _weights(rng, kind, nb, hkv):
    w = np.exp(2.5 * rng.standard_normal((nb, hkv, BS)) - 8).astype(np.float32)
    if kind == "few":       # many ties
        w = rng.integers(0, 4, (nb, hkv, BS)).astype(np.float32)
    elif kind == "one":
        w[:] = 0.25
    elif kind == "special":
        w = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, -1.0, 1e-45, 1.0], np.float32), w.shape)
    elif kind == "close":   # weights that differ in their last bits only
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 60, w.shape).astype(np.int32)).view(np.float32)
    return w


@pytest.mark.parametrize("kind", ["spread", "few", "one", "special", "close"])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (7, 0, 0), (100, 4, 30), (128, 0, 128), (300, 1, 0),
                                              (64, 64, 0), (1000, 3, 500)])
def test_select_rows(kind, keep, sink, recent):
    rng = np.random.default_rng(keep)
    lens = [0, 1, keep, keep + 1, 129, 1500, 640, 77]
    table, nb = make_table(rng, lens, width=13)
    w = _weights(rng, kind, nb, 3)
    st = status()
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints(lens), keep, sink, recent, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    np.testing.assert_array_equal(kept.cpu().numpy(), ev.select_rows(w, table, lens, keep, sink, recent))


@pytest.mark.parametrize("B,hkv,n,keep", [(1, 1, 300000, 5000), (2, 3, 40000, 39999), (40, 8, 5000, 900),
                                          (1, 2, 1048576, 1)])
def test_select_rows_of_long_sequences(B, hkv, n, keep):
    """Against numpy's stable sort."""
    rng = np.random.default_rng(n)
    lens = [n - 3 * b for b in range(B)]
    table, nb = make_table(rng, lens)
    w = _weights(rng, "spread", nb, hkv)
    w[:, 0] = np.round(w[:, 0] * 4096) / 4096  # ties
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints(lens), keep)
    torch.cuda.synchronize()
    got = kept.cpu().numpy()
    for b in range(B):
        blocks = table[b, :-(-lens[b] // BS)]
        for g in range(hkv):
            row = w[blocks, g].reshape(-1)[:lens[b]]
            want = np.sort(np.argsort(-row, kind="stable")[:keep])
            np.testing.assert_array_equal(got[b, g, :len(want)], want)


@pytest.mark.parametrize("kind", ["few", "one", "special", "close", "ascending", "descending", "period", "two levels",
                                  "outliers", "zeros"])
@pytest.mark.parametrize("n,keep,sink,recent", [(9000, 700, 4, 64), (70001, 9000, 0, 1), (200000, 199000, 1, 0)])
def test_select_rows_where_a_sample_misleads(kind, n, keep, sink, recent):
    """Weights of few values, all but equal, in order, or with a period of the blocks': against
    numpy's sort."""
    rng = np.random.default_rng(n)
    lens = [n, n - 129]
    table, nb = make_table(rng, lens)
    w = _weights(rng, kind, nb, 2)
    place = np.zeros(nb * BS)
    for b in range(2):
        p = np.arange(lens[b])
        place[table[b, p // BS] * BS + p % BS] = p
    place = np.broadcast_to(place.reshape(nb, 1, BS), w.shape)
    if kind == "ascending":
        w = place.astype(np.float32)
    elif kind == "descending":
        w = (1e6 - place).astype(np.float32)
    elif kind == "period":      # a block's large weights all in one place
        w = np.where(place % BS < 8, 1.0 + place % 7, 1e-3 * (1 + place % 11)).astype(np.float32)
    elif kind == "two levels":  # the border lies between two plateaus
        w = (1.0 + (rng.random(w.shape) < (keep - sink - recent) / n)).astype(np.float32)
    elif kind == "outliers":
        w = np.where(rng.random(w.shape) < 1e-3, 1e30, 1.0 + 1e-6 * rng.random(w.shape)).astype(np.float32)
    elif kind == "zeros":
        w = np.where(rng.random(w.shape) < 0.01, rng.random(w.shape), 0.0).astype(np.float32)
    kept = api.select_rows(torch.as_tensor(np.ascontiguousarray(w)).cuda(), ints(table), ints(lens), keep, sink,
                           recent)
    torch.cuda.synchronize()
    got = kept.cpu().numpy()
    for b in range(2):
        m = lens[b]
        for g in range(2):
            row = w[table[b, :-(-m // BS)], g].reshape(-1)[:m]
            # Rows always kept, then NaN, then the others by weight; equal ones by position.
            rank = np.where(np.isnan(row), 1, 2)
            rank[:sink] = rank[m - recent:] = 0
            weight = np.where(rank == 2, row, 0.0)
            want = np.sort(np.lexsort((np.arange(m), -weight, rank))[:keep])
            np.testing.assert_array_equal(got[b, g, :len(want)], want)


def test_select_rows_of_bad_blocks_and_lengths():
    rng = np.random.default_rng(3)
    lens = [500, 300]
    table, nb = make_table(rng, lens)
    w = _weights(rng, "spread", nb, 2)
    table[0, 1], table[1, 0] = -9, nb
    st = status()
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints(lens), 400, 10, 5, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    np.testing.assert_array_equal(kept.cpu().numpy(), ev.select_rows(w, table, lens, 400, 10, 5))
    st.zero_()
    table, nb = make_table(rng, lens)
    w = _weights(rng, "spread", nb, 2)
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints([99999, -3]), 50, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 4
    np.testing.assert_array_equal(kept.cpu().numpy()[0], ev.select_rows(w, table, [512], 50)[0])
    assert (kept[1] == -1).all()


# ------------------------------------------------------------------ compact
def _kept(rng, B, hkv, lens, keep):
    kept = np.full((B, hkv, keep), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for g in range(hkv):
            m = min(n, keep)
            kept[b, g, :m] = np.sort(rng.choice(n, m, replace=False))
    return kept


def _caches(rng, nb, bs, hkv):
    """Caches of every kind: bf16 k and v, FP8 codes, 4-bit codes, scales, weights, odd rows."""
    def t(*shape, dtype=torch.uint8):
        return torch.as_tensor(rng.integers(0, 256, shape, dtype=np.uint8)).cuda() if dtype == torch.uint8 else \
            torch.as_tensor(rng.standard_normal(shape), dtype=torch.float32).to(dtype).cuda()
    row = [t(nb, bs, hkv, 128, dtype=torch.bfloat16), t(nb, bs, hkv, 128), t(nb, bs, hkv, 12)]
    head = [t(nb, hkv, bs, 64), t(nb, hkv, bs, 8), t(nb, hkv, bs, dtype=torch.float32),
            t(nb, hkv, bs, 5, 20)]
    return row, head


@pytest.mark.parametrize("own_blocks", [False, True])
@pytest.mark.parametrize("B,hkv,keep,longest,bs", [(3, 2, 100, 700, 128), (1, 1, 1, 400, 128), (2, 3, 2600, 5000, 128),
                                                   (5, 1, 129, 300, 128), (2, 4, 37, 90, 16)])
def test_compact_rows(own_blocks, B, hkv, keep, longest, bs):
    rng = np.random.default_rng(keep + B)
    lens = [longest] + [int(n) for n in rng.integers(0, longest, B - 1)]
    width = -(-keep // bs)
    table, nb = make_table(rng, lens, nb_more=B * width + 1, bs=bs)
    new = None
    if own_blocks:
        free = np.setdiff1d(np.arange(nb), table)
        new = rng.permutation(free)[:B * width].reshape(B, width).astype(np.int32)
    kept = _kept(rng, B, hkv, lens, keep)
    row, head = _caches(rng, nb, bs, hkv)
    before = [t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy() for t in row + head]
    st = status()
    api.compact_rows(ints(kept), ints(table), row, head, None if new is None else ints(new), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for i, t in enumerate(row + head):
        want = ev.compact(before[i], kept, table, table if new is None else new, i >= len(row))
        got = t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
        np.testing.assert_array_equal(got, want, err_msg=f"cache {i}")


def test_compact_rows_in_place_with_every_shift():
    """Lists that drop one row, every other row, the front, or nothing."""
    rng = np.random.default_rng(4)
    n, keep = 1000, 600
    lists = [np.r_[0:300, 301:601], np.arange(0, 1000, 2)[:500], np.arange(400, 1000), np.arange(600),
             np.r_[0, 401:1000], np.arange(999, 1000)]
    kept = np.full((6, 1, keep), -1, dtype=np.int32)
    for b, x in enumerate(lists):
        kept[b, 0, :len(x)] = x
    table, nb = make_table(rng, [n] * 6)
    cache = torch.as_tensor(rng.integers(0, 2**31, (nb, BS, 1, 64), dtype=np.int32)).cuda()
    before = cache.cpu().numpy()
    api.compact_rows(ints(kept), ints(table), row_caches=[cache])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(cache.cpu().numpy(), ev.compact(before, kept, table, table, False))


def test_compact_rows_with_bad_entries():
    rng = np.random.default_rng(5)
    lens = [300, 300]
    table, nb = make_table(rng, lens)
    kept = _kept(rng, 2, 2, lens, 140)
    cache = torch.as_tensor(rng.random((nb, 2, BS)), dtype=torch.float32).cuda()
    before = cache.cpu().numpy()
    bad = table.copy()
    bad[0, 1], bad[1, 2] = nb, -1
    st = status()
    api.compact_rows(ints(kept), ints(bad), head_caches=[cache], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    np.testing.assert_array_equal(cache.cpu().numpy(), ev.compact(before, kept, bad, bad, True))
    st.zero_()
    kept[1, 1, -1] = 128 * 3
    before = cache.cpu().numpy()
    api.compact_rows(ints(kept), ints(table), head_caches=[cache], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 4
    np.testing.assert_array_equal(cache.cpu().numpy(), ev.compact(before, kept, table, table, True))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_a_serving_loop_that_evicts(fmt):
    """Prompts, decode steps that accumulate, an eviction that gives blocks back, more steps: the
    attention after it is that over the kept rows, whose sums moved with them."""
    rng = np.random.default_rng(12)
    H, hkv, scale, keep = 8, 2, 0.09, 128
    lens = [300, 170, 90]
    pool = api.BlockPool(24)
    table = np.zeros((3, 4), dtype=np.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // BS)] = pool.alloc(-(-n // BS))
    w = torch.full((24, hkv, BS), float("nan"), device="cuda")
    if fmt == "bf16":
        caches = [torch.zeros((24, BS, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    else:
        caches = [torch.zeros((24, hkv, BS, m), dtype=torch.uint8, device="cuda") for m in (64, 64, 8, 8)]
    state = {(b, g): [] for b in range(3) for g in range(hkv)}  # (k, v, weight) per row, float64

    def rows(n):
        return torch.as_tensor(rng.standard_normal((n, hkv, D)), dtype=torch.float32).to(torch.bfloat16).cuda()

    def held(x):
        return f64(x) if fmt == "bf16" else f4.dequantise(*f4.quantise(f64(x)))

    def write(start, new):
        k, v = rows(sum(new)), rows(sum(new))
        slots = ints(api.build_slot_mapping(table, start, new, BS))
        if fmt == "bf16":
            api.kv_cache_write(*caches, k, v, slots)
        else:
            api.kv_cache_write_fp4(*caches, k, v, slots)
        at = 0
        for b in range(3):
            for t in range(at, at + new[b]):
                for g in range(hkv):
                    state[b, g].append([held(k)[t, g], held(v)[t, g], 0.0])
            at += new[b]

    def step(seq, fresh):
        q = torch.as_tensor(rng.standard_normal((3, H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
        lse = torch.zeros((3, H), device="cuda")
        t, n = ints(table), ints(seq)
        if fmt == "bf16":
            out = api.paged_attention_decode(q, *caches, t, n, scale, lse=lse)
            api.accumulate_attention_weights(w, q, lse, caches[0], t, n, ints(fresh), scale)
        else:
            out = api.paged_attention_decode_fp4(q, *caches, t, n, scale, lse=lse)
            api.accumulate_attention_weights(w, q, lse, caches[0], t, n, ints(fresh), scale, k_scale=caches[2])
        torch.cuda.synchronize()
        for b in range(3):
            for h in range(H):
                own = state[b, h // 4]
                s = scale * np.array([r[0] for r in own]) @ f64(q)[b, h]
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ np.array([r[1] for r in own])
                assert np.abs(out[b, h].double().cpu().numpy() - o).max() <= 1e-2
                for r, x in zip(own, p):
                    r[2] += x

    write([0, 0, 0], lens)
    step(lens, lens)
    for _ in range(3):
        write(lens, [1, 1, 1])
        lens = [n + 1 for n in lens]
        step(lens, [1, 1, 1])
    t = ints(table)
    kept = api.select_rows(w, t, ints(lens), keep, num_sink=2, num_recent=16)
    if fmt == "bf16":
        api.compact_rows(kept, t, row_caches=caches, head_caches=[w])
    else:
        api.compact_rows(kept, t, head_caches=[*caches, w])
    torch.cuda.synchronize()
    order = kept.cpu().numpy()
    for (b, g), own in state.items():
        mine = order[b, g][order[b, g] >= 0]
        sums = np.array([r[2] for r in own])
        assert len(mine) == min(len(own), keep)
        # The weakest row that stayed outweighs the strongest that went (the sums are fp32 of rounded steps).
        if len(own) > keep:
            free = np.setdiff1d(mine, np.r_[0:2, len(own) - 16:len(own)])
            gone = np.setdiff1d(np.arange(len(own)), mine)
            assert sums[free].min() >= sums[gone].max() * (1 - 1e-2)
        state[b, g] = [own[i] for i in mine]
    for b, n in enumerate(lens):
        spare = table[b, -(-min(n, keep) // BS):-(-n // BS)]
        if len(spare):
            pool.free(spare)
    lens = [min(n, keep) for n in lens]
    for b in range(3):
        if lens[b] % BS == 0:
            table[b, lens[b] // BS] = pool.alloc(1)[0]
    for _ in range(2):
        write(lens, [1, 1, 1])
        lens = [n + 1 for n in lens]
        step(lens, [1, 1, 1])
    got = w.double().cpu().numpy()
    for (b, g), own in state.items():
        p = np.arange(lens[b])
        np.testing.assert_allclose(got[table[b, p // BS], g, p % BS], [r[2] for r in own], rtol=2e-2)


def test_eviction_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(14)
    lens = [500, 260]
    table, nb = make_table(rng, lens)
    cache, _, keys = keys_of("bf16", rng, nb, 2)
    q = torch.as_tensor(rng.standard_normal((2, 4, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    lse = torch.full((2, 4), 3.0, device="cuda")
    w0 = torch.as_tensor(rng.random((nb, 2, BS)), dtype=torch.float32).cuda()
    v0 = cache.clone()
    w, v = w0.clone(), v0.clone()
    t, n, fresh = ints(table), ints(lens), ints([1, 1])
    kept = torch.zeros((2, 2, 200), dtype=torch.int32, device="cuda")

    def evict(stream=None):
        api.accumulate_attention_weights(w, q, lse, cache, t, n, fresh, 0.09, stream=stream)
        api.select_rows(w, t, n, 200, 1, 8, out=kept, stream=stream)
        api.compact_rows(kept, t, row_caches=[v], head_caches=[w], stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    evict(side)
    torch.cuda.synchronize()
    first = w.clone(), v.clone(), kept.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        evict()
    w.copy_(w0)
    v.copy_(v0)
    kept.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (w, v, kept)))
    want, _ = ev.accumulate(w0.double().cpu().numpy(), f64(q)[:, None], lse.double().cpu().numpy()[:, None], keys,
                            table, lens, [1, 1], 0.09)
    rows = ev.select_rows(want, table, lens, 200, 1, 8)
    assert (kept.cpu().numpy() == rows).mean() > 0.99  # fp32 sums may order close rows differently


def test_rows_past_32_bits_of_bytes():
    """Sums, selections and moves more than 4 GB into the caches."""
    nb, hkv = 20000, 8
    rng = np.random.default_rng(15)
    cache = torch.empty((nb, BS, hkv, D), dtype=torch.bfloat16, device="cuda")  # 5.2 GB
    w = torch.empty((nb, hkv, BS), device="cuda")
    table = np.array([[nb - 2, nb - 7]], dtype=np.int32)
    rows = torch.as_tensor(rng.standard_normal((2, BS, hkv, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    cache[torch.as_tensor(table[0].astype(np.int64)).cuda()] = rows
    q = torch.as_tensor(rng.standard_normal((1, 8, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    lse = torch.zeros((1, 8), device="cuda")
    api.paged_attention_decode(q, cache, cache, ints(table), ints([250]), 0.09, lse=lse)
    api.accumulate_attention_weights(w, q, lse, cache, ints(table), ints([250]), ints([250]), 0.09)
    kept = api.select_rows(w, ints(table), ints([250]), 60)
    torch.cuda.synchronize()
    small = rows.double().cpu().numpy()
    want, reach = ev.accumulate(np.zeros((2, hkv, BS)), f64(q)[:, None], lse.double().cpu().numpy()[:, None], small,
                                np.array([[0, 1]]), [250], [250], 0.09)
    check_weights(w[[nb - 2, nb - 7]], want * (np.arange(256).reshape(2, 1, BS) < 250) +
                  w[[nb - 2, nb - 7]].double().cpu().numpy() * (np.arange(256).reshape(2, 1, BS) >= 250), reach,
                  lse.cpu().numpy(), 1)
    got = w[[nb - 2, nb - 7]].cpu().numpy()
    np.testing.assert_array_equal(kept.cpu().numpy(), ev.select_rows(got, np.array([[0, 1]]), [250], 60))
    api.compact_rows(kept, ints(table), row_caches=[cache], head_caches=[w])
    torch.cuda.synchronize()
    after = cache[[nb - 2, nb - 7]].view(torch.int16).cpu().numpy()
    np.testing.assert_array_equal(after, ev.compact(rows.view(torch.int16).cpu().numpy(), kept.cpu().numpy(),
                                                    np.array([[0, 1]]), np.array([[0, 1]]), False))


def test_compact_rows_with_the_same_table_as_the_new_one():
    rng = np.random.default_rng(16)
    table, nb = make_table(rng, [600, 300])
    kept = ints(_kept(rng, 2, 2, [600, 300], 250))
    t = ints(table)
    cache = torch.as_tensor(rng.random((nb, 2, BS)), dtype=torch.float32).cuda()
    before = cache.cpu().numpy()
    api.compact_rows(kept, t, head_caches=[cache], new_block_table=t)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(cache.cpu().numpy(), ev.compact(before, kept.cpu().numpy(), table, table, True))


def test_two_evictions_at_once():
    """The calls have no workspace: two at once on streams of their own give what each gives alone."""
    rng = np.random.default_rng(17)
    jobs = []
    for lens, H, fmt in (([3000, 900], 8, "fp4"), ([2500, 128, 0, 700], 4, "bf16")):
        table, nb = make_table(rng, lens)
        cache, scale, _ = keys_of(fmt, rng, nb, 2)
        q = torch.as_tensor(rng.standard_normal((len(lens), H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
        lse = torch.full((len(lens), H), 4.0, device="cuda")
        w = torch.as_tensor(rng.random((nb, 2, BS)), dtype=torch.float32).cuda()
        kept = torch.zeros((len(lens), 2, 500), dtype=torch.int32, device="cuda")
        own = w.clone(), cache.clone(), kept
        jobs.append((own, (w, cache), q, lse, ints(table), ints(lens), ints([1] * len(lens)), scale, fmt))

    def evict(own, first, q, lse, t, n, fresh, scale, fmt, stream=None):
        w, cache, kept = own
        api.accumulate_attention_weights(w, q, lse, cache, t, n, fresh, 0.09, k_scale=scale, stream=stream)
        api.select_rows(w, t, n, 500, 2, 16, out=kept, stream=stream)
        api.compact_rows(kept, t, [cache] if fmt == "bf16" else [], [w] + ([cache] if fmt == "fp4" else []), stream=stream)

    def back(job):
        for t, x in zip(job[0], job[1]):
            t.copy_(x)
        job[0][2].zero_()

    alone = []
    for job in jobs:
        evict(*job)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in job[0]])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        for job in jobs:
            back(job)
        torch.cuda.synchronize()
        for job, stream in zip(jobs, streams):
            evict(*job, stream=stream)
        torch.cuda.synchronize()
        for job, want in zip(jobs, alone):
            assert all(torch.equal(a, b) for a, b in zip(job[0], want))


@pytest.mark.parametrize("kind", ["spread", "few", "one", "special", "close", "descending", "zeros"])
@pytest.mark.parametrize("per_sm,longest,keep,sink,recent", [(4, 4096, 500, 4, 100), (4, 4096, 2048, 0, 0), (4, 700, 1, 0, 0),
                                                             (2, 16384, 900, 1, 32), (2, 5000, 2500, 0, 7)])
def test_select_rows_of_many_short_sequences(kind, per_sm, longest, keep, sink, recent):
    """Enough rows for every kernel that takes short ones, against numpy's sort."""
    hkv = 8
    B = per_sm * torch.cuda.get_device_properties(0).multi_processor_count // hkv + 4
    rng = np.random.default_rng(longest + keep)
    lens = [longest, 0, keep, keep + 1, max(1, longest - 1)] + [int(n) for n in rng.integers(0, longest + 1, B - 5)]
    table, nb = make_table(rng, lens)
    w = _weights(rng, kind, nb, hkv)
    if kind == "descending":
        w[:] = -np.arange(BS) - BS * rng.permutation(nb)[:, None, None]
    elif kind == "zeros":
        w = np.where(rng.random(w.shape) < 0.01, rng.random(w.shape), 0.0).astype(np.float32)
    st = status()
    kept = api.select_rows(torch.as_tensor(np.ascontiguousarray(w)).cuda(), ints(table), ints(lens), keep, sink,
                           recent, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    got = kept.cpu().numpy()
    for b, m in enumerate(lens):
        rows = w[table[b, :-(-m // BS)]].transpose(1, 0, 2).reshape(hkv, -1)[:, :m]
        for g in range(hkv):
            row = rows[g]
            rank = np.where(np.isnan(row), 1, 2)
            rank[:sink] = rank[max(0, m - recent):] = 0
            weight = np.where(rank == 2, row, 0.0)
            want = np.sort(np.lexsort((np.arange(m), -weight, rank))[:keep])
            np.testing.assert_array_equal(got[b, g, :len(want)], want)
            assert (got[b, g, len(want):] == -1).all()
