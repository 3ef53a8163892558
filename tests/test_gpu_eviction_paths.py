"""Eviction calls directly behind the calls whose results they read (GPU)."""
import numpy as np
import pytest
import torch

from oracle import evict_ref as ev
from oracle import fp4_ref as f4
from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import PagedKVError
from tests.test_gpu_evict import D, check_weights, ints, keys_of, make_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
def test_weights_behind_a_decode_that_leaves_nothing_to_merge(fmt):
    """Sequences of a block each over a wide table: every segment is one CTA's, the merge has no work,
    and the next launch reads the log-sum-exps. The same bits as with a wait between the calls."""
    rng = np.random.default_rng(31)
    lens = [int(n) for n in rng.integers(1, 129, 40)]
    table, nb = make_table(rng, lens, width=20)
    cache, k_scale, _ = keys_of(fmt, rng, nb, 8)
    t, n, fresh = ints(table), ints(lens), ints(lens)
    steps = 20
    q = torch.as_tensor(rng.standard_normal((steps, 40, 8, D)), dtype=torch.float32).to(torch.bfloat16).cuda()

    def run(wait):
        w = torch.full((nb, 8, 128), float("nan"), device="cuda")
        lse = torch.full((40, 8), float("nan"), device="cuda")
        out = torch.empty((40, 8, D), device="cuda")
        got = []
        for i in range(steps):
            if fmt == "bf16":
                api.paged_attention_decode(q[i], cache, cache, t, n, 0.09, out=out, lse=lse)
            else:
                api.paged_attention_decode_fp4(q[i], cache, cache, k_scale, k_scale, t, n, 0.09, out=out, lse=lse)
            if wait:
                torch.cuda.synchronize()
            api.accumulate_attention_weights(w, q[i], lse, cache, t, n, fresh, 0.09, k_scale=k_scale)
            if wait:
                torch.cuda.synchronize()
            got.append(w.clone())
        torch.cuda.synchronize()
        return got

    calm = run(True)
    live = torch.zeros(calm[0].shape, dtype=torch.bool)
    for b, m in enumerate(lens):
        live[table[b, 0], :, :m] = True
    assert torch.isfinite(calm[-1].cpu()[live]).all()
    for _ in range(5):
        for a, b in zip(calm, run(False)):
            assert torch.equal(a.cpu()[live], b.cpu()[live])


# ------------------------------------------------------------------ tables as wide as positions are counted
WIDEST = (2**31 - 1) // 128  # blocks: positions up to 2,147,483,519


def test_decode_over_the_widest_table():
    """2^31 - 128 tokens in a table that names four blocks again and again, the last entries its last
    ones. Keys are zero, so every weight is equal and the sums are exact in fp32: an output is the mean of
    the blocks' values as the cache holds them (1 as 33 / 32), the log-sum-exp the length's logarithm."""
    cache = [torch.zeros((4, 1, 128, w), dtype=torch.uint8, device="cuda") for w in (64, 64, 8, 8)]
    v = torch.arange(4, dtype=torch.bfloat16, device="cuda").repeat_interleave(128).view(512, 1, 1).expand(512, 1, D)
    api.kv_cache_write_fp4(*cache, torch.zeros_like(v).contiguous(), v.contiguous(), ints(np.arange(512)))
    table = torch.arange(WIDEST, dtype=torch.int32, device="cuda").remainder_(4).view(1, WIDEST)
    q = torch.ones((1, 8, D), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros((1, 8), device="cuda")
    out = api.paged_attention_decode_fp4(q, *cache, table, ints([WIDEST * 128]), 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    held = f4.dequantise(*f4.quantise(np.arange(4.0)[:, None].repeat(D, 1)))[:, 0]
    mean = held @ np.bincount(np.arange(WIDEST) % 4) / WIDEST
    # A warp's sums are multiples of 2^11 below 2^35 (exact or off by 2^-24 a step of some 27,600, each way);
    # then 16 warps and 152 CTAs are joined.
    assert (out.double().cpu() - mean).abs().max() <= 28000 * 2.0 ** -24 * 3
    assert (lse.double().cpu() - np.log(WIDEST * 128.0)).abs().max() <= 28000 * 2.0 ** -24


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_weights_over_the_widest_table(fmt):
    """A sequence of 2^31 - 128 positions of which only the last block exists."""
    rng = np.random.default_rng(33)
    cache, k_scale, keys = keys_of(fmt, rng, 2, 1)
    table = torch.full((1, WIDEST), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.as_tensor(rng.standard_normal((1, 8, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    z = 0.09 * (keys[1, :, 0] @ q[0].double().cpu().numpy().T)  # [128, 8]
    lse = torch.full((1, 8), 3.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 1, 128), device="cuda")
    api.accumulate_attention_weights(w, q, lse, cache, table, ints([WIDEST * 128]), ints([1]), 0.09, k_scale=k_scale,
                                     dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 and not w[0].any()
    # Relative error: see the module whose helpers these are; |z| and |lse| are below 16 together.
    np.testing.assert_allclose(w[1, 0].double().cpu().numpy(), np.exp(z - 3.0).sum(-1), rtol=1e-4)


@pytest.mark.parametrize("fmt,H,Q", [("bf16", 1, 1), ("bf16", 3, 4), ("fp8", 5, 4), ("fp4", 5, 4)])
def test_first_weights_of_the_widest_table(fmt, H, Q):
    """The same with the first block alone, for query rows that do not fill the products' 8 columns: what
    fills them counts for nothing, however far the last position is."""
    rng = np.random.default_rng(34)
    cache, k_scale, keys = keys_of(fmt, rng, 2, 1)
    table = torch.full((1, WIDEST), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 1
    q = torch.as_tensor(rng.standard_normal((1, Q, H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    z = 0.09 * (keys[1, :, 0] @ q.double().cpu().numpy().reshape(Q * H, D).T)
    lse = torch.full((1, Q, H), 3.0, device="cuda")
    w = torch.zeros((2, 1, 128), device="cuda")
    api.accumulate_attention_weights(w, q, lse, cache, table, ints([WIDEST * 128]), ints([1]), 0.09, k_scale=k_scale)
    torch.cuda.synchronize()
    assert not w[0].any()
    np.testing.assert_allclose(w[1, 0].double().cpu().numpy(), np.exp(z - 3.0).sum(-1), rtol=1e-4)


# ------------------------------------------------------------------ runs of many pieces
def reference(w0, q, lse, keys, table, lens, fresh, scale, decay):
    """Sums after a step and the reach of their scores (see test_gpu_evict.py), a sequence at a time in
    float64. q [B, Q, H, d], lse [B, Q, H], keys [nb, 128, H_kv, d]; entries outside the cache are skipped."""
    out, reach = w0.astype(np.float64), np.zeros(w0.shape)
    nb, hkv = w0.shape[:2]
    B, Q, H, _ = q.shape
    for b, n in enumerate(lens):
        p = np.arange(n)
        blk = table[b, p // 128]
        p, blk = p[(blk >= 0) & (blk < nb)], blk[(blk >= 0) & (blk < nb)]
        rows = keys[blk, p % 128]                                           # [n, H_kv, d]
        qq = q[b].reshape(Q, hkv, H // hkv, D)
        z = scale * np.einsum("qghd,ngd->ngqh", qq, rows)
        mag = scale * np.einsum("qghd,ngd->ngqh", np.abs(qq), np.abs(rows)).max(axis=(2, 3))
        seen = p[:, None] <= n - Q + np.arange(Q)                            # [n, Q]
        e = np.exp(z - lse[b].reshape(Q, hkv, H // hkv).swapaxes(0, 1)) * seen[:, None, :, None]
        old = np.where(p >= n - min(max(int(fresh[b]), 0), n), 0.0, decay)
        at = blk[:, None], np.arange(hkv)[None], (p % 128)[:, None]
        out[at] = old[:, None] * out[at] + e.sum(axis=(2, 3))
        reach[at] = mag
    return out, reach


def check_step(fmt, rng, lens, H, hkv, Q, table, nb, decay=0.75, code=0):
    cache, k_scale, keys = keys_of(fmt, rng, nb, hkv)
    q = torch.as_tensor(rng.standard_normal((len(lens), Q, H, D)), dtype=torch.float32).to(torch.bfloat16).cuda()
    lse = torch.as_tensor(3 + rng.random((len(lens), Q, H)), dtype=torch.float32).cuda()
    w0 = rng.random((nb, hkv, 128)).astype(np.float32)
    fresh = [n if b % 5 == 0 else b % 5 + Q for b, n in enumerate(lens)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        w = torch.as_tensor(w0).cuda()
        api.accumulate_attention_weights(w, q, lse, cache, ints(table), ints(lens), ints(fresh), 0.09,
                                         k_scale=k_scale, decay=decay, dev_status=st)
        torch.cuda.synchronize()
        got.append(w)
    assert int(st) == code and torch.equal(*got)
    l64 = lse.double().cpu().numpy()
    want, reach = reference(w0, q.double().cpu().numpy(), l64, keys, table, lens, fresh, 0.09, decay)
    check_weights(got[0], want, reach, l64, Q * H // hkv)
    behind = want == w0
    assert np.array_equal(got[0].cpu().numpy()[behind], w0[behind])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("H,Q", [(8, 1), (16, 2), (64, 1), (64, 2)])
def test_weights_of_many_sequences(fmt, H, Q):
    """Some fifteen blocks for every CTA: rings that are refilled, runs that pass from sequence to
    sequence and from kv head to kv head."""
    rng = np.random.default_rng(35)
    lens = [int(n) for n in rng.integers(0, 1500, 90)] + [9000]
    table, nb = make_table(rng, lens)
    check_step(fmt, rng, lens, H, 4, Q, table, nb)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("hkv", [1, 4])
def test_weights_of_runs_that_pass_many_blocks(fmt, hkv):
    """A sequence of ten million positions of which 300 blocks exist: a warp's run is longer than the 32
    table entries that it holds at a time."""
    rng = np.random.default_rng(36)
    width, exist = 84_000 // hkv, 300
    at = np.sort(np.r_[rng.choice(width - 1, exist - 1, replace=False), width - 1])
    table = np.full((1, width), -1, dtype=np.int32)
    table[0, at] = rng.permutation(exist + 2)[:exist]
    check_step(fmt, rng, [width * 128 - 5], 8 * hkv, hkv, 1, table, exist + 2, code=2)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("H,hkv,Q", [(16, 1, 9), (32, 2, 17), (20, 2, 14), (3, 3, 129)])
def test_weights_of_more_rows_than_one_launch_takes(fmt, H, hkv, Q):
    """The second launch adds to what the first one left, with no decay and no fresh start of its own,
    whichever kernel its rows fall to."""
    rng = np.random.default_rng(37)
    lens = [300, 7, 0, 900, 128, 1]
    table, nb = make_table(rng, lens)
    check_step(fmt, rng, lens, H, hkv, Q, table, nb)


# ------------------------------------------------------------------ selections and moves at their limits
@pytest.mark.parametrize("kind", ["spread", "narrow", "levels"])
@pytest.mark.parametrize("n,keep,sink,recent", [(4_194_304, 300_000, 4, 100), (4_194_303, 4_194_300, 0, 2),
                                                (3_999_000, 1, 0, 0)])
def test_selection_from_the_longest_sequence(kind, n, keep, sink, recent):
    """The widest table of a selection, against numpy's stable sort."""
    rng = np.random.default_rng(keep)
    nb = 32768
    table = rng.permutation(nb).astype(np.int32)[None]
    if kind == "spread":
        w = np.exp(2.5 * rng.standard_normal((nb, 1, 128)) - 8).astype(np.float32)
    elif kind == "narrow":  # all in one bin of the selection's first digit
        w = (1.0 + 0.1 * rng.random((nb, 1, 128))).astype(np.float32)
    else:
        w = rng.integers(0, 5, (nb, 1, 128)).astype(np.float32)
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints([n]), keep, sink, recent)
    torch.cuda.synchronize()
    row = w[table[0], 0].reshape(-1)[:n]
    always = np.r_[0:sink, n - recent:n]
    ranked = np.arange(sink, n - recent)
    best = ranked[np.argsort(-row[ranked], kind="stable")[:keep - sink - recent]]
    np.testing.assert_array_equal(kept.cpu().numpy()[0, 0], np.sort(np.r_[always, best]))


@pytest.mark.parametrize("kind", ["narrow", "uniform"])
@pytest.mark.parametrize("B,width", [(3, 2048), (70, 300)])
def test_selection_behind_a_table_wider_than_its_rows(kind, B, width):
    """Clusters by the table's width, rows of a few blocks: most of a cluster's CTAs have none."""
    rng = np.random.default_rng(B)
    lens = [0, 128, 1] + [int(n) for n in rng.integers(1, 3000, B - 3)]
    table, nb = make_table(rng, lens, width=width)
    w = (rng.random((nb, 2, 128)) * (0.01 if kind == "narrow" else 1.0) + 1.0 * (kind == "narrow")).astype(np.float32)
    kept = api.select_rows(torch.as_tensor(w).cuda(), ints(table), ints(lens), 100, 1, 5).cpu().numpy()
    for b, n in enumerate(lens):
        for g in range(2):
            row = w[table[b, :-(-n // 128)], g].reshape(-1)[:n]
            want = np.arange(n)
            if n > 100:
                mid = np.arange(1, n - 5)
                want = np.sort(np.r_[0, n - 5:n, mid[np.argsort(-row[mid], kind="stable")[:94]]])
            np.testing.assert_array_equal(kept[b, g, :len(want)], want)
            assert (kept[b, g, len(want):] == -1).all()


@pytest.mark.parametrize("own_blocks", [False, True])
def test_moves_of_sixteen_caches_and_of_the_longest_rows(own_blocks):
    rng = np.random.default_rng(41)
    lens, hkv, keep = [400, 129], 2, 150
    table, nb = make_table(rng, lens, nb_more=5)
    new = None
    if own_blocks:
        new = rng.permutation(np.setdiff1d(np.arange(nb), table))[:4].reshape(2, 2).astype(np.int32)
    kept = np.full((2, hkv, keep), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for g in range(hkv):
            m = min(n, keep)
            kept[b, g, :m] = np.sort(rng.choice(n, m, replace=False))
    widths = [16384, 16383, 1026, 257, 1, 2, 3, 5]  # of 4 bytes
    row = [torch.as_tensor(rng.integers(0, 2**31, (nb, 128, hkv, x), dtype=np.int32)).cuda() for x in widths]
    head = [torch.as_tensor(rng.integers(0, 2**31, (nb, hkv, 128, x), dtype=np.int32)).cuda() for x in widths]
    before = [t.cpu().numpy() for t in row + head]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.compact_rows(ints(kept), ints(table), row, head, None if new is None else ints(new), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for i, t in enumerate(row + head):
        want = ev.compact(before[i], kept, table, table if new is None else new, i >= len(row))
        assert np.array_equal(t.cpu().numpy(), want), i
    with pytest.raises(PagedKVError, match="16 caches"):
        api.compact_rows(ints(kept), ints(table), row, [*head, torch.zeros((nb, hkv, 128), device="cuda")])
