"""GPU parity of block-sparse decode: key summaries, block selection and attention over the
selected blocks, against the float64 oracle.

Summaries are minima and maxima of bf16 values: compared bit for bit. Selections are whole
numbers: equal. Attention: the weights enter the value product rounded to bf16 (off by at
most 2^-8 of themselves) and divide by the sum of the same rounded weights, so an output
moves by at most 2^-8 / (1 - 2^-8) sum_j p_j |v_j - o|; the fp32 scores (128 products of
magnitude a few, summed in fp32: below 1e-4 for these inputs) add at most 2e-4 of that sum,
and the fp32 sums and the output's own rounding (2^-24, bf16 2^-8) come on top."""
import numpy as np
import pytest
import torch

import synth
from oracle import sparse_ref as sp
from oracle.paged_ref import bf16_bits_to_f64
from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import PagedKVError
from tests.gpu_cases import LSE_TOL

pytestmark = pytest.mark.gpu

BS, D = 128, 128


def f64(t):
    return bf16_bits_to_f64(synth.bf16_bits(t.contiguous()))


def make_table(rng, lens, width=None, nb=None):
    need = [-(-int(n) // BS) for n in lens]
    nb = nb or sum(need) + 1
    order = 1 + rng.permutation(nb - 1)
    table = np.zeros((len(need), width or max(1, max(need))), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, nb


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ summaries
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_summaries_follow_a_growing_cache(Hkv):
    """Prefill chunks, single rows, rows that end on and cross block edges, idle sequences."""
    rng = np.random.default_rng(Hkv)
    final = np.array([700, 130, 1, 513, 0])
    table, nb = make_table(rng, final)
    k = torch.randn((nb, BS, Hkv, D), device="cuda").to(torch.bfloat16)
    s = torch.full((nb, Hkv, 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    want = f64(s)
    steps = [[100, 127, 0, 1, 0], [28, 1, 1, 16, 0], [1, 1, 0, 17, 0], [129, 0, 0, 350, 0],
             [442, 1, 0, 129, 0]]
    assert np.array_equal(np.sum(steps, axis=0), final)
    lens, st = np.zeros(5, dtype=np.int64), status()
    for n, step in enumerate(steps):
        lens = lens + step
        api.update_block_summaries(s, k, ints(table), ints(lens), ints(step), max(step) + 50 * (n == 3),
                                   dev_status=st)
        want = sp.update_summaries(want, synth.bf16_bits(k), table, lens, step, BS)
        assert np.array_equal(f64(s), want), n
    assert int(st.item()) == 0


def test_summaries_take_special_values_and_skip_unwritten_rows():
    rng = np.random.default_rng(7)
    table, nb = make_table(rng, [200])
    k = torch.full((nb, BS, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # unwritten
    for pos in range(200):
        k[int(table[0, pos // BS]), pos % BS] = torch.randn((2, D), device="cuda").to(torch.bfloat16)
    first, second = (int(x) for x in table[0])
    k[first, 3, 0, 5] = float("inf")
    k[first, 4, 0, 6] = float("-inf")
    k[first, 5, 1, 7] = float("nan")
    k[second, 70, 1, 0] = 1e-40  # a subnormal minimum among zeros
    k[second, :70, 1, 0] = 0.0
    k[second, 71, 1, 0] = -1e-40
    s = torch.zeros((nb, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    # Two steps, so that the second block's summary is merged once.
    for lens, new in (([150], [150]), ([200], [50])):
        api.update_block_summaries(s, k, ints(table), ints(lens), ints(new), 150)
    got = f64(s)
    want = sp.update_summaries(np.zeros((nb, 2, 2, D)), synth.bf16_bits(k), table, [200], [200], BS)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[first, 1, :, 7]).all() and np.isnan(got).sum() == 2
    assert got[first, 0, 1, 5] == np.inf and got[first, 0, 0, 6] == -np.inf
    assert got[second, 1, 0, 0] < 0 < got[second, 1, 1, 0]


def test_summaries_flag_bad_lengths_and_blocks_and_leave_them():
    rng = np.random.default_rng(8)
    lens = np.array([300, 300, 300, 300, 300])
    table, nb = make_table(rng, lens)
    k = torch.randn((nb, BS, 2, D), device="cuda").to(torch.bfloat16)
    good, st = sp.update_summaries(np.full((nb, 2, 2, D), 9.0), synth.bf16_bits(k), table, lens,
                                   [300, 0, 0, 0, 0], BS), status()
    for what, lens2, new, bit in (
            ("more new rows than max_new", lens, [300, 301, 0, 0, 0], 4),
            ("more new rows than rows", [300, 5, 300, 300, 300], [300, 6, 0, 0, 0], 4),
            ("negative", lens, [300, 0, -1, 0, 0], 4),
            ("longer than the table", [300, 300, 300, 385, 300], [300, 0, 0, 1, 0], 4)):
        s = torch.full((nb, 2, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        st.zero_()
        api.update_block_summaries(s, k, ints(table), ints(lens2), ints(new), 300, dev_status=st)
        assert int(st.item()) == bit and np.array_equal(f64(s), good), what
    bad = table.copy()
    bad[4, 0], bad[4, 1] = nb, -3
    s = torch.full((nb, 2, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    st.zero_()
    api.update_block_summaries(s, k, ints(bad), ints(lens), ints([300, 0, 0, 0, 300]), 300, dev_status=st)
    want = good.copy()
    want[table[4, 2]] = sp.update_summaries(np.full((nb, 2, 2, D), 9.0), synth.bf16_bits(k), table,
                                            lens, [0, 0, 0, 0, 300], BS)[table[4, 2]]
    assert int(st.item()) == 2 and np.array_equal(f64(s), want)


def test_a_forked_request_copies_its_summaries_with_its_blocks():
    k = torch.randn((4, BS, 2, D), device="cuda").to(torch.bfloat16)
    s = torch.zeros((4, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    api.update_block_summaries(s, k, ints([[1]]), ints([50]), ints([50]), 50)
    for cache in (k, s):  # the incomplete block 1 becomes block 3 of a child
        api.copy_blocks(cache, ints([1]), ints([3]))
    k[3, 50] = torch.randn((2, D), device="cuda").to(torch.bfloat16)
    api.update_block_summaries(s, k, ints([[3]]), ints([51]), ints([1]), 1)
    rows = f64(k)[3, :51]
    assert np.array_equal(f64(s)[3, :, 0], rows.min(0)) and np.array_equal(f64(s)[3, :, 1], rows.max(0))


# ------------------------------------------------------------------ selection
def random_summaries(rng, nb, hkv, scale=1.0):
    a = torch.from_numpy(rng.standard_normal((nb, hkv, 2, D)) * scale).to(torch.bfloat16).cuda()
    return torch.stack([torch.minimum(a[:, :, 0], a[:, :, 1]), torch.maximum(a[:, :, 0], a[:, :, 1])], 2)


def check_select(q, s, table, lens, K, sink=0, recent=1, bit=0):
    st = status()
    got = api.select_blocks(q, s, ints(table), ints(lens), K, sink, recent, dev_status=st)
    q4 = f64(q) if q.dim() == 4 else f64(q)[:, None]
    want = sp.select_blocks(q4, f64(s), table, lens, K, sink, recent, BS)
    assert np.array_equal(got.cpu().numpy().reshape(want.shape), want)
    assert int(st.item()) == bit
    return want


@pytest.mark.parametrize("q_len,H,Hkv,K,sink,recent", [
    (1, 8, 2, 4, 0, 1), (1, 3, 3, 1, 0, 0), (2, 16, 1, 7, 1, 2), (4, 12, 4, 3, 2, 1),
    (1, 10, 2, 5, 0, 5), (3, 4, 2, 6, 6, 0),
])
def test_selection_matches_oracle(q_len, H, Hkv, K, sink, recent):
    rng = np.random.default_rng(K * 31 + H)
    lens = np.array([0, 1, 128, 129, K * 128, K * 128 + 1, 9 * 128 + 5, 2500])
    table, nb = make_table(rng, lens)
    q = torch.from_numpy(rng.standard_normal((8, q_len, H, D))).to(torch.bfloat16).cuda()
    q = q[:, 0].contiguous() if q_len == 1 else q
    check_select(q, random_summaries(rng, nb, Hkv), table, lens, K, sink, recent)


@pytest.mark.parametrize("B,width,n", [(1, 70, 70), (3, 130, 129), (1, 600, 513), (40, 70, 66)])
def test_selection_over_clusters_of_every_width(B, width, n):
    """Tables wide enough for 2 to 8 CTAs a row, rows of them that end inside a round."""
    rng = np.random.default_rng(width)
    lens = rng.integers((n - 5) * BS, n * BS + 1, B)
    table, nb = make_table(rng, lens, width)
    q = torch.from_numpy(rng.standard_normal((B, 2, D))).to(torch.bfloat16).cuda()
    check_select(q, random_summaries(rng, nb, 1), table, lens, 33, 1, 1)


def test_selection_of_short_rows_under_a_wide_table():
    """A table as wide as the model's context: rows far shorter than it, of every length around
    the limit of one CTA, next to long ones."""
    rng = np.random.default_rng(9)
    lens = np.array([300, 256 * BS, 257 * BS, 258 * BS + 1, 259 * BS, 1, 0, 700 * BS])
    table, nb = make_table(rng, lens, 8192)
    for H in (1, 8):
        q = torch.from_numpy(rng.standard_normal((8, H, D))).to(torch.bfloat16).cuda()
        check_select(q, random_summaries(rng, nb, 1), table, lens, 5, 1, 1)


def _torch_select(q, s, table, lens, K, recent=1):
    """The selection of large cases: fp64 scores on the GPU (sums exact for these inputs)."""
    B, H, _ = q.shape
    hkv = s.shape[1]
    x = q.double().view(B, hkv, H // hkv, D)
    w = torch.cat([x.clamp(max=0).sum(2), x.clamp(min=0).sum(2)], -1)
    out = torch.full((B, hkv, K), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        n = -(-int(lens[b]) // BS)
        score = torch.einsum("gd,jgd->gj", w[b], s[table[b, :n].long()].double().flatten(-2))
        score[:, n - recent:] = torch.inf
        idx = score.sort(dim=-1, descending=True, stable=True).indices[:, :K]
        out[b, :, :min(n, K)] = idx.sort(-1).values.to(torch.int32)
    return out


def test_selection_of_the_long_context_batch_and_of_a_million_tokens():
    rng = np.random.default_rng(2)
    for B, hi, H, Hkv, K in ((64, 32768, 64, 8, 32), (2, 1048576, 32, 8, 128)):
        lens = rng.integers(1, hi + 1, B)
        lens[0] = hi
        table, nb = make_table(rng, lens)
        s = random_summaries(rng, nb, Hkv)
        q = torch.from_numpy(rng.standard_normal((B, H, D))).to(torch.bfloat16).cuda()
        t = ints(table)
        got = api.select_blocks(q, s, t, ints(lens), K)
        assert torch.equal(got, _torch_select(q, s, t, lens, K))


def test_selection_decides_ties_and_near_ties_as_in_64_bits():
    rng = np.random.default_rng(3)
    n, K = 40, 9
    table, nb = make_table(rng, [n * BS])
    q = torch.ones((1, 4, D), dtype=torch.bfloat16, device="cuda")
    # All blocks equal: the lowest are taken.
    s = torch.ones((nb, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    assert check_select(q, s, table, [n * BS], K, 0, 0)[0, 0, 0].tolist() == list(range(K))
    # Equal but for one channel that a query weight of 2^-30 brings below fp32's reach.
    q[:, :, 0] = 2.0 ** -30
    s[:, :, :, 0] = torch.from_numpy(rng.permutation(nb)).to(torch.bfloat16).cuda()[:, None, None]
    want = check_select(q, s, table, [n * BS], K, 0, 0)
    best = np.argsort(-s[table[0], 0, 1, 0].float().cpu().numpy(), kind="stable")[:K]
    assert sorted(best) == want[0, 0, 0].tolist()
    # Small whole numbers: many exact ties across the border.
    s = torch.from_numpy(rng.integers(-1, 2, (nb, 2, 2, D)).astype(np.float64))
    s[:, :, :, 2:] = 0
    s = s.sort(dim=2).values.to(torch.bfloat16).cuda()
    q = torch.ones((1, 4, D), dtype=torch.bfloat16, device="cuda")
    check_select(q, s, table, [n * BS], K)
    # A zero query: every score is zero.
    q.zero_()
    assert check_select(q, s, table, [n * BS], K, 0, 1)[0, 0, 0].tolist() == [*range(K - 1), n - 1]


@pytest.mark.parametrize("n,width,H", [(300, 300, 2), (600, 640, 1), (2000, 2000, 4), (1100, 8192, 1)])
def test_selection_by_a_cluster_decides_ties_and_special_values(n, width, H):
    """Rows of more blocks than one CTA selects: ties by the hundred across the border and the
    CTAs, all blocks equal, near ties, NaN, infinities, zero queries, bad blocks."""
    rng = np.random.default_rng(n)
    lens = np.array([n * BS, n * BS - 200])
    table, nb = make_table(rng, lens, width)
    q = torch.ones((2, H, D), dtype=torch.bfloat16, device="cuda")
    s = torch.ones((nb, 1, 2, D), dtype=torch.bfloat16, device="cuda")
    assert check_select(q, s, table, lens, 50, 0, 0)[0, 0, 0].tolist() == list(range(50))
    for K in (1, 33, n // 2, n - 4):
        whole = torch.from_numpy(rng.integers(-1, 2, (nb, 1, 2, D)).astype(np.float64))
        whole[..., 3:] = 0
        check_select(q, whole.sort(dim=2).values.to(torch.bfloat16).cuda(), table, lens, K, 0, 1)
    s[:, :, :, 0] = torch.from_numpy(rng.permutation(nb) % 200).to(torch.bfloat16).cuda()[:, None, None]
    q[:, :, 0] = 2.0 ** -30  # differences that fp32 sums cannot see
    check_select(q, s, table, lens, 70, 1, 2)
    s = random_summaries(rng, nb, 1)
    check_select(torch.zeros_like(q), s, table, lens, 40, 0, 1)
    bad = table.copy()
    bad[0, ::7], bad[1, 5] = -1, nb
    check_select(q, s, bad, lens, n - 60, 2, 2, bit=2)
    t = table[0]
    s[int(t[n - 9]), 0, 1, 3] = float("inf")
    s[int(t[9]), 0, 0, 4] = float("nan")
    with np.errstate(invalid="ignore"):
        want = check_select(q, s, table, lens, 20, 0, 0)
    assert {9, n - 9} <= set(want[0, 0, 0])


@pytest.mark.parametrize("B,Hkv,n,H", [(64, 8, 1500, 8), (16, 8, 2500, 32), (39, 8, 5000, 16),
                                       (40, 8, 8192, 8), (4, 1, 8192, 2)])
def test_selection_of_many_long_rows(B, Hkv, n, H):
    """Runs of thousands of blocks per CTA, with as many rows as leave a row one CTA or a few.
    The rows share their blocks; small whole numbers tie by the thousand."""
    rng = np.random.default_rng(n)
    nb = 9000
    table = rng.integers(0, nb, (B, n)).astype(np.int32)
    lens = rng.integers((n - 200) * BS, n * BS + 1, B)
    lens[-1] = n * BS
    t = ints(table)
    q = torch.from_numpy(rng.standard_normal((B, H, D))).to(torch.bfloat16).cuda()
    g = torch.Generator(device="cuda").manual_seed(n)
    s = torch.randn((nb, Hkv, 2, D), generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    whole = torch.randint(-1, 2, (nb, Hkv, 2, D), generator=g, device="cuda").sort(dim=2).values
    whole[..., 3:] = 0
    for K in (1, 64, n // 2):
        assert torch.equal(api.select_blocks(q, s, t, ints(lens), K), _torch_select(q, s, t, lens, K))
        q1, w = torch.ones_like(q), whole.to(torch.bfloat16)
        assert torch.equal(api.select_blocks(q1, w, t, ints(lens), K), _torch_select(q1, w, t, lens, K))


@pytest.mark.parametrize("n", [40, 256, 700, 3000])
@pytest.mark.parametrize("power", [-8, -13, -20, -28, -36, -42])
def test_selection_at_borders_of_every_closeness(n, power):
    """Scores that differ from their neighbours by steps between fp32's reach and that of 64 bits
    (whole sums below 2^9 and steps of 2^-41 are exact in 53 bits; random scores of bf16 values are
    rounded by less than 2^-42 in any order): in twos, so that borders between equals occur too."""
    rng = np.random.default_rng(n - power)
    table, nb = make_table(rng, [n * BS])
    q = torch.ones((1, 2, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0 ** power
    base = torch.randint(-1, 2, (nb, 1, 1, D), generator=torch.Generator().manual_seed(n))
    base[..., 4:] = 1
    s = base.expand(nb, 1, 2, D).to(torch.bfloat16).cuda().contiguous()
    s[..., 0] = torch.from_numpy(rng.permutation(nb) // 2 % 100).to(torch.bfloat16).cuda()[:, None, None]
    for K in (1, 7, 20, n // 3, n // 2):
        check_select(q, s, table, [n * BS], K, 0, 0)
    for K in (5, n // 4):  # and among random scores
        s = random_summaries(rng, nb, 1)
        s[nb // 2:] = s[:nb - nb // 2].clone()
        s[nb // 2:, :, :, 0] += 2.0
        check_select(q, s, table, [n * BS], K, 0, 1)


def check_rows(q, s, table, lens, K, sink=0, recent=1, bit=0):
    """Every query row as it is selected by itself (with the sequence's length up to that row)."""
    st, Q = status(), q.shape[1]
    got = api.select_blocks(q, s, ints(table), ints(lens), K, sink, recent, dev_status=st)
    assert int(st.item()) == bit
    for i in range(Q):
        alone = api.select_blocks(q[:, i].contiguous(), s, ints(table), ints(np.maximum(lens - Q + 1 + i, 0)),
                                  K, sink, recent)
        assert torch.equal(got[:, i], alone), i


@pytest.mark.parametrize("q_len,H,Hkv,n,check", [
    (2, 2, 1, 263, check_select), (3, 2, 1, 261, check_select), (2, 8, 8, 1300, check_rows),
    (5, 4, 1, 2100, check_rows), (4, 32, 8, 5000, check_rows), (2, 16, 8, 8192, check_rows)])
def test_selection_of_several_query_rows_over_long_tables(q_len, H, Hkv, n, check):
    """Neighbouring query rows that see the same blocks, or one block more, up to the limits where
    a row has nothing to choose and where one warp selects it; ties, bad blocks, infinities."""
    rng = np.random.default_rng(n)
    K = 9
    lens = np.array([n * BS, (n - 1) * BS + 1, (n - 1) * BS, 258 * BS + 1, 257 * BS + 1, K * BS + 1, K * BS, 3, 0])
    width = 5000 if n == 261 else n
    nb = 4000
    table = rng.integers(0, nb, (len(lens), width)).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn((len(lens), q_len, H, D), generator=g, device="cuda").to(torch.bfloat16)
    s = torch.randn((nb, Hkv, 2, D), generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    check(q, s, table, lens, K)
    check(q, s, table, lens, 140, 2, 3)
    for sink, recent in ((0, 0), (4, 5)):  # (the last leaves no place to choose)
        check(q, s, table, lens, K, sink, recent)
    q[:, q_len - 1] = 0  # all of one row's scores are equal
    check(q, s, table, lens, K)
    q[:, 1] = 1
    whole = torch.randint(-1, 2, (nb, Hkv, 2, D), generator=g, device="cuda").sort(dim=2).values
    whole[..., 2:] = 0
    check(q, whole.to(torch.bfloat16), table, lens, 60, 1, 1)
    s[7, 0, 1, 3], s[8, 0, 0, 9] = float("inf"), float("nan")
    bad = table.copy()
    bad[:, 1::9] = nb
    with np.errstate(invalid="ignore"):
        check(q, s, bad, lens, 40, bit=2)


def test_selections_over_long_tables_at_once_and_in_a_graph():
    """Clusters of different widths and shared memory on two streams at a time; replays follow the
    lengths and queries in their buffers."""
    rng = np.random.default_rng(12)
    nb = 3000
    g = torch.Generator(device="cuda").manual_seed(12)
    s = torch.randn((nb, 2, 2, D), generator=g, device="cuda").sort(dim=2).values.to(torch.bfloat16)
    cases = []
    for B, n, K in ((1, 8192, 100), (120, 2100, 20), (3, 300, 7)):
        q = torch.randn((B, 4, D), generator=g, device="cuda").to(torch.bfloat16)
        t = ints(rng.integers(0, nb, (B, n)))
        lens = ints(rng.integers(1, n * BS + 1, B))
        out = torch.empty((B, 2, K), dtype=torch.int32, device="cuda")
        cases.append((q, t, lens, K, out))

    def check():
        for q, t, lens, K, out in cases:
            assert torch.equal(out, _torch_select(q, s, t, lens, K))
            out.zero_()

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (q, t, lens, K, out) in enumerate(cases):
            api.select_blocks(q, s, t, lens, K, out=out, stream=streams[i % 2])
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for q, t, lens, K, out in cases:
            api.select_blocks(q, s, t, lens, K, out=out)
    for _ in range(2):
        graph.replay()
        check()
        for q, t, lens, K, out in cases:
            q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
            lens.copy_(ints(rng.integers(1, t.shape[1] * BS + 1, len(lens))))


def test_blocks_past_four_gigabytes():
    """A cache whose last blocks lie beyond 2^32 bytes: summaries, selection, attention, the
    rotary write and the FP8 read give what a small cache of the same blocks gives."""
    nb, Hkv, H, n = 16500, 8, 16, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    small = [torch.randn((n + 1, BS, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    big = [torch.empty((nb, BS, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = nb - n + torch.arange(n, device="cuda", dtype=torch.int32)
    near = 1 + torch.arange(n, device="cuda", dtype=torch.int32)
    for b, x in zip(big, small):
        b[nb - n:] = x[1:]
    # The rows of the first block are written through the rotary write.
    q, k, v = (torch.randn((BS, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv))
    angle = torch.rand((BS, D // 2), generator=g, device="cuda")
    rope = torch.cat([angle.cos(), angle.sin()], 1)
    row = torch.arange(BS, device="cuda", dtype=torch.int32)
    lens, new = ints([n * BS - 40]), ints([n * BS - 40])
    results = []
    for (kc, vc), t in ((small, near), (big, far)):
        st = status()
        rotated = api.rope_kv_cache_write(kc, vc, q, k, v, rope, row, int(t[0]) * BS + row, dev_status=st)
        s = torch.zeros((kc.shape[0], Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
        api.update_block_summaries(s, kc, t.view(1, n), lens, new, int(new), dev_status=st)
        idx = api.select_blocks(rotated[:1], s, t.view(1, n), lens, 5, dev_status=st)
        out = api.paged_attention_decode_sparse(rotated[:1], kc, vc, t.view(1, n), lens, idx, D ** -0.5,
                                                dev_status=st)
        assert int(st.item()) == 0
        results.append([rotated, s[t.long()], idx, out, kc[t.long()], vc[t.long()]])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    del big, kc, vc
    nb = 33000  # blocks of half the bytes
    codes = [torch.empty((nb, BS, Hkv, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty((nb, Hkv, BS), device="cuda") for _ in range(2)]
    slots = (nb - 1) * BS + row
    st = status()
    api.rope_kv_cache_write_fp8(*codes, *scales, q, k, v, rope, row, slots, dev_status=st)
    got = api.kv_cache_read_fp8(*codes, *scales, slots, dev_status=st)
    last = [c[-1:].clone() for c in codes] + [c[-1:].clone() for c in scales]
    want = api.kv_cache_read_fp8(*last, row, dev_status=st)
    other = [torch.empty_like(x) for x in last]
    api.rope_kv_cache_write_fp8(*other, q, k, v, rope, row, row, dev_status=st)
    assert int(st.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(last, other):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_selection_with_special_values():
    rng = np.random.default_rng(4)
    n, K = 30, 6
    table, nb = make_table(rng, [n * BS])
    q = torch.from_numpy(rng.standard_normal((1, 4, D))).to(torch.bfloat16).cuda()
    s = random_summaries(rng, nb, 2)
    t = table[0]
    s[int(t[7]), 0, 1, 3] = float("inf")
    s[int(t[9]), 0, 0, 4] = float("-inf")
    s[int(t[11]), 0, 0, 5] = float("nan")
    with np.errstate(invalid="ignore"):
        want = check_select(q, s, table, [n * BS], K)
    assert {7, 9, 11} <= set(want[0, 0, 0])
    # Values near the largest and the smallest of the type: sums past fp32's range.
    big = random_summaries(rng, nb, 2, 2.0 ** 126)
    check_select(q * 64, big, table, [n * BS], K)
    tiny = random_summaries(rng, nb, 2, 2.0 ** -132)  # subnormal bf16
    check_select(q, tiny, table, [n * BS], K)
    check_select((q * 2.0 ** -130).contiguous(), big, table, [n * BS], K)
    # Subnormal queries against keys near the largest value: products of ordinary size.
    q_tiny = torch.from_numpy(rng.standard_normal((1, 4, D)) * 2.0 ** -131).to(torch.bfloat16).cuda()
    check_select(q_tiny, big, table, [n * BS], K)
    # A NaN query: every score is NaN.
    q[0, 0, 0] = float("nan")
    assert check_select(q, s, table, [n * BS], K, 0, 0)[0, 0, 0].tolist() == list(range(K))


def test_selection_with_bad_blocks_and_lengths():
    rng = np.random.default_rng(5)
    table, nb = make_table(rng, [30 * BS, 30 * BS])
    q = torch.from_numpy(rng.standard_normal((2, 4, D))).to(torch.bfloat16).cuda()
    s = random_summaries(rng, nb, 2)
    bad = table.copy()
    bad[0, 3], bad[0, 12] = nb, -1
    check_select(q, s, bad, [30 * BS, 30 * BS], 6, bit=2)
    bad[0, :25] = -1  # fewer good blocks than places
    assert check_select(q, s, bad, [30 * BS, 30 * BS], 9, bit=2)[0, 0, 0].tolist() == \
        [0, 1, 2, 3, 25, 26, 27, 28, 29]
    st = status()
    got = api.select_blocks(q, s, ints(table), ints([30 * BS + 1, -4]), 40, dev_status=st).cpu().numpy()
    assert int(st.item()) == 4
    assert got[0, 0].tolist() == list(range(30)) + [-1] * 10 and (got[1] == -1).all()


# ------------------------------------------------------------------ attention
def check_attend(q, kc, vc, table, lens, idx, out_dtype=torch.float32, bit=0, three_dims=False, **kw):
    B, Q, H, _ = q.shape
    o, l, spread = sp.sparse_decode(f64(q), synth.bf16_bits(kc), synth.bf16_bits(vc), table, lens, idx,
                                    BS, D ** -0.5)
    st, lists, lse = status(), ints(idx), torch.full((B, Q, H), 77.0, device="cuda")
    if three_dims and Q == 1:  # the form without a q_len axis
        q, lists, lse = q[:, 0], lists[:, 0], lse[:, 0]
    out = api.paged_attention_decode_sparse(q, kc, vc, ints(table), ints(lens), lists, D ** -0.5, lse=lse,
                                            out_dtype=out_dtype, dev_status=st, **kw)
    assert int(st.item()) == bit and out.shape == q.shape
    got = out.double().cpu().numpy().reshape(o.shape)
    step = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    bound = (2.0 ** -8 / (1 - 2.0 ** -8) + 2e-4) * spread * (1 + 2.0 ** -8) + 1e-5
    assert (np.abs(got - o) <= bound + step * np.abs(o)).all(), np.abs(got - o).max()
    gl = lse.double().cpu().numpy().reshape(l.shape)
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(gl), ~fin)
    assert np.abs(gl[fin] - l[fin]).max(initial=0) <= LSE_TOL
    return out


def caches(nb, hkv, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((nb, BS, hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]


def random_lists(rng, lens, Q, hkv, K, shuffle=False):
    idx = np.full((len(lens), Q, hkv, K), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for i in range(Q):
            blocks = sp.row_blocks(int(n), Q, i, BS)
            for g in range(hkv):
                take = rng.permutation(blocks)[:K]
                idx[b, i, g, :len(take)] = take if shuffle else np.sort(take)
    return idx


def poison_unlisted(kc, vc, table, lens, idx, Q):
    """NaN in every block that no row lists and in every row behind its sequence."""
    used = {int(table[b, j]) for b in range(len(lens)) for i in range(Q)
            for j in idx[b, i].reshape(-1) if 0 <= j < sp.row_blocks(int(lens[b]), Q, i, BS)}
    for blk in range(kc.shape[0]):
        if blk not in used:
            kc[blk] = vc[blk] = float("nan")
    for b, n in enumerate(lens):
        if n % BS:
            kc[int(table[b, n // BS]), int(n % BS):] = float("nan")
            vc[int(table[b, n // BS]), int(n % BS):] = float("nan")


@pytest.mark.parametrize("H,Hkv,Q,K", [(8, 8, 1, 3), (16, 8, 1, 1), (8, 2, 2, 4), (64, 8, 1, 5),
                                       (16, 1, 3, 7), (4, 4, 7, 2)])
def test_sparse_decode_matches_oracle(H, Hkv, Q, K):
    rng = np.random.default_rng(H + Q)
    lens = np.array([0, 1, 2, 127, 128, 129, 640, 1111])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, Hkv, H)
    idx = random_lists(rng, lens, Q, Hkv, K)
    poison_unlisted(kc, vc, table, lens, idx, Q)
    q = torch.from_numpy(rng.standard_normal((8, Q, H, D))).to(torch.bfloat16).cuda()
    check_attend(q, kc, vc, table, lens, idx, three_dims=True)
    check_attend(q, kc, vc, table, lens, idx, out_dtype=torch.bfloat16)


def test_sparse_decode_with_holes_any_order_and_repeated_blocks():
    rng = np.random.default_rng(20)
    lens = np.array([900, 70, 1300])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 2)
    idx = random_lists(rng, lens, 2, 2, 6, shuffle=True)
    idx[0, 0, 0, [0, 2]] = -1
    idx[0, 1, 1] = -7            # a row and head with nothing to attend to
    idx[2, 0, 1, 3] = idx[2, 0, 1, 1]  # listed twice: counted twice
    q = torch.from_numpy(rng.standard_normal((3, 2, 8, D))).to(torch.bfloat16).cuda()
    out = check_attend(q, kc, vc, table, lens, idx)
    assert (out[0, 1, 4:] == 0).all() and (out[0, 1, :4] != 0).any()


def test_sparse_decode_flags_bad_entries_and_skips_them():
    rng = np.random.default_rng(21)
    lens = np.array([900, 500])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 2)
    q = torch.from_numpy(rng.standard_normal((2, 1, 8, D))).to(torch.bfloat16).cuda()
    idx = random_lists(rng, lens, 1, 2, 4)
    idx[0, 0, 0, 1] = 8   # the sequence has blocks 0..7
    idx[1, 0, 1, 2] = 1 << 30
    check_attend(q, kc, vc, table, lens, idx, bit=2)
    idx = random_lists(rng, lens, 1, 2, 4)
    bad = table.copy()
    bad[0, idx[0, 0, 0, 2]] = nb
    gone = idx.copy()
    gone[0][gone[0] == idx[0, 0, 0, 2]] = -1  # the oracle's view: an empty place
    st = status()
    got = api.paged_attention_decode_sparse(q, kc, vc, ints(bad), ints(lens), ints(idx), D ** -0.5,
                                            dev_status=st)
    assert int(st.item()) == 2
    want = check_attend(q, kc, vc, table, lens, gone)
    assert torch.equal(got, want)
    st = status()
    api.paged_attention_decode_sparse(q, kc, vc, ints(table), ints([1 << 20, -1]), ints(idx), D ** -0.5,
                                      dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & 4


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_sparse_decode_of_nan_scores_is_nan(out_dtype):
    """A NaN in a query, or in a key that is attended to, makes the heads that score it NaN, in rows
    that one CTA holds and in rows that the split cuts into many pieces; other heads and rows keep
    every bit."""
    rng = np.random.default_rng(25)
    lens = np.array([300, 200 * BS - 7, 90])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 2)
    idx = random_lists(rng, lens, 2, 2, 190)
    q = torch.from_numpy(rng.standard_normal((3, 2, 8, D))).to(torch.bfloat16).cuda()

    def run():
        st, lse = status(), torch.empty((3, 2, 8), device="cuda")
        out = api.paged_attention_decode_sparse(q, kc, vc, ints(table), ints(lens), ints(idx), D ** -0.5,
                                                lse=lse, out_dtype=out_dtype, dev_status=st)
        assert int(st.item()) == 0
        return out, lse

    out, lse = run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    lost = torch.zeros((3, 2, 8), dtype=torch.bool, device="cuda")
    q[2, 1, 6, 17] = float("nan")
    lost[2, 1, 6] = True
    q[1, 0, 1, 0] = float("nan")
    lost[1, 0, 1] = True
    kc[int(table[0, 1]), 5, 0, 100] = float("nan")  # both rows of sequence 0, the heads of kv head 0
    lost[0, :, :4] = True
    block = int(idx[1, 1, 1, 77])                   # a block in the middle of a cut list
    kc[int(table[1, block]), 64, 1, 3] = float("nan")
    for i in range(2):
        if block in idx[1, i, 1]:
            lost[1, i, 4:] = True
    kc[int(table[2, 0]), 90:, :] = float("nan")     # behind the sequence: nothing attends to it
    out_nan, lse_nan = run()
    assert torch.isnan(out_nan[lost]).all() and torch.isnan(lse_nan[lost]).all()
    assert torch.equal(out_nan[~lost], out[~lost]) and torch.equal(lse_nan[~lost], lse[~lost])


def test_sparse_decode_over_every_block_is_the_dense_decode():
    """With room for every block the lists are whole, the tiles and their split are those of
    the dense kernel, and so is every bit of the result."""
    rng = np.random.default_rng(22)
    lens = np.array([5000, 1, 0, 12345, 333])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 8)
    s = torch.zeros((nb, 8, 2, D), dtype=torch.bfloat16, device="cuda")
    q = torch.from_numpy(rng.standard_normal((5, 64, D))).to(torch.bfloat16).cuda()
    idx = api.select_blocks(q, s, ints(table), ints(lens), 97)
    lse, lse_d = (torch.empty((5, 64), device="cuda") for _ in range(2))
    a = api.paged_attention_decode_sparse(q, kc, vc, ints(table), ints(lens), idx, 0.1, lse=lse)
    b = api.paged_attention_decode(q, kc, vc, ints(table), ints(lens), 0.1, lse=lse_d)
    assert torch.equal(a, b) and torch.equal(lse, lse_d)


def test_sparse_decode_splits_long_lists_and_uses_its_own_workspace():
    rng = np.random.default_rng(23)
    lens = np.array([40000, 200])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 1)
    idx = random_lists(rng, lens, 1, 1, 250)
    q = torch.from_numpy(rng.standard_normal((2, 1, 4, D))).to(torch.bfloat16).cuda()
    need = api.decode_sparse_workspace_size(2, 1, 4, 1, D)
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    check_attend(q, kc, vc, table, lens, idx, workspace=ws)


def test_sparse_decode_of_many_query_rows():
    """Hundreds of rows (a chunk of a prompt, row by row): several seek rounds per CTA."""
    rng = np.random.default_rng(24)
    lens = np.array([333, 0, 90, 1500])
    table, nb = make_table(rng, lens)
    kc, vc = caches(nb, 1)
    Q = 150
    idx = random_lists(rng, lens, Q, 1, 2)
    q = torch.from_numpy(rng.standard_normal((4, Q, 2, D))).to(torch.bfloat16).cuda()
    check_attend(q, kc, vc, table, lens, idx)


def test_summaries_and_selection_after_rejected_drafts():
    """Rows written as drafts and overwritten later go on counting in their block; a block that
    starts over forgets them."""
    k = torch.zeros((3, BS, 1, D), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros((3, 1, 2, D), dtype=torch.bfloat16, device="cuda")
    t = ints([[1, 2]])
    k[1, :127] = torch.randn((127, 1, D), device="cuda").to(torch.bfloat16)
    api.update_block_summaries(s, k, t, ints([127]), ints([127]), 127)
    k[1, 127], k[2, 0] = 50.0, 60.0  # two drafts; the second opens a block
    api.update_block_summaries(s, k, t, ints([129]), ints([2]), 2)
    assert (s[1, 0, 1] == 50).all() and (s[2, 0] == 60).all()
    k[1, 127], k[2, 0] = 1.0, -1.0   # both rejected and written anew
    api.update_block_summaries(s, k, t, ints([129]), ints([2]), 2)
    assert (s[1, 0, 1] == 50).all() and (s[2, 0] == -1).all()


def test_sparse_decode_empty_batches():
    kc, vc = caches(2, 2)
    for shape, lists in (((0, 8, D), (0, 2, 3)), ((0, 2, 8, D), (0, 2, 2, 3)), ((3, 0, 8, D), (3, 0, 2, 3))):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        B = shape[0]
        t, lens = ints(np.zeros((B, 1))), ints(np.zeros(B))
        s = torch.zeros((2, 2, 2, D), dtype=torch.bfloat16, device="cuda")
        assert api.select_blocks(q, s, t, lens, 3).shape == lists
        out = api.paged_attention_decode_sparse(q, kc, vc, t, lens, ints(np.zeros(lists)), 0.1)
        assert out.shape == shape
    api.update_block_summaries(s, kc, ints(np.zeros((0, 1))), ints([]), ints([]), 5)
    api.update_block_summaries(s, kc, ints([[1]]), ints([5]), ints([0]), 0)
    assert int((s != 0).sum()) == 0


# ------------------------------------------------------------------ together
def test_a_decode_loop_with_rotation_summaries_selection_and_attention():
    """Prefill and 20 decode steps driven by the library's allocator: rotary write, summary
    update, selection, sparse attention; each step against the oracle on the same caches."""
    H, Hkv, K = 8, 2, 3
    freq = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    angle = torch.arange(2000, dtype=torch.float64)[:, None] * freq
    rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    mgr = api.KVCacheManager([0], [40], BS, 2048)
    nb, width = 40, 12
    kc, vc = (torch.full((nb, BS, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    s = torch.full((nb, Hkv, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens, first = np.zeros(3, dtype=np.int64), np.array([630, 127, 1])
    host = np.zeros((nb, Hkv, 2, D))
    g = torch.Generator(device="cuda").manual_seed(1)
    ws = torch.empty(api.decode_sparse_workspace_size(3, 1, H, Hkv, D), dtype=torch.uint8, device="cuda")
    for step in range(21):
        new = first if step == 0 else np.ones(3, dtype=np.int64)
        for r in range(3):
            assert mgr.allocate_slots(r, int(lens[r]), int(new[r]))
        table = mgr.block_table(0, [0, 1, 2], width)
        slots = ints(api.build_slot_mapping(table, lens, new, BS))
        pos = np.concatenate([np.arange(lens[r], lens[r] + new[r]) for r in range(3)])
        T = int(new.sum())
        qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        q = api.rope_kv_cache_write(kc, vc, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], rope,
                                    ints(pos), slots)
        lens = lens + new
        t, n = ints(table), ints(lens)
        api.update_block_summaries(s, kc, t, n, ints(new), int(new.max()))
        q = q[np.cumsum(new) - 1].contiguous()
        idx = api.select_blocks(q, s, t, n, K)
        bits = synth.bf16_bits(kc)
        host = sp.update_summaries(host, bits, table, lens, new, BS)
        want = sp.select_blocks(f64(q)[:, None], host, table, lens, K, 0, 1, BS)
        assert np.array_equal(idx.cpu().numpy(), want[:, 0]), step
        check_attend(q[:, None], kc, vc, table, lens, want, workspace=ws)


def test_a_sparse_step_in_a_graph_on_another_stream_and_two_at_once():
    rng = np.random.default_rng(30)
    lens = np.array([3000, 700, 129])
    table, nb = make_table(rng, lens + 5)
    kc, vc = caches(nb, 2)
    s = torch.zeros((nb, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    t, n, new = ints(table), ints(lens), ints(lens)
    api.update_block_summaries(s, kc, t, n, new, int(lens.max()))
    one = ints([1, 1, 1])
    qs = [torch.from_numpy(rng.standard_normal((3, 8, D))).to(torch.bfloat16).cuda() for _ in range(2)]
    bufs = [dict(idx=torch.empty((3, 2, 4), dtype=torch.int32, device="cuda"),
                 out=torch.empty((3, 8, D), device="cuda"),
                 ws=torch.empty(api.decode_sparse_workspace_size(3, 1, 8, 2, D), dtype=torch.uint8,
                                device="cuda")) for _ in range(2)]

    def step(i, stream=None):
        api.update_block_summaries(s, kc, t, n, one, 1, stream=stream)
        api.select_blocks(qs[i], s, t, n, 4, out=bufs[i]["idx"], stream=stream)
        api.paged_attention_decode_sparse(qs[i], kc, vc, t, n, bufs[i]["idx"], 0.1, out=bufs[i]["out"],
                                          workspace=bufs[i]["ws"], stream=stream)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):  # two steps at once, each on its own stream and workspace
        step(i, streams[i])
    torch.cuda.synchronize()
    first = [b["out"].clone() for b in bufs]
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        assert torch.equal(bufs[i]["out"], first[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    bufs[0]["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0]["out"], first[0])
    # The lengths and the queries change in their buffers; the graph follows.
    for k in range(1, 4):
        n.add_(1)
        qs[0].copy_(torch.from_numpy(rng.standard_normal((3, 8, D))).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        host = sp.update_summaries(np.zeros((nb, 2, 2, D)), synth.bf16_bits(kc), table, lens + k,
                                   lens + k, BS)
        want = sp.select_blocks(f64(qs[0])[:, None], host, table, lens + k, 4, 0, 1, BS)
        assert np.array_equal(bufs[0]["idx"].cpu().numpy(), want[:, 0])
        o, _, spread = sp.sparse_decode(f64(qs[0])[:, None], synth.bf16_bits(kc), synth.bf16_bits(vc),
                                        table, lens + k, want, BS, 0.1)
        err = np.abs(bufs[0]["out"].double().cpu().numpy() - o[:, 0])
        assert (err <= (2.0 ** -8 * 1.004 + 2e-4) * spread[:, 0] + 1e-5).all()


def test_entry_points_reject_bad_buffers_before_launch():
    kc, vc = caches(4, 2)
    s = torch.zeros((4, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 8, D), dtype=torch.bfloat16, device="cuda")
    t, n, idx = ints([[1, 2], [3, 0]]), ints([200, 9]), ints(np.zeros((2, 2, 3)))
    ok = dict(q=q, summaries=s, block_table=t, seq_lens=n, num_selected=3)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q[:, :, :64].contiguous()), dict(summaries=s[:, :, 0]),
               dict(summaries=s.float()), dict(block_table=t[:1]), dict(seq_lens=n.long()),
               dict(num_selected=0), dict(out=idx.float()), dict(out=idx[:, :, :2].contiguous()),
               dict(out=idx.cpu())):
        with pytest.raises(ValueError):
            api.select_blocks(**{**ok, **kw})
    with pytest.raises(PagedKVError, match="num_sink"):
        api.select_blocks(**ok, num_sink=3, num_recent=1)
    ok = dict(q=q, k_cache=kc, v_cache=vc, block_table=t, seq_lens=n, block_indices=idx, scale=0.1)
    for kw in (dict(block_indices=idx.long()), dict(block_indices=idx[:, :1].contiguous()),
               dict(block_indices=idx[None]), dict(q=q[:, None]), dict(v_cache=vc[:3]),
               dict(out=torch.empty((2, 8, 64), device="cuda")), dict(lse=torch.empty((2, 4), device="cuda")),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            api.paged_attention_decode_sparse(**{**ok, **kw})
    with pytest.raises(PagedKVError, match="scale"):
        api.paged_attention_decode_sparse(**{**ok, "scale": 0.0})
    for kw in (dict(summaries=s[:3]), dict(k_cache=kc.float()), dict(num_new=ints([1])), dict(seq_lens=ints([1]))):
        with pytest.raises(ValueError):
            api.update_block_summaries(**{**dict(summaries=s, k_cache=kc, block_table=t, seq_lens=n,
                                                 num_new=ints([1, 1]), max_new=1), **kw})
    torch.cuda.synchronize()


@pytest.mark.parametrize("B,q_len,n,width", [
    (2, 1, 300, 300), (90, 1, 300, 300), (1, 2, 600, 640), (160, 2, 600, 600), (1, 1, 2000, 2000),
    (40, 3, 2000, 2000), (1, 1, 700, 8192), (3, 1, 200, 200), (3, 2, 255, 300)])
def test_selection_with_fewer_good_blocks_than_places(B, q_len, n, width):
    """Table entries outside the cache rank last whatever the scores: with fewer good blocks than
    places every good one is in, then the lowest bad ones. With zero queries or zero summaries all
    scores are equal, and the lowest good blocks come first however many there are. Memory around
    the lists keeps its values."""
    rng = np.random.default_rng(n + B)
    K, sink, recent, nb = 40, 1, 2, 500
    want = K - sink - recent
    lens = np.full(B, n * BS)
    q = torch.from_numpy(rng.standard_normal((B, q_len, 2, D))).to(torch.bfloat16).cuda()
    s = random_summaries(rng, nb, 1)
    places, pad = B * q_len * K, 64
    buf = torch.empty(places + 2 * pad, dtype=torch.int32, device="cuda")
    for good in (0, 1, want - 1, want, want + 9):
        table = rng.integers(0, nb, (B, width)).astype(np.int32)
        expect = np.empty((B, q_len, 1, K), dtype=np.int32)
        for b in range(B):
            rivals = np.arange(sink, n - recent)
            keep = np.sort(rng.permutation(rivals)[:good])
            lost = np.setdiff1d(rivals, keep)
            table[b, lost] = rng.choice([-1, nb, -(1 << 31), (1 << 31) - 1], len(lost))
            take = np.sort(np.concatenate([keep, lost])[:want])
            expect[b] = np.concatenate([np.arange(sink), take, np.arange(n - recent, n)])
        kinds = [(torch.zeros_like(q), s), (q, torch.zeros_like(s))] + [(q, s)] * (good < want)
        for qk, sk in kinds:
            buf.fill_(-77)
            st = status()
            out = buf[pad:pad + places].view(B, q_len, 1, K)
            api.select_blocks(qk, sk, ints(table), ints(lens), K, sink, recent, out=out, dev_status=st)
            assert int(st.item()) == 2
            assert (buf[:pad] == -77).all() and (buf[pad + places:] == -77).all(), good
            assert np.array_equal(out.cpu().numpy(), expect), good


def test_sizes_past_int32_are_refused():
    """A count whose low 32 bits would pass for another one (2^32 + 1 rows for one)."""
    kc, _ = caches(4, 2)
    s = torch.zeros((4, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    q, t, n = torch.zeros((1, 8, D), dtype=torch.bfloat16, device="cuda"), ints([[1, 2]]), ints([200])
    with pytest.raises(ValueError, match="max_new"):
        api.update_block_summaries(s, kc, t, n, ints([1]), 2 ** 32 + 1)
    for name in ("num_selected", "num_sink", "num_recent"):
        for x in (2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1):
            with pytest.raises(ValueError, match=name):
                api.select_blocks(q, s, t, n, **{"num_selected": 3, name: x})
    api.update_block_summaries(s, kc, t, n, ints([1]), 2 ** 31 - 1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("spread", [0, 1, 3, 8, 16, 40, 100])
@pytest.mark.parametrize("signs", [False, True])
def test_matrix_products_are_as_exact_as_the_selection_takes_them_to_be(spread, signs):
    """A sum of 16 products of bf16 numbers (exact in fp32 each), added one by one and truncated to
    24 bits each time, is off by at most 16 2^-23 of the sum of their magnitudes, and the order or a
    better rounding only helps. The selection's bound counts 32 2^-24 for it; below 2^-126 it counts
    on nothing. In 64 bits the 16 products and their sum are off by 2^-49 of that sum at most."""
    n = 20000
    g = torch.Generator(device="cuda").manual_seed(spread)

    def numbers(shape):
        e = 127 - torch.randint(0, spread + 1, shape, generator=g, device="cuda", dtype=torch.int32)
        bits = (e << 7) | torch.randint(0, 128, shape, generator=g, device="cuda", dtype=torch.int32)
        x = bits.to(torch.int16).view(torch.bfloat16)
        return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, -x, x) if signs else x

    a, b = numbers((n, 16, 16)), numbers((n, 8, 16))
    if signs and spread:  # sums that cancel: half the terms against the other half, but for one
        a[: n // 2, :, 8:15] = -a[: n // 2, :, :7]
        b[: n // 2, :, 8:15] = b[: n // 2, :, :7]
    d = api.selftest_bf16_products(a, b)
    x, y = a.double(), b.double().transpose(1, 2)
    err, size = (d.double() - x @ y).abs(), x.abs() @ y.abs()
    floor = 2.0 ** -126 * (x.abs().sum(2)[:, :, None] + y.abs().sum(1)[:, None] + 16)
    bound = (32 * 2.0 ** -24 + 2.0 ** -49) * size + floor
    assert (err <= bound).all(), float((err / size).max() * 2 ** 24)
