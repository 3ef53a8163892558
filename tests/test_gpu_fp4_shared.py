"""The 4-bit decode where its tiles are shared out over all SMs and its parts merged: every table here
is wider than those whose sequences get a CTA each. Bounds as derived in test_gpu_fp4.py, but for the
log-sum-exp, whose sum is that of the unrounded weights."""
import numpy as np
import pytest
import torch

from oracle import fp4_ref as f4
from paged_kv_cache_77_gb300 import api
from tests.test_gpu_fp4 import BS, D, Batch, caches, f64, ints, rows_of, status

pytestmark = pytest.mark.gpu


class Wide(Batch):
    """A batch behind a table of at least `width` blocks."""

    def __init__(self, seed, lens, H, hkv, q_len, width=17, **kw):
        super().__init__(seed, lens, H, hkv, q_len, **kw)
        more = max(0, width - self.table.shape[1])
        self.table = np.pad(self.table, ((0, 0), (0, more)), constant_values=-7)

    def oracle(self, scale, window=0):
        o, lse, o_tol, lse_tol = super().oracle(scale, window)
        return o, lse, o_tol, lse_tol - 2.0 ** -11 * np.isfinite(lse)


def run(b, scale=0.09, **kw):
    args = b.args()
    st = status()
    lse = torch.full(args[0].shape[:-1], 7.0, device="cuda")
    out = api.paged_attention_decode_fp4(*args, scale, lse=lse, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return out, lse


SHAPES = [(8, 8, 1), (4, 1, 4), (16, 2, 1), (12, 6, 3), (16, 1, 1), (16, 2, 2), (16, 1, 2), (24, 3, 4), (8, 2, 2)]


@pytest.mark.parametrize("H,hkv,q_len", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode(H, hkv, q_len, out_dtype):
    b = Wide(H * 10 + q_len, [1, 0, 130, 515, 16, 128, 3, 2100, 257, 2], H, hkv, q_len)
    b.check(*run(b, out_dtype=out_dtype), 0.09)


@pytest.mark.parametrize("window", [1, 5, 128, 129, 300, 1000])
@pytest.mark.parametrize("H,hkv,q_len", [(8, 1, 1), (4, 4, 1), (4, 2, 4), (16, 2, 3), (16, 1, 2)])
@pytest.mark.parametrize("lens", [[3000, 128, 1, 0, 259, 3], [700, 0, 2] + [40 * i for i in range(1, 60)]])
def test_decode_with_a_window(H, hkv, q_len, window, lens):
    b = Wide(window, lens, H, hkv, q_len, width=24)
    # Blocks that no row's window touches: their entries name no block.
    for i, n in enumerate(b.lens):
        b.table[i, :max(0, n - q_len + 1 - window) // BS] = -3
    b.check(*run(b, window=window), 0.09, window)


@pytest.mark.parametrize("n_rep,q_len", [(8, 1), (8, 2), (16, 2)])
def test_warps_with_many_pieces(n_rep, q_len):
    """Some twelve blocks and more for every CTA, in few long segments and in many short ones: rings that
    are refilled, segments that end inside a warp's run, between warps and between CTAs."""
    b = Wide(61 + n_rep, [30000, 1, 10000, 0, 20000], 4 * n_rep, 4, q_len)
    b.check(*run(b, 0.05), 0.05)
    rng = np.random.default_rng(62)
    b = Wide(63 + n_rep, [int(n) for n in rng.integers(0, 1100, 120)], 4 * n_rep, 4, q_len)
    b.check(*run(b, out_dtype=torch.bfloat16), 0.09)


@pytest.mark.parametrize("H,hkv,q_len", [(8, 1, 1), (16, 1, 1), (16, 1, 2), (4, 4, 1)])
@pytest.mark.parametrize("window", [0, 5_000_000])
def test_warps_that_pass_many_blocks(H, hkv, q_len, window):
    """A sequence of ten million positions of which 300 blocks exist: a warp's run is longer than the 32
    table entries that it holds at a time, and what it skips counts for nothing."""
    rng = np.random.default_rng(64)
    width, exist = 84_000 // hkv, 300
    b = Batch(65, [exist * BS], H, hkv, q_len)
    at = np.sort(np.r_[rng.choice(width - 1, exist - 1, replace=False), width - 1])
    table = np.full((1, width), -1, dtype=np.int32)
    table[0, at] = b.table[0]
    q, kc, vc, ks, vs, _, _ = b.args()
    st = status()
    lse = torch.zeros(q.shape[:-1], device="cuda")
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, ints(table), ints([width * BS]), 0.09, lse=lse,
                                         window=window, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    if window:  # (the window's first position lies in a block that does not exist)
        first = (width * BS - q_len + 1 - window) // BS
        assert not np.isin(at, [first, first + 1]).any()
        keep = int((at > first).sum()) * BS
        b.key, b.val, b.lens = b.key[-keep:], b.val[-keep:], [keep]
    o, ref_lse, o_tol, lse_tol = b.oracle(0.09)
    assert (np.abs(out.double().cpu().numpy().reshape(o.shape) - o) <= o_tol + 2.0 ** -24 * (np.abs(o) + o_tol)).all()
    assert (np.abs(lse.double().cpu().numpy().reshape(ref_lse.shape) - ref_lse) <= lse_tol - 2.0 ** -11 +
            2.0 ** -22 * np.abs(ref_lse)).all()


@pytest.mark.parametrize("n", [96, 2400])
def test_lse_is_of_the_unrounded_weights(n):
    """Every 16 keys hold one of weight 1 and 15 of a weight just above the middle between two fp16
    numbers, which all round up: their rounded sum is nearly 2^-11 too large, the log-sum-exp is not.
    Bound: scores of one product each (8 2^-24 of their magnitude), exponentials (2^-21), and the fp32
    sums of positive terms, a lane's in a chain of n / 8 and then 8 lanes, 16 warps and the CTAs: 2^-24 a step."""
    weight = 0.5 * (1 + 2.0 ** -11 * (1 + 2.0 ** -6) + 2.0 ** -10 * 3)  # fp16's steps here: 2^-11
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[::16, 0, 0] = 6.0
    k[:, 0, 1] = 6.0  # (one scale of 1 in every row)
    q = torch.zeros((1, 8, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = float(np.float32(-np.log(weight) / 6))
    w = np.exp(-6 * scale)
    rounded = float(np.float16(w * 128)) / 128
    assert 2.0 ** -12 < rounded / w - 1 < 2.0 ** -11
    width = -(-n // BS)
    cache = caches(width, 1, BS)
    api.kv_cache_write_fp4(*cache, k, k, ints(np.arange(n)))
    table = np.pad(np.arange(width, dtype=np.int32), (0, 17))[None]
    for t in (table, table[:, :max(1, width)]):  # shared out; and a CTA for the sequence, if it is short
        lse = torch.zeros((1, 8), device="cuda")
        api.paged_attention_decode_fp4(q, *cache, ints(np.ascontiguousarray(t)), ints([n]), scale, lse=lse)
        torch.cuda.synchronize()
        want = 6 * scale + np.log(n / 16 * (1 + 15 * w))
        bound = 2 * 8 * 2.0 ** -24 * 6 * scale + 2.0 ** -21 + (n / 8 + 8 + 16 + 19) * 2.0 ** -24 + 2.0 ** -22 * want
        assert bound < 0.25 * np.log((1 + 15 * rounded) / (1 + 15 * w))
        assert (lse.double().cpu() - want).abs().max() <= bound


@pytest.mark.parametrize("more", [0, 120])
@pytest.mark.parametrize("H,hkv,q_len", [(8, 1, 2), (16, 1, 2)])
def test_nan_in_keys_and_values(H, hkv, q_len, more):
    """As where a CTA has the sequence: a NaN score makes its heads NaN, in whatever part it lies; a NaN
    among 16 values of V those 16 outputs, in the rows that see the token. (`more` sequences: warps and
    CTAs with parts of several segments.)"""
    n = 1100
    b = Wide(21, [n, 40] + [500] * more, H, hkv, q_len)
    kc, vc, ks, vs = b.cache

    def slot(seq, pos):
        return int(b.table[seq, pos // BS]), pos % BS

    blk, off = slot(0, n - 1)        # the newest token: row 0 does not see it
    vs[blk, 0, off, 2] = 0xFF
    blk0, off0 = slot(0, 400)        # in a part between others
    vs[blk0, 0, off0, 7] = 0xFF
    blk1, off1 = slot(1, 7)
    vs[blk1, 0, off1, 5] = 0xFF
    out, lse = run(b)
    o, _, o_tol, _ = b.oracle(0.09)
    got = out.double().cpu().numpy()
    nan = np.zeros(o.shape, dtype=bool)
    nan[0, 1, :, 32:48] = True
    nan[0, :, :, 112:128] = True
    nan[1, :, :, 80:96] = True
    assert (np.isnan(got) == nan).all()
    assert (np.abs(got - o)[~nan] <= (o_tol + 2.0 ** -24 * (np.abs(o) + o_tol))[~nan]).all()
    assert np.isfinite(lse.cpu().numpy()).all()
    for at in ((blk, off, 2), (blk0, off0, 7), (blk1, off1, 5)):
        vs[at[0], 0, at[1], at[2]] = 15 << 3
    ks[blk, 0, off, 1] = 0xFF        # a NaN key that only the last row sees
    ks[blk1, 0, off1, 0] = 0xFF      # and one that both rows of the other sequence do
    out, lse = run(b)
    bad = torch.isnan(out).all(-1).cpu().numpy()
    assert (torch.isnan(out).any(-1).cpu().numpy() == bad).all()
    assert bad[0, 1].all() and not bad[0, 0].any() and bad[1].all() and not bad[2:].any()
    assert (torch.isnan(lse).cpu().numpy() == bad).all()


@pytest.mark.parametrize("H,q_len", [(8, 1), (16, 2)])
def test_bad_blocks_and_lengths_are_flagged_and_skipped(H, q_len):
    b = Wide(31, [2300, 200], H, 1, q_len, width=18)
    q, kc, vc, ks, vs, table, lens = b.args()
    st = status()
    table[0, 1], table[0, 9] = kc.shape[0], -1
    lse = torch.zeros(q.shape[:-1], device="cuda")
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, table, lens, 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    c = Wide(31, [2300, 200], H, 1, q_len, width=18)
    keep = np.r_[0:128, 256:9 * 128, 10 * 128:2500]
    c.key, c.val, c.lens = b.key[keep], b.val[keep], [2300 - 256, 200]
    c.check(out, lse, 0.09)
    st.zero_()
    long = ints([b.table.shape[1] * BS + 1, -4])
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, table, long, 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) & 4 and not out[1].any() and torch.isneginf(lse[1]).all()


def test_a_graph_replayed_with_other_lengths():
    """Lengths, and with them the shares and the parts to merge, are read when the graph runs."""
    lens = [2300, 1, 90, 700]
    b = Wide(41, lens, 16, 2, 2)
    args = b.args()
    ws = torch.empty(api.decode_spec_workspace_size(4, 2, 16, 2, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((4, 2, 16, D), device="cuda"), torch.zeros((4, 2, 16), device="cuda")
    api.paged_attention_decode_fp4(*args, 0.09, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        api.paged_attention_decode_fp4(*args, 0.09, out=out, lse=lse, workspace=ws)
    key, val = np.split(b.key, np.cumsum(lens)[:-1]), np.split(b.val, np.cumsum(lens)[:-1])
    for now in ([2300, 1, 90, 700], [128, 0, 5, 1], [0, 0, 0, 0], [1900, 1, 90, 513]):
        args[-1].copy_(ints(now))
        out.fill_(7)
        lse.fill_(7)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        b.lens = now
        b.key = np.concatenate([x[:n] for x, n in zip(key, now)])
        b.val = np.concatenate([x[:n] for x, n in zip(val, now)])
        b.check(out, lse, 0.09)


def test_a_stream_of_its_own_and_no_tokens_at_all():
    b = Wide(42, [2600, 1, 90], 16, 2, 1)
    args = b.args()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    lse = torch.zeros((3, 16), device="cuda")
    out = api.paged_attention_decode_fp4(*args, 0.09, lse=lse, stream=side)
    torch.cuda.synchronize()
    b.check(out, lse, 0.09)
    out = api.paged_attention_decode_fp4(*args[:-1], ints([0, 0, 0]), 0.09, lse=lse)
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()


def test_decodes_repeat_themselves_and_run_two_at_once():
    batches = [Wide(73, [2000, 17, 900], 16, 2, 1), Wide(74, [13000, 5, 0, 4000], 8, 1, 4), Wide(75, [3000], 32, 2, 2)]
    jobs = [b.args() for b in batches]
    alone = [api.paged_attention_decode_fp4(*args, 0.09) for args in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        outs = [api.paged_attention_decode_fp4(*args, 0.09, stream=s) for args, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone))


def test_blocks_past_32_bits_of_bytes():
    nb, hkv = 70000, 8
    kc, vc = (torch.empty((nb, hkv, BS, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((nb, hkv, BS, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    b = Batch(51, [200], 16, hkv, 1)
    table = np.full((1, 17), -1, dtype=np.int32)
    table[0, :2] = nb - 1, nb - 3
    slots = table[0, np.arange(200) // BS] * BS + np.arange(200) % BS
    api.kv_cache_write_fp4(kc, vc, ks, vs, b.k, b.v, ints(slots))
    lse = torch.zeros((1, 16), device="cuda")
    out = api.paged_attention_decode_fp4(b.q[:, 0].contiguous(), kc, vc, ks, vs, ints(table), ints([200]), 0.09, lse=lse)
    torch.cuda.synchronize()
    b.check(out, lse, 0.09)


def test_a_fork_that_writes_on():
    """A child that shares full blocks and copies the last one decodes as its parent, then on its own."""
    b = Wide(71, [300], 8, 2, 1, nb_more=4)
    free = np.setdiff1d(np.arange(b.cache[0].shape[0]), b.table)
    child = b.table.copy()
    child[0, 2] = free[0]
    for t in b.cache:
        api.copy_blocks(t, ints(b.table[0, 2:3]), ints(free[:1]))
    q, *cache, table, _ = b.args()
    both, two = torch.cat([table, ints(child)]), torch.cat([q, q])
    out = api.paged_attention_decode_fp4(two, *cache, both, ints([300, 300]), 0.09)
    new = rows_of(np.random.default_rng(72), 1, 2, D)
    api.kv_cache_write_fp4(*b.cache, new, new, ints([child[0, 2] * BS + 44]))
    lse = torch.zeros((2, 8), device="cuda")
    after = api.paged_attention_decode_fp4(two, *cache, both, ints([300, 301]), 0.09, lse=lse)
    torch.cuda.synchronize()
    held = f4.dequantise(*f4.quantise(f64(new)))
    c = Wide(71, [300, 301], 8, 2, 1)
    c.q = two[:, None]
    c.key, c.val = np.concatenate([b.key, b.key, held]), np.concatenate([b.val, b.val, held])
    c.check(after, lse, 0.09)
    # (Other lengths, other shares: the parent's parts may be cut elsewhere.)
    assert torch.allclose(after[0], out[0], rtol=1e-3, atol=1e-3)
