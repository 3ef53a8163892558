"""GPU parity of the 4-bit cache against its float64 oracle.

The write is bit-exact (codes and scales), the read exact. Decode: K and V are exact in fp16 and
so is q (its row scaled by a power of two), so what is left is
  - the scores: 128 products in fp32 matrix sums, off by at most 512 2^-24 of the sum of their
    magnitudes, and a few fp32 roundings of the score itself (8 2^-24 of its magnitude): a
    weight moves by at most twice that much of itself (against the maximum's score as well);
  - the weights' exponential (2^-21 of a weight) and their rounding to fp16 (2^-11 of a weight;
    the rounded ones divide, so an output moves by 2^-11 / (1 - 2^-11) sum_j p_j |v_j - o|) and,
    below 2^-21 of the largest, 2^-32 of the largest per key;
  - the fp32 sums over n keys (n 2^-24 relative at most) and the output's own rounding."""
import numpy as np
import pytest
import torch

import synth
from oracle import fp4_ref as f4
from oracle.paged_ref import bf16_bits_to_f64
from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import PagedKVError

pytestmark = pytest.mark.gpu

BS, D = 128, 128


def f64(t):
    return bf16_bits_to_f64(synth.bf16_bits(t.contiguous()))


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def rows_of(rng, *shape):
    """bf16 rows whose groups differ in magnitude, with ties, zeros and equal values in some."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 6, shape[:-1] + (1,)))
    x[..., 16:32] *= np.exp2(rng.integers(-16, 10, shape[:-1] + (1,)))
    x[..., 32:48] = rng.integers(-12, 13, shape[:-1] + (16,)) / 2.0
    x[..., 47] = 6.0  # scale 1 (or near it): halves are borders between codes
    x[..., 48:64] *= rng.integers(0, 2, shape[:-1] + (1,))
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def caches(nb, hkv, bs, fill=None):
    out = []
    for width in (64, 64, 8, 8):
        t = torch.randint(0, 256, (nb, hkv, bs, width), dtype=torch.uint8, device="cuda")
        out.append(t if fill is None else t.fill_(fill))
    return out


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("T,hkv,bs,strided", [(1, 1, 128, False), (37, 3, 128, True), (700, 8, 128, False),
                                              (129, 2, 16, True), (1500, 1, 7, False), (2500, 8, 128, True)])
def test_write_is_bit_exact_and_read_exact(T, hkv, bs, strided):
    rng = np.random.default_rng(T)
    nb = -(-T // bs) + 3
    k = rows_of(rng, T, hkv, D)
    v = rows_of(rng, T, 3 * hkv, D)[:, hkv:2 * hkv] if strided else rows_of(rng, T, hkv, D)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    slots[::13] = -1 - slots[::13]
    kc, vc, ks, vs = caches(nb, hkv, bs)
    before = [t.cpu().numpy() for t in (kc, vc, ks, vs)]
    st = status()
    api.kv_cache_write_fp4(kc, vc, ks, vs, k, v, ints(slots), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for rows, c, s, c0, s0 in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        want_c, want_s = f4.cache_write(c0, s0, f64(rows), slots)
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)
        np.testing.assert_array_equal(c.cpu().numpy(), want_c)
    got = api.kv_cache_read_fp4(kc, vc, ks, vs, ints(slots), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for rows, out in ((k, got[0]), (v, got[1])):
        want = f4.dequantise(*f4.quantise(f64(rows)))
        want[slots < 0] = 0
        np.testing.assert_array_equal(f64(out), want)


def test_every_scale_and_code_reads_as_its_value():
    kc, vc, ks, vs = caches(2, 1, 128, fill=0)
    byte = torch.arange(256, dtype=torch.uint8, device="cuda")
    ks.view(256, 8)[:] = byte[:, None]
    kc.view(256, 8, 8)[:] = byte.view(256, 1, 1) * 0 + torch.tensor(
        [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], dtype=torch.uint8, device="cuda")
    vs.fill_(15 << 3)
    vc.view(256, 64)[:] = byte[:, None]
    k, v = api.kv_cache_read_fp4(kc, vc, ks, vs, ints(np.arange(256)))
    torch.cuda.synchronize()
    want = f4.dequantise(kc.cpu().numpy(), ks.cpu().numpy()).reshape(256, 128)
    keep = np.arange(256) <= f4.MAX_SCALE
    np.testing.assert_array_equal(f64(k)[keep, 0], want[keep])
    assert np.isnan(f64(k)[255]).all()
    np.testing.assert_array_equal(f64(v)[:, 0],
                                  f4.dequantise(vc.cpu().numpy(), vs.cpu().numpy()).reshape(256, 128))


def test_every_bf16_magnitude_as_a_groups_largest():
    """All 32,640 finite magnitudes, each alone in its group and beside its halves."""
    mag = np.arange(0x7f80, dtype=np.uint32)
    x = torch.from_numpy((mag << 16).view(np.float32)).to(torch.bfloat16)
    rows = torch.zeros((len(mag) // 8, 1, 8, 16), dtype=torch.bfloat16)
    rows[:, 0, :, 3] = x.view(-1, 8)
    rows[:, 0, :, 4:8] = (x.view(-1, 8, 1).float() * torch.tensor([-0.5, 0.25, -0.125, 0.0625])).to(torch.bfloat16)
    rows = rows.flatten(2).cuda()
    T = len(rows)
    nb = -(-T // 128)
    kc, vc, ks, vs = caches(nb, 1, 128, fill=0)
    api.kv_cache_write_fp4(kc, vc, ks, vs, rows, -rows, ints(np.arange(T)))
    torch.cuda.synchronize()
    for c, s, sign in ((kc, ks, 1), (vc, vs, -1)):
        want_c, want_s = f4.quantise(sign * f64(rows)[:, 0])
        np.testing.assert_array_equal(s.cpu().numpy().reshape(-1, 8)[:T], want_s)
        got = c.cpu().numpy().reshape(-1, 64)[:T]
        # Zeros may carry a sign.
        np.testing.assert_array_equal(f4.dequantise(got, want_s), f4.dequantise(want_c, want_s))


def test_infinities_and_nan_in_a_row():
    rng = np.random.default_rng(8)
    k = rows_of(rng, 3, 2, D)
    k[0, 0, 5], k[1, 1, 40], k[2, 0, 127] = float("inf"), float("nan"), -float("inf")
    kc, vc, ks, vs = caches(1, 2, 128)
    api.kv_cache_write_fp4(kc, vc, ks, vs, k, k, ints([7, 0, 127]))
    torch.cuda.synchronize()
    got_k, got_v = api.kv_cache_read_fp4(kc, vc, ks, vs, ints([7, 0, 127]))
    torch.cuda.synchronize()
    codes, scales = f4.quantise(f64(k))
    np.testing.assert_array_equal(ks[0, :, 7].cpu().numpy(), scales[0])
    np.testing.assert_array_equal(f64(got_k), f4.dequantise(codes, scales))
    np.testing.assert_array_equal(f64(got_v), f4.dequantise(codes, scales))


def test_slots_past_the_cache_are_flagged():
    kc, vc, ks, vs = caches(2, 2, 128)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    rows = torch.ones((2, 2, D), dtype=torch.bfloat16, device="cuda")
    st = status()
    api.kv_cache_write_fp4(kc, vc, ks, vs, rows, rows, ints([256, -5]), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 1 and all(torch.equal(a, b) for a, b in zip(before, (kc, vc, ks, vs)))
    st.zero_()
    k, v = api.kv_cache_read_fp4(kc, vc, ks, vs, ints([300, -1]), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 1 and not k.any() and not v.any()
    # No rows at all.
    none = rows[:0]
    api.kv_cache_write_fp4(kc, vc, ks, vs, none, none, ints([]))
    assert api.kv_cache_read_fp4(kc, vc, ks, vs, ints([]))[0].shape == (0, 2, D)


# ------------------------------------------------------------------ decode
class Batch:
    """Sequences of given lengths in a 4-bit cache whose other rows hold any bytes."""

    def __init__(self, seed, lens, H, hkv, q_len, spread=1.0, nb_more=3):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.hkv, self.q_len = list(lens), H, hkv, q_len
        need = [-(-int(n) // BS) for n in lens]
        nb = sum(need) + nb_more
        order = rng.permutation(nb)
        self.table = np.full((len(lens), max(1, max(need, default=1))), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = caches(nb, hkv, BS)
        total = int(sum(lens))
        self.k = (rows_of(rng, total, hkv, D).float() * 0.25).clamp(-8, 8).to(torch.bfloat16)
        self.v = rows_of(rng, total, hkv, D)
        slots = np.concatenate([self.table[b, np.arange(n) // BS] * BS + np.arange(n) % BS
                                for b, n in enumerate(lens)] or [np.zeros(0)])
        api.kv_cache_write_fp4(*self.cache, self.k, self.v, ints(slots))
        q = rng.standard_normal((len(lens), q_len, H, D)) * spread
        self.q = torch.as_tensor(q, dtype=torch.float32).to(torch.bfloat16).cuda()
        self.key = f4.dequantise(*f4.quantise(f64(self.k)))
        self.val = f4.dequantise(*f4.quantise(f64(self.v)))

    def args(self):
        q = self.q[:, 0].contiguous() if self.q_len == 1 else self.q
        return q, *self.cache, ints(self.table), ints(self.lens)

    def oracle(self, scale, window=0):
        """o, lse, and the bounds of their errors."""
        B, Q, H, n_rep = len(self.lens), self.q_len, self.H, self.H // self.hkv
        q = f64(self.q)
        o, lse = np.zeros((B, Q, H, D)), np.full((B, Q, H), -np.inf)
        o_tol, lse_tol = np.zeros((B, Q, H, D)), np.zeros((B, Q, H))
        at = 0
        for b, n in enumerate(self.lens):
            K, V = self.key[at:at + n], self.val[at:at + n]
            at += n
            for i in range(Q):
                end = n - Q + 1 + i
                lo = max(0, end - window) if window else 0
                if end <= 0:
                    continue
                for h in range(H):
                    kk, vv = K[lo:end, h // n_rep], V[lo:end, h // n_rep]
                    s = scale * (kk @ q[b, i, h])
                    mag = scale * (np.abs(kk) @ np.abs(q[b, i, h])).max()
                    p = np.exp(s - s.max())
                    total = p.sum()
                    lse[b, i, h] = s.max() + np.log(total)
                    p /= total
                    o[b, i, h] = p @ vv
                    spread = p @ np.abs(vv - o[b, i, h])
                    ds = mag * 512 * 2.0 ** -24 + np.abs(s).max() * 8 * 2.0 ** -24 + 2.0 ** -21
                    count = end - lo
                    o_tol[b, i, h] = (2.0 ** -11 / (1 - 2.0 ** -11) + 2 * ds) * spread + (
                        count * 2.0 ** -23 + 2.0 ** -21) * (p @ np.abs(vv)) + (
                        2.0 ** -32 * p.max()) * np.abs(vv - o[b, i, h]).sum(0)
                    # The sum is of rounded weights: off by 2^-11 of itself at most.
                    lse_tol[b, i, h] = ds + 2.0 ** -11 + count * 2.0 ** -23 + 2.0 ** -21
        return o, lse, o_tol, lse_tol

    def check(self, out, lse, scale, window=0):
        o, ref_lse, o_tol, lse_tol = self.oracle(scale, window)
        half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
        got = out.double().cpu().numpy().reshape(o.shape)
        err = np.abs(got - o)
        assert (err <= o_tol + half * (np.abs(o) + o_tol)).all(), (err - o_tol).max()
        got = lse.double().cpu().numpy().reshape(ref_lse.shape)
        assert (np.isneginf(got) == np.isneginf(ref_lse)).all()
        live = np.isfinite(ref_lse)
        assert (np.abs(got[live] - ref_lse[live]) <= lse_tol[live] + 2.0 ** -22 * np.abs(ref_lse[live])).all()


@pytest.mark.parametrize("H,hkv,q_len", [(8, 8, 1), (4, 1, 4), (16, 2, 1), (12, 6, 3), (16, 1, 1), (16, 2, 2),
                                         (16, 1, 2), (24, 3, 4), (8, 2, 2)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode(H, hkv, q_len, out_dtype):
    b = Batch(H * 10 + q_len, [1, 0, 130, 515, 16, 128, 3, 1000, 257, 2], H, hkv, q_len)
    st = status()
    args = b.args()
    lse = torch.full(args[0].shape[:-1], 7.0, device="cuda")
    out = api.paged_attention_decode_fp4(*args, 0.09, lse=lse, out_dtype=out_dtype, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    b.check(out, lse, 0.09)


@pytest.mark.parametrize("window", [1, 5, 128, 129, 300])
@pytest.mark.parametrize("H,hkv,q_len", [(8, 1, 1), (4, 2, 4), (16, 2, 3)])
def test_decode_with_a_window(H, hkv, q_len, window):
    b = Batch(window, [700, 128, 1, 0, 259, 3], H, hkv, q_len)
    q, kc, vc, ks, vs, table, lens = b.args()
    # Blocks that no row's window touches: their entries name no block.
    for i, n in enumerate(b.lens):
        first = max(0, n - q_len + 1 - window) // BS
        table[i, :first] = -3
    lse = torch.zeros(q.shape[:-1], device="cuda")
    st = status()
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, table, lens, 0.09, window=window, lse=lse,
                                         dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    b.check(out, lse, 0.09, window)


@pytest.mark.parametrize("spread", [1e-30, 30.0])
def test_decode_of_flat_and_of_peaked_scores(spread):
    b = Batch(3, [2000, 77], 8, 1, 1, spread=spread)
    lse = torch.zeros((2, 8), device="cuda")
    out = api.paged_attention_decode_fp4(*b.args(), 0.09, lse=lse)
    torch.cuda.synchronize()
    b.check(out, lse, 0.09)


def test_decode_long_and_many():
    """A sequence over many CTAs beside short ones; more segments than CTAs."""
    b = Batch(11, [20000, 5, 300], 8, 1, 1)
    lse = torch.zeros((3, 8), device="cuda")
    out = api.paged_attention_decode_fp4(*b.args(), 0.05, lse=lse)
    torch.cuda.synchronize()
    b.check(out, lse, 0.05)
    b = Batch(12, [int(n) for n in np.random.default_rng(1).integers(0, 400, 60)], 16, 8, 2)
    lse = torch.zeros((60, 2, 16), device="cuda")
    out = api.paged_attention_decode_fp4(*b.args(), 0.09, lse=lse, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    b.check(out, lse, 0.09)


@pytest.mark.parametrize("H,hkv,q_len", [(8, 1, 2), (16, 1, 2)])
def test_nan_in_keys_and_values(H, hkv, q_len):
    """A NaN score makes its heads NaN; a NaN among 16 values of V those 16 outputs, in the rows
    that see the token and in no other."""
    n = 300
    b = Batch(21, [n, 40], H, hkv, q_len)
    kc, vc, ks, vs = b.cache

    def slot(seq, pos):
        return int(b.table[seq, pos // BS]), pos % BS

    blk, off = slot(0, n - 1)        # the newest token: row 0 does not see it
    vs[blk, 0, off, 2] = 0xFF
    blk, off = slot(1, 7)            # seen by both rows
    vs[blk, 0, off, 5] = 0xFF
    lse = torch.zeros((2, q_len, H), device="cuda")
    out = api.paged_attention_decode_fp4(*b.args(), 0.09, lse=lse)
    torch.cuda.synchronize()
    o, ref_lse, o_tol, _ = b.oracle(0.09)
    got = out.double().cpu().numpy()
    nan = np.zeros(o.shape, dtype=bool)
    nan[0, 1, :, 32:48] = True
    nan[1, :, :, 80:96] = True
    assert (np.isnan(got) == nan).all()
    # The newest token's group counts as NaN only: the other outputs are as without it.
    assert (np.abs(got - o)[~nan] <= (o_tol + 2.0 ** -24 * (np.abs(o) + o_tol))[~nan]).all()
    assert np.isfinite(lse.cpu().numpy()).all()
    vs[blk, 0, off, 5] = 15 << 3
    blk, off = slot(0, n - 1)
    vs[blk, 0, off, 2] = 15 << 3
    ks[blk, 0, off, 1] = 0xFF        # a NaN key that only the last row sees
    out = api.paged_attention_decode_fp4(*b.args(), 0.09, lse=lse)
    torch.cuda.synchronize()
    bad = torch.isnan(out).all(-1).cpu().numpy()
    assert (torch.isnan(out).any(-1).cpu().numpy() == bad).all()
    assert bad[0, 1].all() and not bad[0, 0].any() and not bad[1].any()
    assert (torch.isnan(lse).cpu().numpy() == bad).all()


def test_bad_blocks_and_lengths_are_flagged_and_skipped():
    b = Batch(31, [300, 200], 8, 1, 1)
    q, kc, vc, ks, vs, table, lens = b.args()
    st = status()
    bad = table.clone()
    bad[0, 1] = kc.shape[0]
    lse = torch.zeros((2, 8), device="cuda")
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, bad, lens, 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 2
    # The skipped block is as if it were not there.
    c = Batch(31, [300, 200], 8, 1, 1)
    keep = np.r_[0:128, 256:300, 300:500]
    c.key, c.val, c.lens = b.key[keep], b.val[keep], [172, 200]
    c.check(out, lse, 0.09)
    st.zero_()
    long = ints([b.table.shape[1] * BS + 1, -4])
    out = api.paged_attention_decode_fp4(q, kc, vc, ks, vs, table, long, 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) & 4 and not out[1].any() and torch.isneginf(lse[1]).all()


def test_graph_stream_and_no_sequences():
    b = Batch(41, [600, 1, 90], 16, 2, 1)
    args = b.args()
    ws = torch.empty(api.decode_spec_workspace_size(3, 1, 16, 2, D), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros((3, 16, D), device="cuda"), torch.zeros((3, 16), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    api.paged_attention_decode_fp4(*args, 0.09, out=out, lse=lse, workspace=ws, stream=side)
    torch.cuda.synchronize()
    b.check(out, lse, 0.09)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention_decode_fp4(*args, 0.09, out=out, lse=lse, workspace=ws)
    args[-1][0] = 333
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    b.lens[0] = 333
    b.key = np.concatenate([b.key[:333], b.key[600:]])
    b.val = np.concatenate([b.val[:333], b.val[600:]])
    b.check(out, lse, 0.09)
    assert not torch.equal(first, out)
    q, kc, vc, ks, vs, table, lens = args
    none = api.paged_attention_decode_fp4(q[:0], kc, vc, ks, vs, table[:0], lens[:0], 0.09)
    assert none.shape == (0, 16, D)
    with pytest.raises(PagedKVError, match="workspace"):
        api.paged_attention_decode_fp4(*args, 0.09, workspace=ws.new_empty(1 << 20)[1:])


def test_blocks_past_32_bits_of_bytes():
    """Rows more than 4 GB into every cache."""
    nb, hkv = 70000, 8
    kc, vc = (torch.empty((nb, hkv, BS, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((nb, hkv, BS, 8), dtype=torch.uint8, device="cuda") for _ in range(2))
    b = Batch(51, [200], 16, hkv, 1)
    table = np.array([[nb - 1, nb - 3]], dtype=np.int32)
    slots = table[0, np.arange(200) // BS] * BS + np.arange(200) % BS
    api.kv_cache_write_fp4(kc, vc, ks, vs, b.k, b.v, ints(slots))
    k, v = api.kv_cache_read_fp4(kc, vc, ks, vs, ints(slots))
    lse = torch.zeros((1, 16), device="cuda")
    out = api.paged_attention_decode_fp4(b.q[:, 0].contiguous(), kc, vc, ks, vs, ints(table), ints([200]),
                                         0.09, lse=lse)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(k), b.key)
    np.testing.assert_array_equal(f64(v), b.val)
    b.check(out, lse, 0.09)


def test_a_fork_of_4_bit_blocks():
    """copy_blocks copies codes and scales: the child reads what the parent does, and what it then
    writes is its own."""
    b = Batch(71, [300], 8, 2, 1, nb_more=4)
    free = np.setdiff1d(np.arange(b.cache[0].shape[0]), b.table)
    child = b.table.copy()
    child[0, 2] = free[0]  # shared full blocks, a copy of the last one
    for t in b.cache:
        api.copy_blocks(t, ints(b.table[0, 2:3]), ints(free[:1]))
    q, k_cache, v_cache, k_scale, v_scale, table, lens = b.args()
    both = torch.cat([table, ints(child)])
    args = torch.cat([q, q]), k_cache, v_cache, k_scale, v_scale, both, ints([300, 300])
    out = api.paged_attention_decode_fp4(*args, 0.09)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])
    new = rows_of(np.random.default_rng(72), 1, 2, D)
    api.kv_cache_write_fp4(*b.cache, new, new, ints([child[0, 2] * BS + 44]))
    after = api.paged_attention_decode_fp4(*args[:-1], ints([300, 301]), 0.09)
    torch.cuda.synchronize()
    assert torch.equal(after[0], out[0]) and not torch.equal(after[1], out[1])


def test_two_decodes_at_once():
    """Workspaces of their own on streams of their own: the results of each alone."""
    batches = [Batch(73, [2000, 17, 900], 16, 2, 1), Batch(74, [1300, 5], 8, 1, 3)]
    jobs = [b.args() for b in batches]
    alone = [api.paged_attention_decode_fp4(*args, 0.09) for args in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        outs = [api.paged_attention_decode_fp4(*args, 0.09, stream=s) for args, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone))


@pytest.mark.parametrize("B,H,hkv,q_len,width", [
    (3, 8, 2, 1, 16), (3, 8, 2, 1, 17), (3, 8, 4, 3, 16), (3, 8, 4, 3, 17), (1, 1, 1, 1, 16), (1, 1, 1, 1, 17),
    (9, 16, 16, 1, 16), (10, 16, 16, 1, 16), (3, 8, 2, 3, 8), (3, 8, 2, 3, 9), (3, 16, 2, 4, 8), (3, 16, 2, 4, 9),
    (3, 16, 1, 1, 8), (3, 16, 1, 1, 9)])
def test_decode_with_a_cta_for_a_sequence_or_shared_out(B, H, hkv, q_len, width):
    """Tables on either side of the rule that gives a sequence and kv head a CTA of its own: the
    same attention, with lengths of zero, of one token, of whole tables, and past the table."""
    full = 128 * (width // 8 * 8)
    lens = ([full, 0, 1] + [37 * i for i in range(3, 10)])[:B]
    b = Batch(80 + B + q_len, lens, H, hkv, q_len)
    table = np.full((B, width), -3, dtype=np.int32)
    table[:, :b.table.shape[1]] = b.table[:, :width]
    args = list(b.args())
    args[5] = ints(table)
    st = status()
    lse = torch.full(args[0].shape[:-1], 7.0, device="cuda")
    out = api.paged_attention_decode_fp4(*args, 0.09, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    b.check(out, lse, 0.09)
    args[6] = ints([5000 if n == full else n for n in lens])  # clamped to the table
    if width % 8 == 0:
        again = api.paged_attention_decode_fp4(*args, 0.09, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == 4 and torch.equal(again, out)


def test_a_write_of_no_rows_takes_any_strides():
    cache = caches(2, 3, BS)
    before = [t.clone() for t in cache]
    none = torch.empty(1024, dtype=torch.bfloat16, device="cuda").as_strided((0, 3, D), (1, 1, 1))
    api.kv_cache_write_fp4(*cache, none, none, ints([]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cache, before))


def test_binding_refuses_wrong_buffers():
    b = Batch(90, [300, 20], 8, 2, 1)
    args = b.args()
    q, kc, vc, ks, vs, table, lens = args
    need = api.decode_spec_workspace_size(2, 1, 8, 2, D)

    def refused(match, *positional, **kw):
        with pytest.raises(ValueError, match=match):
            api.paged_attention_decode_fp4(*(positional or args), 0.09, **kw)

    refused(f"needs {need}", workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    refused("workspace must be contiguous", workspace=torch.empty((need, 2), dtype=torch.uint8, device="cuda")[:, 0])
    refused("v_cache", q, kc, None, ks, vs, table, lens)
    refused("v_scale", q, kc, vc, ks, None, table, lens)
    refused("v_cache", q, kc, vc[:1].contiguous(), ks, vs, table, lens)
    refused("k_scale", q, kc, vc, ks[..., :4].contiguous(), vs, table, lens)
    refused("k_cache", q, kc[0], vc, ks, vs, table, lens)
    refused("block_table", q, kc, vc, ks, vs, table[:1], lens)
    refused("block_table", q, kc, vc, ks, vs, table[0], lens)
    refused("seq_lens", q, kc, vc, ks, vs, table, lens.long())
    refused("seq_lens", q, kc, vc, ks, vs, table, lens[:1])
    refused("lse", lse=torch.empty((2, 8), dtype=torch.float64, device="cuda"))
    refused("out", out=torch.empty((2, 8, 64), device="cuda"))
    for call in (lambda: api.kv_cache_read_fp4(kc, vc, ks, None, ints([0])),
                 lambda: api.select_rows(torch.zeros((4, 2, BS), device="cuda"), table.long(), lens, 5),
                 lambda: api.select_rows(torch.zeros((4, 2, BS), device="cuda"), table[:1], lens, 5)):
        with pytest.raises(ValueError):
            call()
