"""GPU parity: fused rotary embedding + paged write (bf16 and FP8 caches) and the FP8 read.

A rotated element is x1 c - x2 s in fp32: one product rounded, one fused multiply-add
rounded, so it is off by at most 2^-24 (|x2 s| + |result|) <= 2^-23 m with
m = |x1 c| + |x2 s|. Rounding to bf16 then adds at most half a step, 2^-8 of the value.
Elements that pass through, v rows and rows that are not written are bit-identical.

FP8: codes are E4M3 of the fp32 value over the row's scale. A code times its scale is off
the exact value by at most half an E4M3 step: 2^-4 of the value for normal codes, half the
subnormal step (2^-10 scales) below; the fp32 errors of the rotation, of the scale (amax of
values off by 2^-23 m, one division) and of the quotient add to that."""
import numpy as np
import pytest
import torch

import synth
from oracle import fp8_ref
from oracle import rope_write_ref as rw
from oracle.paged_ref import bf16_bits_to_f64
from paged_kv_cache_77_gb300 import api
from paged_kv_cache_77_gb300._lib import PagedKVError

pytestmark = pytest.mark.gpu

BS = 128


class Case:
    """Random rows, a table, positions and a pool; the rows are slices of one buffer when
    `strided`."""

    def __init__(self, T, H, Hkv, d, rope_dim, axis=None, interleaved=False, strided=False, seed=0,
                 max_pos=4096, blocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.Hkv, self.d, self.rope_dim = T, H, Hkv, d, rope_dim
        self.interleaved = interleaved
        self.axis = None if axis is None else np.asarray(axis, dtype=np.int32)
        axes = 1 if axis is None else int(self.axis.max()) + 1
        qkv = torch.randn((T, H + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        parts = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        self.qkv = qkv
        self.q, self.k, self.v = parts if strided else [p.contiguous() for p in parts]
        freq = 10000.0 ** (-torch.arange(rope_dim // 2, dtype=torch.float64) * 2 / rope_dim)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.pos = torch.randint(0, max_pos, (axes, T), generator=g, device="cuda",
                                 dtype=torch.int32)
        self.nb = blocks or T // BS + 3
        self.slots = torch.randperm(self.nb * BS, generator=g, device="cuda")[:T].to(torch.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def host(self, x):
        """Rows as the oracle reads them, taken before any in-place rotation."""
        return bf16_bits_to_f64(synth.bf16_bits(x.contiguous()))

    def exact(self, x):
        args = (self.table.cpu().numpy(), self.pos.cpu().numpy(), self.axis, self.interleaved)
        h = self.host(x)
        return rw.rotate_rows(h, *args), rw.rotate_magnitude(h, *args)

    def kwargs(self):
        return dict(pair_axis=self.axis, interleaved=self.interleaved, dev_status=self.status)


def _check_rotated(got, want, mag, rope_dim, what):
    """got [n, heads, d] float64 of bf16 results."""
    err = np.abs(got - want)
    bound = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 2.0 ** -23 * mag
    assert (err <= bound).all(), f"{what}: {(err - bound).max():.3e} beyond the bound"
    assert np.array_equal(got[..., rope_dim:], want[..., rope_dim:]), what


CASES = [
    # T, H, Hkv, d, rope_dim, axis, interleaved, strided
    (1, 1, 1, 16, 16, None, False, False),
    (1, 64, 8, 128, 128, None, False, False),
    (7, 8, 2, 64, 32, None, True, False),
    (33, 4, 4, 128, 128, np.repeat([0, 1, 2], [16, 24, 24]), False, True),
    (129, 6, 2, 80, 48, np.arange(24) % 3, False, True),
    (130, 6, 3, 96, 96, np.arange(48) % 4, True, True),
    (5, 3, 1, 256, 256, np.repeat([1, 0], [60, 68]), False, False),
    (700, 5, 5, 192, 64, None, False, True),
    (2051, 32, 8, 128, 128, np.repeat([0, 1, 2], [16, 24, 24]), True, True),
]


@pytest.mark.parametrize("T,H,Hkv,d,rope_dim,axis,interleaved,strided", CASES)
def test_rope_write_matches_oracle(T, H, Hkv, d, rope_dim, axis, interleaved, strided):
    c = Case(T, H, Hkv, d, rope_dim, axis, interleaved, strided, seed=T + d)
    kc = torch.randn((c.nb, BS, Hkv, d), device="cuda").to(torch.bfloat16)
    vc = torch.randn((c.nb, BS, Hkv, d), device="cuda").to(torch.bfloat16)
    pre_k, pre_v = synth.bf16_bits(kc), synth.bf16_bits(vc)
    if T > 3:
        c.slots[1] = -1  # a padded row: its q is rotated, its k and v are not written
    out = api.rope_kv_cache_write(kc, vc, c.q, c.k, c.v, c.table, c.pos, c.slots, **c.kwargs())
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    _check_rotated(c.host(out), *c.exact(c.q), rope_dim, "q")
    slots = c.slots.cpu().numpy()
    on = slots >= 0
    got_k = bf16_bits_to_f64(synth.bf16_bits(kc)).reshape(-1, Hkv, d)
    want, mag = c.exact(c.k)
    _check_rotated(got_k[slots[on]], want[on], mag[on], rope_dim, "k")
    flat_v = synth.bf16_bits(vc).reshape(-1, Hkv, d)
    assert np.array_equal(flat_v[slots[on]], synth.bf16_bits(c.v.contiguous())[on])
    left = np.ones(c.nb * BS, dtype=bool)
    left[slots[on]] = False
    assert np.array_equal(synth.bf16_bits(kc).reshape(-1, Hkv, d)[left],
                          pre_k.reshape(-1, Hkv, d)[left])
    assert np.array_equal(flat_v[left], pre_v.reshape(-1, Hkv, d)[left])


@pytest.mark.parametrize("T,H,Hkv,rope_dim,axis,interleaved,strided", [
    (1, 8, 1, 128, None, False, False),
    (19, 5, 3, 64, None, True, True),
    (300, 64, 8, 128, np.repeat([0, 1, 2], [16, 24, 24]), False, True),
])
def test_rope_write_fp8_matches_oracle(T, H, Hkv, rope_dim, axis, interleaved, strided):
    c = Case(T, H, Hkv, 128, rope_dim, axis, interleaved, strided, seed=T)
    kc, vc = (torch.full((c.nb, BS, Hkv, 128), 0x55, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    ks, vs = (torch.full((c.nb, Hkv, BS), 7.0, device="cuda") for _ in range(2))
    c.k[0, 0] = 0  # an all-zero row: scale 0, zero codes
    if T > 3:
        c.slots[2] = -1
    out = api.rope_kv_cache_write_fp8(kc, vc, ks, vs, c.q, c.k, c.v, c.table, c.pos, c.slots,
                                      **c.kwargs())
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    _check_rotated(c.host(out), *c.exact(c.q), rope_dim, "q")
    slots = c.slots.cpu().numpy()
    on = slots >= 0
    # v: the same fp32 divisions and roundings as the oracle, bit for bit.
    codes, scales = fp8_ref.quantize_rows(synth.bf16_bits(c.v.contiguous()))
    got_vc = vc.cpu().numpy().reshape(-1, Hkv, 128)
    got_vs = vs.cpu().numpy().transpose(0, 2, 1).reshape(-1, Hkv)
    assert np.array_equal(got_vc[slots[on]], codes[on])
    assert np.array_equal(got_vs[slots[on]], scales[on])
    # k: within half a step of the exact rotation.
    want, mag = c.exact(c.k)
    got_ks = ks.cpu().numpy().transpose(0, 2, 1).reshape(-1, Hkv)[slots[on]].astype(np.float64)
    exact_scale = np.abs(want[on]).max(-1) / 448.0
    err32 = 2.0 ** -23 * mag[on].max(-1)  # of any fp32 value of the row, and so of its amax
    assert (np.abs(got_ks - exact_scale) <= (err32 / 448 + 2.0 ** -24 * exact_scale) * 1.001).all()
    deq = fp8_ref.e4m3_decode(kc.cpu().numpy().reshape(-1, Hkv, 128)[slots[on]]) * got_ks[..., None]
    half = np.maximum(2.0 ** -4 * np.abs(want[on]), 2.0 ** -10 * got_ks[..., None])
    slack = 2 * err32[..., None] + 2.0 ** -22 * np.abs(want[on])
    assert (np.abs(deq - want[on]) <= half + slack).all()
    assert (deq[0, 0] == 0).all() and got_ks[0, 0] == 0
    left = np.ones(c.nb * BS, dtype=bool)
    left[slots[on]] = False
    assert (got_vc[left] == 0x55).all() and (got_vs[left] == 7.0).all()
    assert (kc.cpu().numpy().reshape(-1, Hkv, 128)[left] == 0x55).all()


def test_rope_write_fp8_rows_of_extreme_magnitude():
    """Rows near the type's ends and subnormal rows: v's codes and scales are those of IEEE
    fp32 divisions, bit for bit."""
    c = Case(8, 2, 2, 128, 128, seed=21)
    for t, e in enumerate((-126, -130, -133, -100, 0, 60, 120, 126)):
        c.v[t] = (c.v[t].double() * 2.0 ** e).clamp(-3e38, 3e38).to(torch.bfloat16)
    kc, vc = (torch.zeros((c.nb, BS, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((c.nb, 2, BS), device="cuda") for _ in range(2))
    api.rope_kv_cache_write_fp8(kc, vc, ks, vs, c.q, c.k, c.v, c.table, c.pos, c.slots, **c.kwargs())
    slots = c.slots.cpu().numpy()
    codes, scales = fp8_ref.quantize_rows(synth.bf16_bits(c.v))
    assert (scales[1:3] > 0).all() and (scales[1:3] < 2.0 ** -126).all()
    assert np.array_equal(vs.cpu().numpy().transpose(0, 2, 1).reshape(-1, 2)[slots], scales)
    assert np.array_equal(vc.cpu().numpy().reshape(-1, 2, 128)[slots], codes)


def test_rope_write_fp8_codes_at_every_tie():
    """Rows whose largest value has each of bf16's 128 significands, holding every significand
    at exponents over E4M3's whole range: quotients at and next to the midpoints of codes. The
    codes are those of correctly rounded fp32 quotients, bit for bit, at three magnitudes."""
    rng = np.random.default_rng(23)
    rows = np.empty((3 * 128, 9, 128))
    for r in range(3 * 128):
        top = (128 + r % 128) * 2.0 ** (-7 + (0, -60, 55)[r // 128])
        for h in range(9):
            rows[r, h] = rng.permutation(128 + np.arange(128)) * 2.0 ** (-8 - 2 * h) * 2.0 ** (
                (0, -60, 55)[r // 128]) * rng.choice([-1, 1], 128)
            rows[r, h, rng.integers(128)] = top
    c = Case(3 * 128, 1, 9, 128, 16, seed=24)
    c.v = torch.from_numpy(rows).to(torch.bfloat16).cuda()
    assert np.array_equal(c.host(c.v), rows)  # all of them bf16 values
    kc, vc = (torch.zeros((c.nb, BS, 9, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((c.nb, 9, BS), device="cuda") for _ in range(2))
    api.rope_kv_cache_write_fp8(kc, vc, ks, vs, c.q, c.k, c.v, c.table, c.pos, c.slots, **c.kwargs())
    slots = c.slots.cpu().numpy()
    codes, scales = fp8_ref.quantize_rows(synth.bf16_bits(c.v))
    assert np.array_equal(vs.cpu().numpy().transpose(0, 2, 1).reshape(-1, 9)[slots], scales)
    assert np.array_equal(vc.cpu().numpy().reshape(-1, 9, 128)[slots], codes)


def test_rope_write_fp8_rows_with_nan_and_infinities():
    """A row's scale is its largest magnitude over 448: NaN if a value is NaN, whatever the others
    are, infinite if one is infinite; either way no value of the row can be told, and all of them
    read back as NaN. Other rows of the token, and other tokens, do not change."""
    nan, inf = float("nan"), float("inf")
    c = Case(9, 4, 3, 128, 64, seed=21)
    clean = [t.clone() for t in (c.k, c.v)]
    for t in (c.k, c.v):
        t[0, 0] = nan                       # nothing but NaN
        t[1, 1] = 0
        t[1, 1, 100] = nan                  # NaN and zeros
        t[2, 2, 5] = nan                    # some NaN, in the rotated part
        t[3, 0, 127] = nan                  # and behind it
        t[4, 1, 70], t[4, 1, 71] = inf, 2.0
        t[5, 2, 90], t[5, 2, 64] = -inf, nan
    lost = torch.zeros((9, 3), dtype=torch.bool, device="cuda")
    lost[range(6), [0, 1, 2, 0, 1, 2]] = True
    got = []
    for k, v in ((c.k, c.v), clean):
        caches = [torch.full((c.nb, BS, 3, 128), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.full((c.nb, 3, BS), 7.0, device="cuda") for _ in range(2)]
        api.rope_kv_cache_write_fp8(*caches, *scales, c.q, k, v, c.table, c.pos, c.slots, **c.kwargs())
        read = api.kv_cache_read_fp8(*caches, *scales, c.slots)
        slots = c.slots.long()
        got.append([(codes.view(-1, 3, 128)[slots], s.transpose(1, 2).reshape(-1, 3)[slots], r)
                    for codes, s, r in zip(caches, scales, read)])
    assert int(c.status.item()) == 0
    for special, plain in zip(*got):
        codes, scale, rows = special
        assert torch.isnan(rows[lost]).all() and torch.isnan(scale[:4][lost[:4]]).all()
        assert torch.isinf(scale[4, 1]) and torch.isnan(scale[5, 2])
        assert ((codes[:4][lost[:4]] & 0x7F) == 0x7F).all()
        for a, b in zip(special, plain):
            assert torch.equal(a[~lost], b[~lost]) and torch.isfinite(b.float()).all()


def test_rope_write_in_place_on_a_projection_buffer():
    c = Case(200, 8, 2, 128, 128, seed=3, strided=True)
    kc, vc = (torch.zeros((c.nb, BS, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want, mag = c.exact(c.q)
    kv = c.qkv[:, 8:].clone()
    out = api.rope_kv_cache_write(kc, vc, c.q, c.k, c.v, c.table, c.pos, c.slots, q_out=c.q,
                                  **c.kwargs())
    torch.cuda.synchronize()
    assert out.data_ptr() == c.qkv.data_ptr()
    _check_rotated(c.host(c.qkv[:, :8]), want, mag, 128, "q in place")
    assert torch.equal(c.qkv[:, 8:], kv)  # the k and v columns stay as they were


def test_rope_write_bad_slot_and_bad_position_are_flagged_and_skipped():
    for fp8 in (False, True):
        c = Case(40, 4, 2, 128, 64, np.arange(32) % 3, seed=5)
        c.slots[4] = c.nb * BS
        c.pos[1, 9] = 4096
        c.pos[2, 10] = -1
        caches = [torch.zeros((c.nb, BS, 2, 128), dtype=torch.uint8 if fp8 else torch.bfloat16,
                              device="cuda") for _ in range(2)]
        q_out = torch.full((40, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        if fp8:
            scales = [torch.zeros((c.nb, 2, BS), device="cuda") for _ in range(2)]
            api.rope_kv_cache_write_fp8(*caches, *scales, c.q, c.k, c.v, c.table, c.pos, c.slots,
                                        q_out=q_out, **c.kwargs())
        else:
            api.rope_kv_cache_write(*caches, c.q, c.k, c.v, c.table, c.pos, c.slots, q_out=q_out,
                                    **c.kwargs())
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1 | api.DEV_BAD_POSITION
        assert (q_out[[9, 10]] == 3.0).all() and not (q_out[4] == 3.0).any()
        written = torch.zeros(c.nb * BS, dtype=torch.bool, device="cuda")
        keep = [t for t in range(40) if t not in (4, 9, 10)]
        written[c.slots[keep].long()] = True
        for cache in caches:
            touched = (cache.view(c.nb * BS, -1) != 0).any(1)
            assert torch.equal(touched, written)


def test_rope_write_empty_batch_and_last_slot_of_a_large_cache():
    c = Case(0, 4, 2, 128, 128, seed=6)
    small = torch.zeros((2, BS, 2, 128), dtype=torch.bfloat16, device="cuda")
    out = api.rope_kv_cache_write(small, small.clone(), c.q, c.k, c.v, c.table, c.pos, c.slots)
    assert out.shape == (0, 4, 128) and int((small != 0).sum()) == 0
    # Row offsets past 2^32 bytes: 18,000 blocks of 8 heads are 4.7 GB a cache.
    nb = 18000
    c = Case(3, 8, 8, 128, 128, seed=7, blocks=nb)
    c.slots.copy_(torch.tensor([nb * BS - 1, nb * BS - 2, 5], dtype=torch.int32))
    kc, vc = (torch.zeros((nb, BS, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.rope_kv_cache_write(kc, vc, c.q, c.k, c.v, c.table, c.pos, c.slots, **c.kwargs())
    rows = c.slots.long()
    want, mag = c.exact(c.k)
    _check_rotated(c.host(kc.view(-1, 8, 128)[rows]), want, mag, 128, "far rows")
    assert torch.equal(vc.view(-1, 8, 128)[rows], c.v)
    assert int((vc != 0).view(-1, 1024).any(1).sum()) == 3


@pytest.mark.parametrize("T,Hkv", [(1, 1), (37, 3), (1000, 8)])
def test_read_fp8_matches_oracle(T, Hkv):
    g = torch.Generator(device="cuda").manual_seed(T)
    nb = T // BS + 2
    kc, vc = (torch.randint(0, 256, (nb, BS, Hkv, 128), generator=g, device="cuda").to(torch.uint8)
              for _ in range(2))
    for t in (kc, vc):
        t[(t & 0x7F) == 0x7F] = 0x80
    ks, vs = (torch.rand((nb, Hkv, BS), generator=g, device="cuda") * 0.1 for _ in range(2))
    slots = torch.randperm(nb * BS, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 1:
        slots[0] = -5
        slots[3] = nb * BS + 1
        slots[5] = slots[4]  # the same row twice
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = api.kv_cache_read_fp8(kc, vc, ks, vs, slots, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == (1 if T > 1 else 0)
    sl = slots.cpu().numpy().copy()
    sl[sl >= nb * BS] = -1
    for got, codes, scales in ((k, kc, ks), (v, vc, vs)):
        want = rw.read_fp8(codes.cpu().numpy(), scales.cpu().numpy(), sl)
        # One fp32 product (2^-24) and one rounding to bf16 (2^-8), of a value far from the
        # subnormals.
        err = np.abs(bf16_bits_to_f64(synth.bf16_bits(got)) - want)
        assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()


def test_quantised_prefix_reaches_the_prefill_attention():
    """A prefix written with the rotary FP8 write, read back into a bf16 cache together with
    the new rows of a chunk, gives the prefill attention of the dequantised rows."""
    from oracle import paged_ref as ref

    H, Hkv, prior, new = 8, 2, 300, 45
    c = Case(prior, H, Hkv, 128, 128, seed=11)
    nb = 4
    table = np.array([[2, 0, 3]], dtype=np.int32)
    slots_np = api.build_slot_mapping(table, [0], [prior + new], BS)
    slots = torch.from_numpy(slots_np).cuda()
    c.slots = slots[:prior].contiguous()
    kc, vc = (torch.zeros((nb, BS, Hkv, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, Hkv, BS), device="cuda") for _ in range(2))
    api.rope_kv_cache_write_fp8(kc, vc, ks, vs, c.q, c.k, c.v, c.table, c.pos, c.slots)
    k, v = api.kv_cache_read_fp8(kc, vc, ks, vs, c.slots)
    kb, vb = (torch.zeros((nb, BS, Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    api.kv_cache_write(kb, vb, k, v, c.slots)
    n = Case(new, H, Hkv, 128, 128, seed=12)
    n.slots = slots[prior:].contiguous()
    q = api.rope_kv_cache_write(kb, vb, n.q, n.k, n.v, n.table, n.pos, n.slots)
    cu = torch.tensor([new], dtype=torch.int32, device="cuda")
    lens = torch.tensor([prior + new], dtype=torch.int32, device="cuda")
    out = api.paged_attention_prefill(q, cu, kb, vb, torch.from_numpy(table).cuda(), lens, 128 ** -0.5)
    o_ref, _ = ref.paged_prefill(q.double().cpu().numpy(), np.array([new]), synth.bf16_bits(kb),
                                 synth.bf16_bits(vb), table, np.array([prior + new]), BS, 128 ** -0.5)
    assert np.abs(out.cpu().numpy() - o_ref).max() <= 1e-2
    # The prefix the attention saw is the dequantised cache, rounded once to bf16.
    want = rw.read_fp8(kc.cpu().numpy(), ks.cpu().numpy(), c.slots.cpu().numpy())
    got = bf16_bits_to_f64(synth.bf16_bits(kb).reshape(-1, Hkv, 128)[c.slots.cpu().numpy()])
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()


def test_rope_write_and_read_in_a_graph_on_another_stream():
    c = Case(64, 8, 2, 128, 128, seed=13)
    caches = [torch.zeros((c.nb, BS, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((c.nb, 2, BS), device="cuda") for _ in range(2)]
    q_out = torch.empty_like(c.q)
    k, v = (torch.empty((64, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(stream=None):
        api.rope_kv_cache_write_fp8(*caches, *scales, c.q, c.k, c.v, c.table, c.pos, c.slots,
                                    q_out=q_out, stream=stream, **c.kwargs())
        api.kv_cache_read_fp8(*caches, *scales, c.slots, k_out=k, v_out=v, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)  # the stream argument, while another stream is current
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = [t.clone() for t in (q_out, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q_out, k, v):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (q_out, k, v)):
        assert torch.equal(a, b)
    # New inputs in the same buffers.
    c.q.copy_(torch.randn_like(c.q))
    c.pos.add_(17).remainder_(4096)
    graph.replay()
    torch.cuda.synchronize()
    _check_rotated(c.host(q_out), *c.exact(c.q), 128, "replayed q")


def test_entry_points_reject_bad_buffers_before_launch():
    c = Case(6, 4, 2, 128, 128, seed=14)
    kc, vc = (torch.zeros((c.nb, BS, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ok = dict(q=c.q, k=c.k, v=c.v, rope_table=c.table, positions=c.pos, slot_mapping=c.slots)
    bad = [
        dict(q=c.q.float()), dict(q=c.q[:5]), dict(q=c.q.cpu()), dict(q=c.q[..., :64]),
        dict(q=c.q.transpose(0, 1)), dict(k=c.k[:, :1]), dict(v=c.v[:, :, :64]),
        dict(rope_table=c.table.double()), dict(rope_table=c.table[0]),
        dict(positions=c.pos.long()), dict(positions=c.pos[:, :5]), dict(positions=c.pos[None]),
        dict(slot_mapping=c.slots.long()), dict(pair_axis=np.zeros(63)),
        dict(q_out=torch.empty((6, 4, 64), dtype=torch.bfloat16, device="cuda")),
        dict(q_out=torch.empty((6, 4, 128), device="cuda")),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            api.rope_kv_cache_write(kc, vc, **{**ok, **kw})
    with pytest.raises(PagedKVError, match="pair_axis"):
        api.rope_kv_cache_write(kc, vc, **ok, pair_axis=np.ones(64))
    buf = torch.zeros((7, 4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(PagedKVError, match="overlaps"):  # one token further on in the same buffer
        api.rope_kv_cache_write(kc, vc, **{**ok, "q": buf[:6]}, q_out=buf[1:])
    with pytest.raises(PagedKVError, match="aligned"):
        api.rope_kv_cache_write(kc, vc, **{**ok, "q": torch.zeros(6 * 512 + 1, dtype=torch.bfloat16,
                                                                  device="cuda")[1:].view(6, 4, 128)})
    with pytest.raises(ValueError):
        api.rope_kv_cache_write_fp8(kc, vc, c.table, c.table, **ok)
    codes = torch.zeros((c.nb, BS, 2, 128), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((c.nb, 2, BS), device="cuda")
    with pytest.raises(ValueError):
        api.kv_cache_read_fp8(codes, codes, sc, sc[:1], c.slots)
    with pytest.raises(ValueError):
        api.kv_cache_read_fp8(codes, codes, sc, sc, c.slots, k_out=torch.empty((6, 2, 128), device="cuda"))
    torch.cuda.synchronize()


def test_positions_need_a_token_axis():
    c = Case(1, 4, 2, 128, 128, seed=15)
    kc, vc = (torch.zeros((c.nb, BS, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for pos in (c.pos[0, 0], c.pos[None]):
        with pytest.raises(ValueError, match="positions"):
            api.rope_kv_cache_write(kc, vc, c.q, c.k, c.v, c.table, pos, c.slots)
    for pos in (c.pos, c.pos[0]):
        api.rope_kv_cache_write(kc, vc, c.q, c.k, c.v, c.table, pos, c.slots)
    torch.cuda.synchronize()
