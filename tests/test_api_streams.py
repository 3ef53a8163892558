"""Tensors that the binding makes for a launch on a stream other than the current one.

The caching allocator hands a freed block out again to the stream it was made for, without
waiting for work on any other: a workspace that a call drops at its return, and an output whose
memory the current stream may still be using, have to be made for the launch's own stream."""
import contextlib

import numpy as np
import pytest
import torch

from paged_kv_cache_77_gb300 import api

CPU = torch.device("cpu")


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeCuda:
    """torch.cuda's current stream, and what was made and recorded under which."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.recorded = FakeStream(7), [], []
        real = torch.empty

        @contextlib.contextmanager
        def under(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        class Made(torch.Tensor):
            def record_stream(t, stream):
                self.recorded.append(stream.cuda_stream)

        def empty(*args, **kw):
            self.made.append(self.current.cuda_stream)
            return real(*args, **kw).as_subclass(Made)

        monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("stream,made", [(None, 7), (FakeStream(7), 7), (FakeStream(9), 9)])
def test_buffers_are_made_for_the_stream_of_the_launch(monkeypatch, stream, made):
    cuda = FakeCuda(monkeypatch)
    ws, n = api.workspace_buffer(None, 1000, CPU, stream=stream)
    assert n >= 1000 and cuda.made == [made] and cuda.recorded == []
    out = api.out_buffer(None, (2, 3), torch.float32, CPU, stream=stream)
    assert out.shape == (2, 3) and cuda.made == [made, made]
    # A tensor that the caller gets is used on the current stream too.
    assert cuda.recorded == ([] if made == 7 else [7])
    assert cuda.current.cuda_stream == 7


def test_buffers_that_are_given_are_used_as_they_are(monkeypatch):
    cuda = FakeCuda(monkeypatch)
    ws = torch.zeros(1000, dtype=torch.uint8)
    assert api.workspace_buffer(ws, 1000, CPU, stream=FakeStream(9))[0] is ws
    out = torch.zeros((2, 3))
    assert api.out_buffer(out, (2, 3), torch.float32, CPU, stream=FakeStream(9)) is out
    assert cuda.made == cuda.recorded == []


class Calls:
    """Every call that makes tensors, on small inputs."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)
        rows = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        q, q2, kc, vc = rows(2, 8, 128), rows(2, 2, 8, 128), rows(9, 128, 2, 128), rows(9, 128, 2, 128)
        t, lens, idx = ints([[1, 2, 3, 4], [5, 6, 7, 8]]), ints([500, 300]), ints([[[0, 2]] * 2] * 2)
        codes = [torch.zeros((9, 128, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((9, 2, 128), device="cuda") for _ in range(2)]
        rope, pos = torch.rand((600, 128), generator=g, device="cuda"), ints(list(range(500)))
        slots = (torch.arange(500, device="cuda") + 128).int()
        qr, kr, vr = rows(500, 8, 128), rows(500, 2, 128), rows(500, 2, 128)
        s = rows(9, 2, 2, 128)
        fp8 = (*codes, *scales)
        api.kv_cache_write_fp8(*fp8, kr, vr, slots)
        qn, qp, cn, cp = rows(2, 16, 512), rows(2, 16, 64), rows(9, 128, 1, 512), rows(9, 128, 1, 64)
        qn2, qp2 = rows(2, 2, 16, 512), rows(2, 2, 16, 64)
        cu = ints([5, 8])
        side = dict(k_cache=torch.zeros_like(kc), v_cache=torch.zeros_like(vc))
        self.calls = {
            "rope": lambda **k: api.rope_kv_cache_write(**side, q=qr, k=kr, v=vr, rope_table=rope,
                                                        positions=pos, slot_mapping=slots, **k),
            "rope fp8": lambda **k: api.rope_kv_cache_write_fp8(*fp8, qr, kr, vr, rope, pos, slots, **k),
            "read": lambda **k: torch.stack(api.kv_cache_read_fp8(*fp8, slots, **k)),
            "select": lambda **k: api.select_blocks(q, s, t, lens, 2, **k),
            "sparse": lambda **k: api.paged_attention_decode_sparse(q, kc, vc, t, lens, idx, 0.1, **k),
            "decode": lambda **k: api.paged_attention_decode(q, kc, vc, t, lens, 0.1, **k),
            "fp8": lambda **k: api.paged_attention_decode_fp8(q, *fp8, t, lens, 0.1, **k),
            "spec": lambda **k: api.paged_attention_decode_spec(q2, kc, vc, t, lens, 0.1, **k),
            "static": lambda **k: api.paged_attention_decode_static(q, kc, vc, t, lens, 0.1, **k),
            "prefill": lambda **k: api.paged_attention_prefill(qr[:8], cu, kc, vc, t, lens, 0.1, **k),
            "mla": lambda **k: api.mla_paged_decode(qn, qp, cn, cp, t, lens, 0.1, **k),
            "mla spec": lambda **k: api.mla_paged_decode_spec(qn2, qp2, cn, cp, t, lens, 0.1, **k),
        }


@pytest.mark.gpu
def test_every_call_makes_its_tensors_for_its_own_stream(monkeypatch):
    calls, side = Calls().calls, torch.cuda.Stream()
    torch.cuda.synchronize()
    want = {name: call() for name, call in calls.items()}
    torch.cuda.synchronize()
    real, made = torch.empty, []

    def empty(*args, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return real(*args, **kw)

    for handle in (side, type("Handle", (), {"cuda_stream": side.cuda_stream})()):
        for name, call in calls.items():
            made.clear()
            with monkeypatch.context() as m:
                m.setattr(torch, "empty", empty)
                if name == "read":  # (stacked on the current stream)
                    m.setattr(torch, "stack", lambda x: x)
                got = call(stream=handle)
            assert made and set(made) == {side.cuda_stream}, name
            torch.cuda.synchronize()
            got = torch.stack(got) if name == "read" else got
            assert torch.equal(got, want[name]), name


@pytest.mark.gpu
def test_two_calls_at_once_on_two_streams_with_tensors_of_their_own():
    """Long queues on two streams, no buffer given, while the current stream fills memory of the
    same sizes: every result is that of the call alone."""
    rng = np.random.default_rng(5)
    B, hkv, nb, K = 8, 8, 300, 24
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (torch.randn((nb, 128, hkv, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    t = torch.from_numpy(rng.integers(0, nb, (B, 64)).astype(np.int32)).cuda()
    lens = torch.from_numpy(rng.integers(5000, 8193, B).astype(np.int32)).cuda()
    idx = torch.from_numpy(rng.integers(0, 39, (B, hkv, K)).astype(np.int32)).cuda()
    qs = [torch.randn((B, 64, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [api.paged_attention_decode_sparse(q, kc, vc, t, lens, idx, 0.1) for q in qs]
    need = api.decode_sparse_workspace_size(B, 1, 64, hkv, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for i in range(2):
            got.append((i, api.paged_attention_decode_sparse(qs[i], kc, vc, t, lens, idx, 0.1,
                                                             stream=streams[i])))
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
            torch.empty(want[0].shape, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    for i, out in got:
        assert torch.equal(out, want[i])


@pytest.mark.gpu
def test_calls_on_a_forked_stream_inside_a_capture_make_their_tensors_in_the_graph():
    """Selection and sparse attention on a side stream of a captured graph, no buffer given: the
    replays follow their inputs while other graphs and eager calls use the allocator."""
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc, s, q = rows(9, 128, 2, 128), rows(9, 128, 2, 128), rows(9, 2, 2, 128), rows(1, 16, 128)
    t = torch.arange(9, dtype=torch.int32, device="cuda").view(1, 9)
    lens = torch.tensor([1100], dtype=torch.int32, device="cuda")

    def step(stream=None):
        idx = api.select_blocks(q, s, t, lens, 4, stream=stream)
        return api.paged_attention_decode_sparse(q, kc, vc, t, lens, idx, 0.1, stream=stream)

    side = torch.cuda.Stream()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
