"""Eviction calls directly behind the calls whose results they read (GPU)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_77_gb300 import api
from tests.test_gpu_evict import D, ints, keys_of, make_table

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
