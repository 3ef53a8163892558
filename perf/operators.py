"""Measured cases of the rotary cache writes, the FP8 cache read and block-sparse decode.

Six operators around the paged cache, each at sizes from one decode step to the largest
batch this repository's workloads use (`synth/workloads.py`: 64/8, 32/8 and 32/32 heads of
128, blocks of 128 tokens, sequences up to 32,768 tokens, 262,144 scattered rows):

  rope       rotary embedding of new q and k rows (one or several position axes) and the
             write of k and v into the bf16 paged cache
  rope_fp8   the same, k and v quantised to E4M3 codes with one scale per row
  read_fp8   rows of the FP8 cache widened back to bf16
  summaries  per-channel minimum and maximum of the keys of each block a step touched
  select     the blocks with the largest score bound, for each query row and kv head
  sparse     decode attention over the selected blocks

`run` computes the operators from elementary torch operations, or, where `own` is set, with
the library's calls. `exact` computes them in 64 bits from their definitions.
"""
from __future__ import annotations

import numpy as np
import torch

own = False

BS = 128          # tokens per block
D = 128           # head dimension
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def _rope(name, tokens, heads, kv_heads, sections="64", rope_dim=128, interleaved=False,
          strided=False, max_pos=32768, fp8=False):
    return {"name": name, "op": "rope_fp8" if fp8 else "rope", "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "sections": sections, "rope_dim": rope_dim,
            "interleaved": interleaved, "strided": strided, "max_pos": max_pos}


def _read(name, tokens, kv_heads):
    return {"name": name, "op": "read_fp8", "tokens": tokens, "kv_heads": kv_heads}


def _summaries(name, batch, kv_heads, new_lo, new_hi, len_hi, ragged):
    return {"name": name, "op": "summaries", "batch": batch, "kv_heads": kv_heads,
            "new_lo": new_lo, "new_hi": new_hi, "len_hi": len_hi, "ragged": ragged}


def _select(name, batch, q_len, heads, kv_heads, len_lo, len_hi, keep, ragged):
    return {"name": name, "op": "select", "batch": batch, "q_len": q_len, "heads": heads,
            "kv_heads": kv_heads, "len_lo": len_lo, "len_hi": len_hi, "keep": keep,
            "ragged": ragged}


def _sparse(name, batch, q_len, heads, kv_heads, len_lo, len_hi, keep, ragged):
    return {**_select(name, batch, q_len, heads, kv_heads, len_lo, len_hi, keep, ragged),
            "op": "sparse"}


def listed():
    return [
        # One decode step of the long-context GQA batch: one new token per sequence.
        _rope("rope decode", 64, 64, 8),
        # A prefill step over a video prompt: three position axes, q / k / v as slices of
        # one projection's output.
        _rope("rope video prefill", 16001, 32, 8, sections="16,24,24", strided=True),
        # A few decode rows into the FP8 cache, neighbouring elements paired.
        _rope("rope fp8 decode", 7, 32, 8, interleaved=True, fp8=True),
        # Prefill into the FP8 cache, half of each head rotated.
        _rope("rope fp8 prefill", 9001, 64, 8, sections="32", rope_dim=64, fp8=True),
        # The FP8 prefix of one resumed request, read back for its next prefill chunk.
        _read("read fp8 prefix", 1900, 8),
        # The prefixes of a whole batch.
        _read("read fp8 batch", 131071, 8),
        # One new key per sequence of the long-context batch.
        _summaries("summaries decode", 64, 8, 1, 1, 32768, 11),
        # Prefill chunks of 16 sequences.
        _summaries("summaries prefill", 16, 8, 1, 8192, 16384, 12),
        # Block selection of one decode step, 32 of up to 256 blocks.
        _select("select decode", 64, 1, 64, 8, 1, 32768, 32, 13),
        # Two sequences of up to a million tokens, a verified token and one draft each.
        _select("select long", 2, 2, 32, 8, 900000, 1048576, 128, 14),
        # Attention of the small MHA batch over 4 blocks per head.
        _sparse("sparse mha", 2, 1, 32, 32, 1, 2048, 4, 15),
        # Attention of the long-context batch over 32 blocks per kv head.
        _sparse("sparse gqa", 64, 1, 64, 8, 1, 32768, 32, 16),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (16, 1), (8, 4), (24, 12)])
    op = rng.choice(["rope", "rope_fp8", "read_fp8", "summaries", "select", "sparse"])
    ragged = rng.randrange(1 << 20)
    if op in ("rope", "rope_fp8"):
        rope_dim = rng.choice([128, 128, 64, 32])
        pairs = rope_dim // 2
        axes = rng.choice([1, 3])
        a = rng.randrange(1, pairs // 2)
        b = rng.randrange(1, pairs // 2)
        sections = str(pairs) if axes == 1 else "%d,%d,%d" % (a, b, pairs - a - b)
        c = _rope("", _log_int(rng, 1, 8000), heads, kv_heads, sections, rope_dim,
                  rng.random() < 0.5, rng.random() < 0.5, _log_int(rng, 512, 131072),
                  op == "rope_fp8")
    elif op == "read_fp8":
        c = _read("", _log_int(rng, 1, 100000), rng.choice([1, 4, 8]))
    elif op == "summaries":
        hi = _log_int(rng, 1, 4096)
        c = _summaries("", _log_int(rng, 1, 64), rng.choice([1, 4, 8]), 1, hi,
                       hi + rng.randrange(1, 4096), ragged)
    elif op == "select":
        q_len, batch = rng.choice([1, 1, 2, 3, 4]), _log_int(rng, 1, 64)
        c = _select("", batch, q_len, heads, kv_heads, 1,
                    _log_int(rng, 100, 2000000 // (batch * kv_heads // 8 + 1)),
                    _log_int(rng, 1, 200), ragged)
        c["len_hi"] = min(c["len_hi"], 1048576)
    else:
        q_len = rng.choice([1, 1, 2, 4])
        batch, keep = _log_int(rng, 1, 32), _log_int(rng, 1, 48)
        c = _sparse("", batch, q_len, heads, kv_heads, 1, _log_int(rng, 50, 16384), keep, ragged)
        while batch * q_len * kv_heads * c["keep"] > 8192:  # 0.5 GB of selected keys and values
            c["keep"] = c["keep"] // 2
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that a case fixes
def _lens(case):
    rng = np.random.default_rng(case["ragged"])
    if case["op"] == "summaries":
        new = rng.integers(case["new_lo"], case["new_hi"] + 1, case["batch"])
        return new + rng.integers(0, case["len_hi"] - case["new_hi"] + 1, case["batch"]), new
    return rng.integers(case["len_lo"], case["len_hi"] + 1, case["batch"]), None


def _row_blocks(case):
    """Blocks that each query row sees, [batch, q_len]."""
    lens, _ = _lens(case)
    row_len = lens[:, None] - case["q_len"] + 1 + np.arange(case["q_len"])
    return -(-np.maximum(row_len, 0) // BS)


def work(case):
    op = case["op"]
    if op in ("rope", "rope_fp8"):
        t, h, hk, rd = case["tokens"], case["heads"], case["kv_heads"], case["rope_dim"]
        axes = len(case["sections"].split(","))
        kv_out = 2 * hk * D * 2 if op == "rope" else 2 * hk * (D + 4)
        table = min(t, case["max_pos"]) * rd * 4
        return {"bytes": t * (2 * h * D * 2 + 2 * hk * D * 2 + kv_out + 4 * axes + 4) + table,
                "flops": 3 * t * (h + hk) * rd}
    if op == "read_fp8":
        rows = 2 * case["tokens"] * case["kv_heads"]
        return {"bytes": rows * (D + 4 + 2 * D) + 4 * case["tokens"], "flops": rows * D}
    if op == "summaries":
        lens, new = _lens(case)
        first = lens - new
        blocks = -(-lens // BS) - first // BS
        old = (first % BS > 0).sum()
        return {"bytes": int(case["kv_heads"] * D * 2 * (new.sum() + 2 * blocks.sum() + 2 * old)),
                "flops": int(case["kv_heads"] * D * 2 * new.sum())}
    n = _row_blocks(case)
    rows = case["batch"] * case["q_len"]
    q_bytes = rows * case["heads"] * D * 2
    if op == "select":
        # A row with no more blocks than it keeps takes them all: nothing is scored.
        scored = np.where(n > case["keep"], n, 0)
        return {"bytes": int(q_bytes + case["kv_heads"] * (scored.max(1).sum() * 2 * D * 2
                                                           + rows * case["keep"] * 4)),
                "flops": int(4 * D * case["kv_heads"] * scored.sum())}
    kept = np.minimum(n, case["keep"])
    read = np.minimum(kept.sum(1), n.max(1)).sum() * case["kv_heads"]
    return {"bytes": int(read * 2 * BS * D * 2 + 2 * q_bytes + rows * case["heads"] * 4
                         + rows * case["kv_heads"] * case["keep"] * 4),
            "flops": int(4 * BS * D * case["heads"] * kept.sum())}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _table(gen, lens, max_blocks=None):
    """Block table with distinct random blocks for every sequence; block 0 is unused."""
    need = [-(-int(n) // BS) for n in lens]
    width = max_blocks or max(1, max(need))
    order = 1 + torch.randperm(sum(need), generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 1


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, hk = case["op"], case["kv_heads"]
    s = {"case": case, "op": op}
    dev = {"device": "cuda"}
    if op in ("rope", "rope_fp8"):
        t, h, rd = case["tokens"], case["heads"], case["rope_dim"]
        sections = [int(x) for x in case["sections"].split(",")]
        qkv = _normal(gen, t, h + 2 * hk, D)
        parts = [qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]]
        if not case["strided"]:
            parts = [p.contiguous() for p in parts]
        s["q"], s["k"], s["v"] = parts
        # Rows of cos and sin per position, as a server builds them once.
        freq = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64, **dev) * 2 / rd)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, **dev)[:, None] * freq
        s["rope_table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, case["max_pos"], (len(sections), t), generator=gen,
                                       dtype=torch.int32, **dev)
        s["pair_axis"] = [a for a, n in enumerate(sections) for _ in range(n)]
        s["pair_axis_dev"] = torch.tensor(s["pair_axis"], **dev)
        nb = -(-t // BS) + 64
        s["slots"] = torch.randperm(nb * BS, generator=gen, **dev)[:t].to(torch.int32)
        if op == "rope":
            s["k_cache"], s["v_cache"] = _normal(gen, nb, BS, hk, D), _normal(gen, nb, BS, hk, D)
        else:
            s["k_cache"], s["v_cache"] = (torch.zeros((nb, BS, hk, D), dtype=torch.uint8, **dev)
                                          for _ in range(2))
            s["k_scale"], s["v_scale"] = (torch.zeros((nb, hk, BS), **dev) for _ in range(2))
        s["q_out"] = torch.empty((t, h, D), dtype=torch.bfloat16, **dev)
    elif op == "read_fp8":
        t = case["tokens"]
        nb = -(-t // BS) + 8
        for n in ("k", "v"):
            s[n + "_cache"] = (_normal(gen, nb, BS, hk, D).float() * 100).clamp(-448, 448).to(
                E4M3).view(torch.uint8)
            s[n + "_scale"] = torch.rand((nb, hk, BS), generator=gen, **dev) * 0.02 + 1e-3
            s[n + "_out"] = torch.empty((t, hk, D), dtype=torch.bfloat16, **dev)
        s["slots"] = torch.randperm(nb * BS, generator=gen, **dev)[:t].to(torch.int32)
    elif op == "summaries":
        lens, new = _lens(case)
        s["table"], nb = _table(gen, lens)
        s["k_cache"] = _normal(gen, nb, BS, hk, D)
        # Every block's summary as the steps before left it.
        a, b = _normal(gen, nb, hk, D), _normal(gen, nb, hk, D)
        s["summaries"] = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2).contiguous()
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, **dev)
        s["num_new"] = torch.tensor(new, dtype=torch.int32, **dev)
        s["max_new"] = int(new.max())
    else:
        lens, _ = _lens(case)
        b, ql, h, keep = case["batch"], case["q_len"], case["heads"], case["keep"]
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, **dev)
        s["table"], nb = _table(gen, lens)
        s["q"] = _normal(gen, b, ql, h, D)
        if op == "select":
            # Keys of a block scatter around the block's own direction.
            mid = 0.5 * _normal(gen, nb, hk, D).float()
            half = 2.0 + 0.5 * torch.rand((nb, hk, D), generator=gen, **dev)
            s["summaries"] = torch.stack([mid - half, mid + half], 2).to(torch.bfloat16)
            s["out"] = torch.empty((b, ql, hk, keep), dtype=torch.int32, **dev)
        else:
            s["k_cache"], s["v_cache"] = _normal(gen, nb, BS, hk, D), _normal(gen, nb, BS, hk, D)
            # Each row's last block and random ones before it, ascending, as the selection
            # returns them.
            n = torch.tensor(_row_blocks(case), **dev)[:, :, None, None]
            j = torch.arange(s["table"].shape[1], **dev)
            key = torch.rand((b, ql, hk, len(j)), generator=gen, **dev)
            key = torch.where(j == n - 1, 2.0, torch.where(j < n, key, -1.0))
            k_eff = min(keep, len(j))
            top = key.topk(k_eff, -1)
            idx = torch.where(top.values >= 0, top.indices, 1 << 30).sort(-1).values
            idx = torch.where(idx == 1 << 30, -1, idx).to(torch.int32)
            s["block_indices"] = torch.full((b, ql, hk, keep), -1, dtype=torch.int32, **dev)
            s["block_indices"][..., :k_eff] = idx
            s["out"] = torch.empty((b, ql, h, D), dtype=torch.bfloat16, **dev)
            s["lse"] = torch.empty((b, ql, h), **dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_cache_77_gb300 import api

    op = s["op"]
    if op == "rope":
        api.rope_kv_cache_write(s["k_cache"], s["v_cache"], s["q"], s["k"], s["v"],
                                s["rope_table"], s["positions"], s["slots"],
                                pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"],
                                q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "rope_fp8":
        api.rope_kv_cache_write_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q"],
                                    s["k"], s["v"], s["rope_table"], s["positions"], s["slots"],
                                    pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"],
                                    q_out=s["q_out"])
        return (s["q_out"], s["k_cache"].view(E4M3), s["v_cache"].view(E4M3), s["k_scale"],
                s["v_scale"])
    if op == "read_fp8":
        return api.kv_cache_read_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                     s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    if op == "summaries":
        api.update_block_summaries(s["summaries"], s["k_cache"], s["table"], s["seq_lens"],
                                   s["num_new"], s["max_new"])
        return s["summaries"]
    if op == "select":
        return api.select_blocks(s["q"], s["summaries"], s["table"], s["seq_lens"],
                                 s["case"]["keep"], out=s["out"])
    if "workspace" not in s:  # kept for the process, as a server keeps it
        b, ql, h, _ = s["q"].shape
        s["workspace"] = torch.empty(
            api.decode_sparse_workspace_size(b, ql, h, s["case"]["kv_heads"], D),
            dtype=torch.uint8, device="cuda")
    api.paged_attention_decode_sparse(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                      s["seq_lens"], s["block_indices"], D ** -0.5, out=s["out"],
                                      lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _rotate(x, cos, sin, interleaved):
    """Rotary embedding of the leading dimensions of [T, heads, D], in 32 bits."""
    x = x.float()
    pairs = cos.shape[1]
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        rot = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        rot = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([rot, x[..., 2 * pairs:]], -1)


def _run_plain(s):
    op, case = s["op"], s["case"]
    if op in ("rope", "rope_fp8"):
        pairs = case["rope_dim"] // 2
        at = s["positions"].long()[s["pair_axis_dev"]].t()  # [T, pairs]: the row of each pair
        cos = s["rope_table"][:, :pairs].gather(0, at)
        sin = s["rope_table"][:, pairs:].gather(0, at)
        s["q_out"].copy_(_rotate(s["q"], cos, sin, case["interleaved"]))
        k = _rotate(s["k"], cos, sin, case["interleaved"])
        slots = s["slots"].long()
        hk = case["kv_heads"]
        if op == "rope":
            s["k_cache"].view(-1, hk, D)[slots] = k.to(torch.bfloat16)
            s["v_cache"].view(-1, hk, D)[slots] = s["v"]
            return s["q_out"], s["k_cache"], s["v_cache"]
        for name, x in (("k", k), ("v", s["v"].float())):
            scale = x.abs().amax(-1) / 448.0
            code = (x / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(-448, 448).to(E4M3)
            s[name + "_cache"].view(-1, hk, D)[slots] = code.view(torch.uint8)
            s[name + "_scale"][slots // BS, :, slots % BS] = scale
        return (s["q_out"], s["k_cache"].view(E4M3), s["v_cache"].view(E4M3), s["k_scale"],
                s["v_scale"])
    if op == "read_fp8":
        slots = s["slots"].long()
        hk = case["kv_heads"]
        k = s["k_cache"].view(-1, hk, D)[slots].view(E4M3).float()
        v = s["v_cache"].view(-1, hk, D)[slots].view(E4M3).float()
        k = k * s["k_scale"][slots // BS, :, slots % BS][..., None]
        v = v * s["v_scale"][slots // BS, :, slots % BS][..., None]
        s["k_out"].copy_(k)
        s["v_out"].copy_(v)
        return s["k_out"], s["v_out"]
    if op == "summaries":
        lens, new, table = s["seq_lens"].long(), s["num_new"].long(), s["table"].long()
        span = (s["max_new"] + BS - 2) // BS + 1
        j = (lens - new)[:, None] // BS + torch.arange(span, device="cuda")  # [B, span]
        live = j * BS < lens[:, None]
        block = torch.where(live, table.gather(1, j.clamp(max=table.shape[1] - 1)), 0)
        rows = s["k_cache"][block]  # [B, span, BS, Hkv, D]
        pos = j[:, :, None] * BS + torch.arange(BS, device="cuda")
        fresh = (pos >= (lens - new)[:, None, None]) & (pos < lens[:, None, None])
        fresh = fresh[..., None, None]
        lo = torch.where(fresh, rows, torch.inf).amin(2)
        hi = torch.where(fresh, rows, -torch.inf).amax(2)
        old = s["summaries"][block]  # [B, span, Hkv, 2, D]
        begun = (j * BS < (lens - new)[:, None])[..., None, None]
        lo = torch.where(begun, torch.minimum(lo, old[..., 0, :]), lo)
        hi = torch.where(begun, torch.maximum(hi, old[..., 1, :]), hi)
        both = torch.where(live[..., None, None, None], torch.stack([lo, hi], 3), old)
        s["summaries"][block] = both
        return s["summaries"]
    b, ql, h, _ = s["q"].shape
    hk = case["kv_heads"]
    row_len = s["seq_lens"][:, None] - ql + 1 + torch.arange(ql, device="cuda")  # [B, ql]
    if op == "select":
        # Which block is the last one kept can hang on the last bits of two scores: 64 bits.
        q = s["q"].double().view(b, ql, hk, h // hk, D)
        weight = torch.cat([q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)], -1)  # [B, ql, Hkv, 2D]
        ends = s["summaries"][s["table"].long()].double().flatten(-2)  # [B, n, Hkv, 2D]
        score = weight.transpose(1, 2) @ ends.permute(0, 2, 3, 1)  # [B, Hkv, ql, n]
        score = score.transpose(1, 2)
        n = ((row_len.clamp(min=0) + BS - 1) // BS)[:, :, None, None]
        j = torch.arange(score.shape[-1], device="cuda")
        score = torch.where(j == n - 1, torch.inf, score)  # the newest block is always kept
        score = torch.where(j < n, score, -torch.inf)
        idx = score.sort(dim=-1, descending=True, stable=True).indices[..., :case["keep"]]
        idx = torch.where(idx < n, idx, 1 << 30).sort(-1).values
        s["out"].fill_(-1)
        s["out"][..., :idx.shape[-1]] = torch.where(idx == 1 << 30, -1, idx).to(torch.int32)
        return s["out"]
    idx = s["block_indices"].long()  # [B, ql, Hkv, keep]
    seq = torch.arange(b, device="cuda")[:, None, None, None]
    block = s["table"].long()[seq, idx.clamp(min=0)]
    kv = torch.arange(hk, device="cuda")[:, None]
    keys = s["k_cache"][block, :, kv].flatten(3, 4).float()  # [B, ql, Hkv, keep * BS, D]
    vals = s["v_cache"][block, :, kv].flatten(3, 4).float()
    pos = (idx[..., None] * BS + torch.arange(BS, device="cuda")).flatten(3)
    seen = (idx >= 0).repeat_interleave(BS, -1) & (pos < row_len[:, :, None, None])
    q = s["q"].float().view(b, ql, hk, h // hk, D)
    score = (q @ keys.transpose(-1, -2)) * D ** -0.5
    score = torch.where(seen[..., None, :], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ vals) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.reshape(b, ql, h, D))
    s["lse"].copy_((top + total.log()).reshape(b, ql, h))
    return s["out"], s["lse"]


# ------------------------------------------------------------------ 64-bit results
def _e4m3(x):
    """x rounded to the nearest E4M3 value (ties to even, largest 448), in 64 bits."""
    mag = x.abs()
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(((mag / step).round() * step).clamp(max=448.0), x)


def exact(case, seed):
    s = prepare(case, seed)
    op, hk = case["op"], case["kv_heads"]
    if op in ("rope", "rope_fp8"):
        pairs = case["rope_dim"] // 2
        table = s["rope_table"].double()
        turn = torch.empty((case["tokens"], pairs), dtype=torch.complex128, device="cuda")
        for i, axis in enumerate(s["pair_axis"]):
            p = s["positions"][axis].long()
            turn[:, i] = torch.complex(table[p, i], table[p, pairs + i])

        def rotated(x):
            y = x.double().clone()
            first = slice(0, 2 * pairs, 2) if case["interleaved"] else slice(0, pairs)
            second = slice(1, 2 * pairs, 2) if case["interleaved"] else slice(pairs, 2 * pairs)
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        out = [rotated(s["q"])]
        rows = {"k": rotated(s["k"]), "v": s["v"].double()}
        slots, scales = s["slots"].long(), []
        for name in ("k", "v"):
            x = rows[name]
            if op == "rope_fp8":
                scale = x.abs().amax(-1) / 448.0
                x = _e4m3(x / scale.clamp(min=1e-300)[..., None])
                full = s[name + "_scale"].double().transpose(1, 2).reshape(-1, hk)
                full[slots] = scale
                scales.append(full.view(-1, BS, hk).transpose(1, 2).contiguous())
                cache = s[name + "_cache"].view(E4M3).double()
            else:
                cache = s[name + "_cache"].double()
            cache.view(-1, hk, D)[slots] = x
            out.append(cache)
        return tuple(out + scales)
    if op == "read_fp8":
        slots = s["slots"].long()
        return tuple(
            s[n + "_cache"].view(-1, hk, D)[slots].view(E4M3).double()
            * s[n + "_scale"].double().transpose(1, 2).reshape(-1, hk)[slots][..., None]
            for n in ("k", "v"))
    if op == "summaries":
        out = s["summaries"].double()
        lens, new = _lens(case)
        table = s["table"].cpu().numpy()
        for b in range(case["batch"]):
            end, pos = int(lens[b]), int(lens[b] - new[b])
            while pos < end:
                block = int(table[b, pos // BS])
                stop = min(end, (pos // BS + 1) * BS)
                rows = s["k_cache"][block, pos % BS:(stop - 1) % BS + 1].double()
                lo, hi = rows.amin(0), rows.amax(0)
                if pos % BS:
                    lo = torch.minimum(lo, out[block, :, 0])
                    hi = torch.maximum(hi, out[block, :, 1])
                out[block, :, 0], out[block, :, 1] = lo, hi
                pos = stop
        return out
    if op == "select":
        return None  # whole numbers
    b, ql, h, _ = s["q"].shape
    out = torch.zeros((b, ql, h, D), dtype=torch.float64, device="cuda")
    lse = torch.full((b, ql, h), -torch.inf, dtype=torch.float64, device="cuda")
    lens, _ = _lens(case)
    for i in range(b):
        for r in range(ql):
            end = int(lens[i]) - ql + 1 + r
            if end <= 0:
                continue
            idx = s["block_indices"][i, r].long()  # [Hkv, keep]
            block = s["table"][i].long()[idx.clamp(min=0)]
            pos = idx[..., None] * BS + torch.arange(BS, device="cuda")
            seen = ((pos >= 0) & (pos < end)).flatten(1)
            kv = torch.arange(hk, device="cuda")[:, None]
            keys = s["k_cache"][block, :, kv].double().flatten(1, 2)
            vals = s["v_cache"][block, :, kv].double().flatten(1, 2)
            q = s["q"][i, r].double().view(hk, h // hk, D)
            score = torch.einsum("gnd,gtd->gnt", q, keys) / D ** 0.5
            score.masked_fill_(~seen[:, None], -torch.inf)
            lse[i, r] = torch.logsumexp(score, -1).flatten()
            weight = torch.exp(score - lse[i, r].view(hk, -1, 1))
            out[i, r] = torch.einsum("gnt,gtd->gnd", weight, vals).reshape(h, D)
    return out, lse
