"""Measured cases of the 4-bit cache and of eviction by accumulated attention weight.

Six operators that make a paged cache hold more, each at sizes from one decode step to the
largest batch this repository's workloads use (`synth/workloads.py`: 64/8, 32/8 and 32/32
heads of 128, blocks of 128 tokens, sequences up to 32,768 tokens):

  write    new k and v rows quantised to 4 bits (E2M1 codes, one 8-bit scale per 16 values)
           and written into the paged cache, then read back: a prompt chunk whose prefill
           attends to what the later decode steps will attend to
  read     rows of the 4-bit cache widened to bf16
  decode   attention of one or a few new tokens per sequence over the 4-bit cache
  weights  the attention that a step pays to each cached row, added to the row's running sum
  select   the rows of each sequence and kv head with the largest sums, sinks and newest kept
  compact  the kept rows moved to the front of the sequence, in place or into new blocks (and
           read back from the 4-bit cache, for the next prefill chunk)

A 4-bit row of 128 values is 64 bytes (element 2i in the low half of byte i) and 8 scales. A
scale is the upper 8 of the 15 bits of a positive fp16 (5 bits of exponent, 3 of fraction):
the nearest one to a sixth of the 16 values' largest magnitude, 10240 at most. A code is the
nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) to the quotient; ties go
to the even code.

`run` computes the operators from elementary torch operations, or, where `own` is set, with
the library's calls. `exact` computes them in 64 bits from their definitions.
"""
from __future__ import annotations

import numpy as np
import torch

own = False

BS = 128          # tokens per block
D = 128           # head dimension
GROUP = 16        # values per scale
E4M3 = torch.float8_e4m3fn
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE_MAX = 10240.0   # 6 of it still fit fp16
ROW_BYTES = {"bf16": 256, "fp8": 132, "fp4": 72}  # codes and scales of one row


# ------------------------------------------------------------------ cases
def _rows(op, name, tokens, kv_heads, strided=False):
    return {"name": name, "op": op, "tokens": tokens, "kv_heads": kv_heads, "strided": strided}


def _batch(op, name, batch, kv_heads, len_lo, len_hi, ragged, **more):
    return {"name": name, "op": op, "batch": batch, "kv_heads": kv_heads, "len_lo": len_lo,
            "len_hi": len_hi, "ragged": ragged, **more}


def listed():
    return [
        # One decode step of the long-context GQA batch: one new token per sequence.
        _rows("write", "write decode", 64, 8),
        # A prefill step of one long prompt, v as a slice of the projection's output.
        _rows("write", "write prefill", 16001, 8, strided=True),
        # The prefix of one resumed request, read back for its next prefill chunk.
        _rows("read", "read prefix", 1900, 8),
        # The prefixes of a whole batch.
        _rows("read", "read batch", 131071, 8),
        # A small batch of short sequences, one kv head per query head.
        _batch("decode", "decode mha", 2, 32, 1, 2048, 21, q_len=1, heads=32),
        # The long-context GQA batch.
        _batch("decode", "decode gqa", 64, 8, 1, 32768, 22, q_len=1, heads=64),
        # A few sequences with three draft tokens each, over the 4-bit cache.
        _batch("weights", "weights draft fp4", 7, 8, 1, 8192, 23, q_len=4, heads=32, cache="fp4"),
        # One decode step of the long-context batch over the bf16 cache.
        _batch("weights", "weights decode bf16", 64, 8, 1, 32768, 24, q_len=1, heads=64,
               cache="bf16"),
        # The long-context batch cut down to 4,096 rows per sequence and kv head.
        _batch("select", "select batch", 64, 8, 1, 32768, 25, keep=4096, sink=4, recent=256),
        # Two sequences of about a million tokens.
        _batch("select", "select long", 2, 8, 900000, 1048576, 26, keep=65536, sink=4,
               recent=1024),
        # Every 128 steps a batch of sequences that holds 2,048 rows each drops the newest excess.
        _batch("compact", "compact in place bf16", 64, 8, 2049, 2176, 27, keep=2048, sink=4,
               recent=256, cache="bf16", fresh_blocks=False),
        # Prompts cut down after their prefill, into blocks of their own (the old ones may be
        # shared with other requests).
        _batch("compact", "compact prompts fp4", 16, 8, 1, 16384, 28, keep=2000, sink=4,
               recent=64, cache="fp4", fresh_blocks=True),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (16, 1), (8, 4), (24, 12)])
    op = rng.choice(["write", "read", "decode", "weights", "select", "compact"])
    ragged = rng.randrange(1 << 20)
    if op in ("write", "read"):
        c = _rows(op, "", _log_int(rng, 1, 12000 if op == "write" else 100000),
                  rng.choice([1, 4, 8]), op == "write" and rng.random() < 0.5)
    elif op in ("decode", "weights"):
        q_len = rng.choice([1, 1, 2, 3, 4] if heads // kv_heads <= 8 else [1, 1, 2])
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 50, min(131072, 6000000 // (batch * kv_heads)))
        c = _batch(op, "", batch, kv_heads, 1, hi, ragged, q_len=q_len, heads=heads)
        if op == "weights":
            c["cache"] = rng.choice(["bf16", "fp8", "fp4"])
    elif op == "select":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 100, min(1048576, 8000000 // (batch * kv_heads)))
        keep = _log_int(rng, 10, max(10, hi // 2))
        c = _batch(op, "", batch, kv_heads, 1, hi, ragged, keep=keep, sink=rng.choice([0, 1, 4]),
                   recent=rng.randrange(0, keep - 4))
    else:
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 100, min(32768, 1000000 // (batch * kv_heads)))
        keep = _log_int(rng, 20, max(20, hi // 2))
        c = _batch(op, "", batch, kv_heads, 1, hi, ragged, keep=keep, sink=rng.choice([0, 1, 4]),
                   recent=rng.randrange(0, keep - 4), cache=rng.choice(["bf16", "fp4"]),
                   fresh_blocks=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that a case fixes
def _lens(case):
    rng = np.random.default_rng(case["ragged"])
    return rng.integers(case["len_lo"], case["len_hi"] + 1, case["batch"])


def work(case):
    op, hk = case["op"], case["kv_heads"]
    if op in ("write", "read"):
        rows = 2 * case["tokens"] * hk
        if op == "read":
            return {"bytes": rows * (72 + 2 * D) + 4 * case["tokens"], "flops": rows * D}
        return {"bytes": rows * (2 * D + 72 + 2 * D) + 4 * case["tokens"], "flops": 4 * rows * D}
    lens = _lens(case)
    total = int(lens.sum())
    if op == "select":
        # A sequence with no more rows than it keeps takes them all: nothing is ranked.
        ranked = int(lens[lens > case["keep"]].sum())
        return {"bytes": 4 * hk * (ranked + case["batch"] * case["keep"]), "flops": hk * ranked}
    if op == "compact":
        kept = np.minimum(lens, case["keep"])
        if not case["fresh_blocks"]:  # the rows in front of the first one dropped stay
            kept = np.where(lens > case["keep"], case["keep"] - case["sink"], 0)
        row = {"bf16": 512, "fp4": 144}[case["cache"]] + 4
        back = 512 * int(np.minimum(lens, case["keep"]).sum()) if case["cache"] == "fp4" else 0
        return {"bytes": int(hk * (kept.sum() * 2 * row + back + case["batch"] * case["keep"] * 4)),
                "flops": 0}
    rows, h = case["batch"] * case["q_len"], case["heads"]
    if op == "decode":
        return {"bytes": total * hk * 144 + rows * h * (4 * D + 4),
                "flops": 4 * D * h * case["q_len"] * total}
    return {"bytes": total * hk * (ROW_BYTES[case["cache"]] + 8) + rows * h * (2 * D + 4),
            "flops": 2 * D * h * case["q_len"] * total}


# ------------------------------------------------------------------ the 4-bit format
def _fp4_pairs():
    """[256, 2] fp32: the two values of a byte of codes."""
    one = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    byte = torch.arange(256, device="cuda")
    return torch.stack([one[byte & 15], one[byte >> 4]], 1)


def _fp4_scale(u):
    """fp32 values of scale bytes."""
    return (u.to(torch.int16) << 7).view(torch.float16).float()


def _fp4_values(codes, scales, pairs):
    """fp32 [..., 128] of codes [..., 64] and scales [..., 8]."""
    x = pairs[codes.long()].flatten(-2).unflatten(-1, (-1, GROUP))
    return (x * _fp4_scale(scales)[..., None]).flatten(-2)


def _fp4_quantise(x):
    """(codes [..., 64], scales [..., 8]) of rows [..., 128]. What decides is compared in 64
    bits, where every product and quotient at a border between two codes is exact."""
    g = x.double().unflatten(-1, (-1, GROUP))
    want = (g.abs().amax(-1) / 6).clamp(max=SCALE_MAX)
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -14))) - 3)
    scale = torch.round(want / step) * step
    scale16 = scale.to(torch.float16).view(torch.int16) >> 7
    r = g / torch.where(scale > 0, scale, torch.inf)[..., None]
    mag = r.abs()
    code = sum((mag > t).to(torch.uint8) for t in (0.25, 1.25, 2.5, 5.0))
    code = code + sum((mag >= t).to(torch.uint8) for t in (0.75, 1.75, 3.5))
    code = code | ((r < 0).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale16.to(torch.uint8)


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _table(gen, lens):
    """Block table with distinct random blocks for every sequence; block 0 is unused."""
    need = [-(-int(n) // BS) for n in lens]
    order = 1 + torch.randperm(sum(need), generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 1


def _fp4_cache(gen, nb, hk):
    """A cache of normal values whose channels differ in magnitude, as those of keys do."""
    codes = torch.empty((nb, hk, BS, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((nb, hk, BS, D // GROUP), dtype=torch.uint8, device="cuda")
    channel = 0.25 + 2.0 * torch.rand((hk, 1, D), generator=gen, device="cuda")
    for lo in range(0, nb, 512):
        x = _normal(gen, min(512, nb - lo), hk, BS, D).float() * channel
        codes[lo:lo + 512], scales[lo:lo + 512] = _fp4_quantise(x.to(torch.bfloat16))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, hk = case["op"], case["kv_heads"]
    dev = {"device": "cuda"}
    s = {"case": case, "op": op, "pairs": _fp4_pairs()}
    if op in ("write", "read"):
        t = case["tokens"]
        nb = -(-t // BS) + 8
        s["slots"] = torch.randperm(nb * BS, generator=gen, **dev)[:t].to(torch.int32)
        s["k_cache"], s["k_scale"] = _fp4_cache(gen, nb, hk)
        s["v_cache"], s["v_scale"] = _fp4_cache(gen, nb, hk)
        s["k_out"], s["v_out"] = (torch.empty((t, hk, D), dtype=torch.bfloat16, **dev)
                                  for _ in range(2))
        if op == "write":
            s["k"] = _normal(gen, t, hk, D)
            s["v"] = _normal(gen, t, 3 * hk, D)[:, 2 * hk:] if case["strided"] else _normal(
                gen, t, hk, D)
        return s
    lens = _lens(case)
    s["lens"] = lens
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, **dev)
    s["table"], nb = _table(gen, lens)
    b = case["batch"]
    if op in ("decode", "weights"):
        ql, h = case["q_len"], case["heads"]
        cache = case.get("cache", "fp4")
        s["q"] = _normal(gen, b, ql, h, D)
        if cache == "fp4":
            s["k_cache"], s["k_scale"] = _fp4_cache(gen, nb, hk)
        elif cache == "fp8":
            s["k_cache"] = (_normal(gen, nb, BS, hk, D).float() * 100).clamp(-448, 448).to(
                E4M3).view(torch.uint8)
            s["k_scale"] = torch.rand((nb, hk, BS), generator=gen, **dev) * 0.01 + 5e-3
        else:
            s["k_cache"], s["k_scale"] = _normal(gen, nb, BS, hk, D), None
        if op == "decode":
            s["v_cache"], s["v_scale"] = _fp4_cache(gen, nb, hk)
            s["out"] = torch.empty((b, ql, h, D), dtype=torch.bfloat16, **dev)
            s["lse"] = torch.empty((b, ql, h), **dev)
        else:
            # The log-sum-exp that the step's attention returned for each query row.
            s["lse"] = _lse(s)
            s["weights"] = torch.rand((nb, hk, BS), generator=gen, **dev) * 0.1
            # The step's own rows are new; what their places held before does not count.
            s["num_fresh"] = torch.minimum(s["seq_lens"],
                                           torch.tensor(ql, dtype=torch.int32, **dev))
        return s
    if op == "select":
        # Sums of attention weights spread over orders of magnitude.
        s["weights"] = torch.exp(2.5 * torch.randn((nb, hk, BS), generator=gen, **dev) - 8)
        s["out"] = torch.empty((b, hk, case["keep"]), dtype=torch.int32, **dev)
        return s
    # compact: sinks, the newest rows and random ones between them, as the selection returns them
    n = s["seq_lens"].long()[:, None, None]
    j = torch.arange(int(lens.max()), **dev)
    key = torch.rand((b, hk, len(j)), generator=gen, **dev)
    key = torch.where((j < case["sink"]) | (j >= n - case["recent"]), 2.0, key)
    key = torch.where(j < n, key, -1.0)
    top = key.topk(min(case["keep"], len(j)), -1)
    kept = torch.where(top.values >= 0, top.indices, 1 << 30).sort(-1).values
    s["kept"] = torch.full((b, hk, case["keep"]), -1, dtype=torch.int32, **dev)
    s["kept"][..., :kept.shape[-1]] = torch.where(kept == 1 << 30, -1, kept).to(torch.int32)
    width = -(-case["keep"] // BS)
    s["new_table"] = None
    if case["fresh_blocks"]:
        s["new_table"] = nb + torch.randperm(b * width, generator=gen, **dev).to(
            torch.int32).view(b, width)
        nb += b * width
    if case["cache"] == "bf16":
        s["row_caches"] = [_normal(gen, nb, BS, hk, D), _normal(gen, nb, BS, hk, D)]
        s["head_caches"] = []
    else:
        s["row_caches"] = []
        (k, ks), (v, vs) = _fp4_cache(gen, nb, hk), _fp4_cache(gen, nb, hk)
        s["head_caches"] = [k, v, ks, vs]
        # Where the kept rows end up, to read them back for the sequences' next prefill chunk.
        to = (s["table"] if s["new_table"] is None else s["new_table"]).long()
        place = torch.arange(case["keep"], **dev)
        at = (to.repeat_interleave(BS, 1) * BS + torch.arange(to.shape[1] * BS, **dev) % BS)
        live = place < n[:, 0]
        at = torch.nn.functional.pad(at, (0, max(0, case["keep"] - at.shape[1])))
        s["slots"] = at[:, :case["keep"]][live].to(torch.int32)
        s["k_out"], s["v_out"] = (torch.empty((len(s["slots"]), hk, D), dtype=torch.bfloat16, **dev)
                                  for _ in range(2))
    s["head_caches"].append(torch.rand((nb, hk, BS), generator=gen, **dev))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_cache_77_gb300 import api

    op = s["op"]
    if op in ("write", "read"):
        caches = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if op == "write":
            api.kv_cache_write_fp4(*caches, s["k"], s["v"], s["slots"])
        return api.kv_cache_read_fp4(*caches, s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    if op == "decode":
        if "workspace" not in s:  # kept for the process, as a server keeps it
            b, ql, h, _ = s["q"].shape
            s["workspace"] = torch.empty(
                api.decode_spec_workspace_size(b, ql, h, s["case"]["kv_heads"], D),
                dtype=torch.uint8, device="cuda")
        api.paged_attention_decode_fp4(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                       s["v_scale"], s["table"], s["seq_lens"], D ** -0.5,
                                       out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    if op == "weights":
        api.accumulate_attention_weights(s["weights"], s["q"], s["lse"], s["k_cache"], s["table"],
                                         s["seq_lens"], s["num_fresh"], D ** -0.5,
                                         k_scale=s["k_scale"])
        return s["weights"]
    if op == "select":
        c = s["case"]
        return api.select_rows(s["weights"], s["table"], s["seq_lens"], c["keep"],
                               num_sink=c["sink"], num_recent=c["recent"], out=s["out"])
    api.compact_rows(s["kept"], s["table"], row_caches=s["row_caches"],
                     head_caches=s["head_caches"], new_block_table=s["new_table"])
    if s["row_caches"]:
        return s["row_caches"] + s["head_caches"]
    k, v, ks, vs, weights = s["head_caches"]
    return [*api.kv_cache_read_fp4(k, v, ks, vs, s["slots"], k_out=s["k_out"], v_out=s["v_out"]),
            weights]


def _key_rows(s, name="k"):
    """Keys (values) of every position of the batch, fp32 [B, Hkv, n, D]."""
    block = s["table"].long()
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        return cache[block].permute(0, 3, 1, 2, 4).flatten(2, 3).float()
    if scale.dtype == torch.float32:
        x = cache[block].view(E4M3).permute(0, 3, 1, 2, 4).flatten(2, 3).float()
        return x * scale[block].transpose(1, 2).flatten(2)[..., None]
    x = _fp4_values(cache[block], scale[block], s["pairs"])  # [B, blocks, Hkv, BS, D]
    return x.transpose(1, 2).flatten(2, 3)


def _scores(s):
    """Scaled scores fp32 [B, Hkv, q_len * group, n], -inf where a row does not look."""
    b, ql, h, _ = s["q"].shape
    hk = s["case"]["kv_heads"]
    q = s["q"].float().view(b, ql, hk, h // hk, D).transpose(1, 2).flatten(2, 3)
    score = (q @ _key_rows(s).transpose(-1, -2)) * D ** -0.5
    row_len = s["seq_lens"][:, None] - ql + 1 + torch.arange(ql, device="cuda")  # [B, ql]
    seen = torch.arange(score.shape[-1], device="cuda") < row_len[..., None]
    seen = seen[:, None].repeat_interleave(h // hk, 2)
    return torch.where(seen, score, -torch.inf)


def _row_heads(x, ql):
    """[B, q_len, H, ...] of [B, Hkv, q_len * group, ...]."""
    return x.unflatten(2, (ql, -1)).transpose(1, 2).flatten(2, 3)


def _lse(s):
    score = _scores(s)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    lse = top.squeeze(-1) + torch.exp(score - top).sum(-1).log()
    return _row_heads(lse, s["q"].shape[1]).contiguous()


def _run_plain(s):
    op, case = s["op"], s["case"]
    hk = case["kv_heads"]
    if op in ("write", "read"):
        slots = s["slots"].long()
        block, off = (slots // BS)[:, None], (slots % BS)[:, None]
        head = torch.arange(hk, device="cuda")
        out = []
        for n in ("k", "v"):
            cache, scale = s[n + "_cache"], s[n + "_scale"]
            if op == "write":
                cache[block, head, off], scale[block, head, off] = _fp4_quantise(s[n])
            out.append(s[n + "_out"].copy_(_fp4_values(cache[block, head, off],
                                                       scale[block, head, off], s["pairs"])))
        return tuple(out)
    if op == "decode":
        score = _scores(s)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        o = (p @ _key_rows(s, "v")) / torch.where(total > 0, total, 1.0)
        ql = case["q_len"]
        s["out"].copy_(_row_heads(o, ql))
        s["lse"].copy_(_row_heads((top + total.log()).squeeze(-1), ql))
        return s["out"], s["lse"]
    n = s["seq_lens"].long()[:, None, None]
    block = s["table"].long()
    if op == "weights":
        b, ql, h, _ = s["q"].shape
        lse = s["lse"].view(b, ql, hk, h // hk).transpose(1, 2).flatten(2)
        score = _scores(s)
        p = torch.where(score == -torch.inf, 0.0, torch.exp(score - lse[..., None])).sum(2)
        j = torch.arange(p.shape[-1], device="cuda")
        old = s["weights"][block].transpose(1, 2).flatten(2)  # [B, Hkv, n]
        new = torch.where(j < n - s["num_fresh"].long()[:, None, None], old, 0.0) + p
        new = torch.where(j < n, new, old)
        # Rows behind a sequence's last block land in the unused block 0, whose rows stay.
        s["weights"][block] = torch.where((block > 0)[..., None, None],
                                          new.unflatten(2, (-1, BS)).transpose(1, 2),
                                          s["weights"][block])
        return s["weights"]
    if op == "select":
        key = s["weights"][block].transpose(1, 2).flatten(2)
        j = torch.arange(key.shape[-1], device="cuda")
        key = torch.where((j < case["sink"]) | (j >= n - case["recent"]), torch.inf, key)
        key = torch.where(j < n, key, -torch.inf)
        idx = key.sort(dim=-1, descending=True, stable=True).indices[..., :case["keep"]]
        idx = torch.where(idx < n, idx, 1 << 30).sort(-1).values
        s["out"].fill_(-1)
        s["out"][..., :idx.shape[-1]] = torch.where(idx == 1 << 30, -1, idx).to(torch.int32)
        return s["out"]
    kept = s["kept"].long()
    live = (kept >= 0).nonzero(as_tuple=True)  # (sequence, kv head, place)
    src, to = kept[live], s["table"] if s["new_table"] is None else s["new_table"]
    at = block[live[0], src // BS], src % BS
    put = to.long()[live[0], live[2] // BS], live[2] % BS
    for c in s["row_caches"]:
        c[put[0], put[1], live[1]] = c[at[0], at[1], live[1]]
    for c in s["head_caches"]:
        c[put[0], live[1], put[1]] = c[at[0], live[1], at[1]]
    if s["row_caches"]:
        return s["row_caches"] + s["head_caches"]
    k, v, ks, vs, weights = s["head_caches"]
    slots = s["slots"].long()
    pick = (slots // BS)[:, None], torch.arange(hk, device="cuda"), (slots % BS)[:, None]
    s["k_out"].copy_(_fp4_values(k[pick], ks[pick], s["pairs"]))
    s["v_out"].copy_(_fp4_values(v[pick], vs[pick], s["pairs"]))
    return [s["k_out"], s["v_out"], weights]


# ------------------------------------------------------------------ 64-bit results
def _value64(codes, scales):
    """64-bit values of 4-bit rows, from the bits of codes and scales."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    sign = torch.where(nib >= 8, -1.0, 1.0)
    mag = nib % 8
    exp, frac = torch.floor(mag / 2), mag % 2
    val = torch.where(exp > 0, (1 + frac / 2) * torch.exp2(exp - 1), frac / 2)
    u = scales.double()
    exp, frac = torch.floor(u / 8), u % 8
    scale = torch.where(exp > 0, (1 + frac / 8) * torch.exp2(exp - 15), frac * 2.0 ** -17)
    return sign * val * scale.repeat_interleave(GROUP, -1)


def _rounded64(x):
    """Rows as their 4-bit values, in 64 bits: for every group the scale nearest to a sixth of
    its largest magnitude, for every value the nearest of the eight multiples."""
    g = x.double().unflatten(-1, (-1, GROUP))
    scales = torch.tensor([(8 + f) / 8 * 2.0 ** (e - 15) if e else f * 2.0 ** -17
                           for e in range(29) for f in range(8) if e < 28 or f < 3],
                          dtype=torch.float64, device=x.device)
    want = g.abs().amax(-1) / 6
    hi = torch.searchsorted(scales, want).clamp(max=len(scales) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = scales[hi] - want, want - scales[lo]
    scale = scales[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device) * scale[..., None]
    pick = grid[..., 0][..., None].expand_as(g)
    for i in range(1, 8):
        a, b = grid[..., i - 1][..., None], grid[..., i][..., None]
        past = g.abs() * 2 - (a + b)
        pick = torch.where((past > 0) | ((past == 0) & (i % 2 == 0)), b, pick)
    return (pick * torch.sign(g)).flatten(-2)


def _keys64(s, i, end, name="k"):
    """[Hkv, end, D] of sequence i in 64 bits."""
    block = s["table"][i, :-(-end // BS)].long()
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        x = cache[block].double().permute(2, 0, 1, 3)
    elif scale.dtype == torch.float32:
        x = (cache[block].view(E4M3).double().permute(2, 0, 1, 3)
             * scale[block].double().transpose(0, 1)[..., None])
    else:
        x = _value64(cache[block], scale[block]).transpose(0, 1)
    return x.flatten(1, 2)[:, :end]


def exact(case, seed):
    s = prepare(case, seed)
    op, hk = case["op"], case["kv_heads"]
    if op == "write":
        return _rounded64(s["k"]), _rounded64(s["v"])
    if op == "read":
        block, off = s["slots"].long() // BS, s["slots"].long() % BS
        return tuple(_value64(s[n + "_cache"].transpose(1, 2)[block, off],
                              s[n + "_scale"].transpose(1, 2)[block, off]) for n in ("k", "v"))
    if op == "select":
        return None  # whole numbers
    if op == "compact":
        out = []
        to = s["table"] if s["new_table"] is None else s["new_table"]
        count = np.minimum(s["lens"], case["keep"])
        for c in s["row_caches"] + s["head_caches"]:
            by_head = c.transpose(1, 2) if any(c is x for x in s["row_caches"]) else c
            after = by_head.clone()
            for b in range(case["batch"]):
                n, blocks = int(count[b]), s["table"][b].long()
                rows = s["kept"][b, :, :n].long()  # [Hkv, n]
                head = torch.arange(hk, device="cuda")[:, None]
                i = torch.arange(n, device="cuda")
                after[to[b].long()[i // BS], head, i % BS] = by_head[blocks[rows // BS], head,
                                                                     rows % BS]
            out.append(after.transpose(1, 2) if by_head is not c else after)
        if s["row_caches"]:
            return [x.double() for x in out]
        k, v, ks, vs, weights = out
        both = [torch.cat([_value64(codes[to[b].long()], scales[to[b].long()]).transpose(1, 2)
                           .flatten(0, 1)[:int(count[b])] for b in range(case["batch"])])
                for codes, scales in ((k, ks), (v, vs))]
        return both + [weights.double()]
    b, ql, h, _ = s["q"].shape
    if op == "weights":
        out = s["weights"].double()
    else:
        out = torch.zeros((b, ql, h, D), dtype=torch.float64, device="cuda")
        lse = torch.full((b, ql, h), -torch.inf, dtype=torch.float64, device="cuda")
    for i in range(b):
        end = int(s["lens"][i])
        keys = _keys64(s, i, end)
        vals = _keys64(s, i, end, "v") if op == "decode" else None
        added = torch.zeros((hk, end), dtype=torch.float64, device="cuda")
        for r in range(ql):
            n = end - ql + 1 + r
            if n <= 0:
                continue
            q = s["q"][i, r].double().view(hk, h // hk, D)
            score = torch.einsum("gnd,gtd->gnt", q, keys[:, :n]) / D ** 0.5
            if op == "weights":
                norm = s["lse"][i, r].double().view(hk, -1, 1)
                added[:, :n] += torch.exp(score - norm).sum(1)
                continue
            lse[i, r] = torch.logsumexp(score, -1).flatten()
            weight = torch.exp(score - lse[i, r].view(hk, -1, 1))
            out[i, r] = torch.einsum("gnt,gtd->gnd", weight, vals[:, :n]).reshape(h, D)
        if op == "weights":
            fresh = end - int(s["num_fresh"][i])
            for j in range(-(-end // BS)):
                blk, lo, hi = int(s["table"][i, j]), j * BS, min(end, (j + 1) * BS)
                old = out[blk, :, :hi - lo].clone()
                old[:, max(0, fresh - lo):] = 0.0
                out[blk, :, :hi - lo] = old + added[:, lo:hi]
    return out if op == "weights" else (out, lse)
