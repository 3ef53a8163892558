"""Oracle for eviction by accumulated attention weight: the sums, the choice of rows, the move.

TEST INFRASTRUCTURE. Only tests/ and ``__graft_entry__.smoke()`` may import this module; the
product library never does. numpy, float64, written from the definitions:

* a step adds to each position's sum, per kv head, the softmax weights that the step's query
  rows give it, summed over the query heads of the kv head and the rows that see it;
* of a sequence longer than num_keep the positions with the largest sums stay, sinks and the
  newest always, equal sums lowest position first, NaN above all;
* row i of what stays becomes what row kept[i] was, per kv head.
"""
from __future__ import annotations

import numpy as np


def accumulate(weights, q, lse, keys, block_table, seq_lens, num_fresh, scale, decay=1.0):
    """The sums [nb, H_kv, bs] after one step, and the sums of the added terms' magnitudes
    sum |q||k| (for error bounds), laid out the same. keys [nb, bs, H_kv, d] float64."""
    out = np.array(weights, dtype=np.float64)
    nb, hkv, bs = out.shape
    reach = np.zeros_like(out)
    B, Q, H, _ = q.shape
    n_rep = H // hkv
    for b in range(B):
        n = min(int(seq_lens[b]), block_table.shape[1] * bs)
        fresh = n - min(max(int(num_fresh[b]), 0), n)
        for p in range(n):
            blk, off = int(block_table[b][p // bs]), p % bs
            if blk < 0 or blk >= nb:
                continue
            for g in range(hkv):
                k = keys[blk, off, g]
                first = max(0, p - (n - Q))  # the first row that sees p
                rows = q[b, first:, g * n_rep:(g + 1) * n_rep]
                z = scale * (rows @ k) - lse[b, first:, g * n_rep:(g + 1) * n_rep]
                old = 0.0 if p >= fresh else decay * out[blk, g, off]
                out[blk, g, off] = old + np.exp(z).sum()
                reach[blk, g, off] = scale * (np.abs(rows) @ np.abs(k)).max(initial=0.0)
    return out, reach


def select_rows(weights, block_table, seq_lens, num_keep, num_sink=0, num_recent=0):
    """int32 [B, H_kv, num_keep]: kept positions, ascending, -1 behind the last."""
    nb, hkv, bs = weights.shape
    out = np.full((len(seq_lens), hkv, num_keep), -1, dtype=np.int32)
    for b, n in enumerate(seq_lens):
        n = min(max(int(n), 0), block_table.shape[1] * bs)
        for g in range(hkv):
            if n <= num_keep:
                out[b, g, :n] = np.arange(n)
                continue
            always = set(range(num_sink)) | set(range(n - num_recent, n))
            rank = []
            for p in range(n):
                if p in always:
                    continue
                blk = int(block_table[b][p // bs])
                if blk < 0 or blk >= nb:
                    rank.append((2, 0.0, p))
                    continue
                w = float(weights[blk, g, p % bs])
                rank.append((0, 0.0, p) if np.isnan(w) else (1, -w, p))
            rank.sort()
            out[b, g] = sorted(always | {p for _, _, p in rank[:num_keep - len(always)]})
    return out


def compact(cache, kept, block_table, new_table, head_major):
    """A copy of one cache with the kept rows moved (bad entries are left out)."""
    rows = cache if head_major else np.swapaxes(cache, 1, 2)  # [nb, H_kv, bs, ...]
    out = rows.copy()
    nb, _, bs = rows.shape[:3]
    for b in range(kept.shape[0]):
        for g in range(kept.shape[1]):
            for i, p in enumerate(kept[b, g]):
                if p < 0 or p // bs >= block_table.shape[1] or i // bs >= new_table.shape[1]:
                    continue
                src, dst = int(block_table[b][p // bs]), int(new_table[b][i // bs])
                if 0 <= src < nb and 0 <= dst < nb:
                    out[dst, g, i % bs] = rows[src, g, p % bs]
    return out if head_major else np.swapaxes(out, 1, 2)
