"""Oracle for block-sparse decode: key summaries per block, the selection of blocks by their
score, and decode attention over listed blocks.

TEST INFRASTRUCTURE. Only tests/, ``__graft_entry__.smoke()`` and bench.py's
cpu_baseline / reference leg may import this module; the product library never
does. float64 numpy and exact sums, written from the definitions:

* Summary of a block, per kv head and channel: the smallest and the largest key of its rows.
* Score of block j for a query row and kv head: sum_d (P_d max_jd + N_d min_jd) with
  P_d = sum_h max(q_hd, 0) and N_d = sum_h min(q_hd, 0) over the kv head's query heads. It
  bounds sum_h q_h . k for every key k of the block.
* Row i of q_len sits at position len - q_len + i (the pages' bottom-right alignment for
  multi-token steps) and sees the blocks up to its own position's.
"""
from __future__ import annotations

import math

import numpy as np

from .paged_ref import bf16_bits_to_f64, softmax_combine


def update_summaries(summaries, k_cache, block_table, seq_lens, num_new, block_size):
    """Summaries [nb, Hkv, 2, d] float64 after the newest num_new[b] rows of each sequence."""
    out = np.array(summaries, dtype=np.float64)
    for b, n in enumerate(seq_lens):
        for pos in range(int(n) - int(num_new[b]), int(n)):
            blk, off = int(block_table[b][pos // block_size]), pos % block_size
            row = k_cache[blk, off]
            row = bf16_bits_to_f64(row) if row.dtype == np.uint16 else row
            if off == 0:
                out[blk, :, 0], out[blk, :, 1] = row, row
            else:
                out[blk, :, 0] = np.minimum(out[blk, :, 0], row)  # numpy's propagate NaN
                out[blk, :, 1] = np.maximum(out[blk, :, 1], row)
    return out


def block_score(q_heads, low, high) -> float:
    """Score of one block, the sum rounded once (q_heads [n_rep, d]; low, high [d])."""
    P = [math.fsum(max(x, 0.0) for x in q_heads[:, d]) for d in range(q_heads.shape[1])]
    N = [math.fsum(min(x, 0.0) for x in q_heads[:, d]) for d in range(q_heads.shape[1])]
    terms = [p * h for p, h in zip(P, high)] + [n * lo for n, lo in zip(N, low)]
    if not np.isfinite(terms).all():
        return float(np.sum(terms))
    return math.fsum(terms)


def row_blocks(length: int, q_len: int, i: int, block_size: int) -> int:
    """Blocks that row i of q_len of a sequence sees."""
    return -(-max(length - q_len + 1 + i, 0) // block_size)


def select_blocks(q, summaries, block_table, seq_lens, num_selected, num_sink, num_recent,
                  block_size):
    """[B, Q, Hkv, num_selected] blocks of each sequence, ascending, -1 behind the last.

    q [B, Q, H, d], summaries [nb, Hkv, 2, d] float64. Table entries outside the cache score
    below everything; NaN scores above everything; ties go to the lower block."""
    B, Q, H, _ = q.shape
    nb, hkv = summaries.shape[:2]
    n_rep = H // hkv
    out = np.full((B, Q, hkv, num_selected), -1, dtype=np.int32)
    for b in range(B):
        for i in range(Q):
            n = row_blocks(int(seq_lens[b]), Q, i, block_size)
            for g in range(hkv):
                if n <= num_selected:
                    out[b, i, g, :n] = np.arange(n)
                    continue
                always = set(range(num_sink)) | set(range(n - num_recent, n))
                rank = []
                for j in range(n):
                    blk = int(block_table[b][j])
                    if j in always:
                        continue
                    if blk < 0 or blk >= nb:
                        rank.append((2, 0.0, j))
                        continue
                    s = block_score(q[b, i, g * n_rep:(g + 1) * n_rep], *summaries[blk, g])
                    rank.append((0, 0.0, j) if np.isnan(s) else (1, -s, j))
                rank.sort()
                taken = sorted(always | {j for _, _, j in rank[:num_selected - len(always)]})
                out[b, i, g] = taken
    return out


def sparse_decode(q, k_cache, v_cache, block_table, seq_lens, block_indices, block_size, scale):
    """Attention of row (b, i) and head h over the positions up to the row's own in the blocks
    block_indices[b, i, h // n_rep].

    q [B, Q, H, d]; caches bf16 bits or float64. Returns o, lse and, for error bounds, the
    spread sum_j p_j |v_j - o| of every output."""
    B, Q, H, d = q.shape
    hkv = k_cache.shape[2]
    n_rep = H // hkv
    o = np.zeros((B, Q, H, d))
    lse = np.full((B, Q, H), -np.inf)
    spread = np.zeros((B, Q, H, d))
    widen = (lambda x: bf16_bits_to_f64(x)) if k_cache.dtype == np.uint16 else \
        (lambda x: np.asarray(x, dtype=np.float64))
    for b in range(B):
        for i in range(Q):
            end = int(seq_lens[b]) - Q + 1 + i
            n = row_blocks(int(seq_lens[b]), Q, i, block_size)
            for g in range(hkv):
                K, V = [], []
                for j in block_indices[b, i, g][:n]:
                    if j < 0 or j >= n:
                        continue
                    blk, rows = int(block_table[b][j]), min(block_size, end - int(j) * block_size)
                    K.append(widen(k_cache[blk, :rows, g]))
                    V.append(widen(v_cache[blk, :rows, g]))
                if not K:
                    continue
                K, V = np.concatenate(K), np.concatenate(V)
                seen = np.ones(len(K), dtype=bool)
                for h in range(g * n_rep, (g + 1) * n_rep):
                    o[b, i, h], lse[b, i, h], p = softmax_combine(scale * (K @ q[b, i, h]), V, seen)
                    spread[b, i, h] = p @ np.abs(V - o[b, i, h])
    return o, lse, spread
