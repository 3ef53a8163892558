// The tile list of the decode kernels over any kind of rows: the balanced split of
// device_common.cuh, whose functions walk the sequences of a dense call, with what a row
// reads given by a policy.
#pragma once

#include "device_common.cuh"

namespace pkv {

// The rows whose tiles a decode call walks. Dense attention: one per sequence, reading its
// live blocks in order. Sparse attention: one per query row, reading at most `keep` blocks
// of the row's own list; row r is query r % q_len of sequence r / q_len and sees the first
// len - q_len + 1 + r % q_len positions of it.
struct DenseRows {
  const int* seq_lens;
  int bs, window, cap;
  __device__ __forceinline__ int raw(int b) const { return __ldg(seq_lens + b); }
  __device__ __forceinline__ int len(int b) const { return clamp_len(raw(b), cap); }
  __device__ __forceinline__ SeqRange blocks(int len) const { return live_blocks(len, bs, window); }
};
struct SparseRows {
  const int* seq_lens;
  int bs, q_len, keep, cap;
  __device__ __forceinline__ int raw(int r) const { return __ldg(seq_lens + r / q_len); }
  __device__ __forceinline__ int len(int r) const {
    const int n = clamp_len(raw(r), cap) - q_len + 1 + r % q_len;
    return n > 0 ? n : 0;
  }
  __device__ __forceinline__ SeqRange blocks(int len) const {
    SeqRange s;
    s.jlo = 0;
    s.n = (len + bs - 1) / bs;
    if (s.n > keep) s.n = keep;
    return s;
  }
};

// Sum of live blocks over all rows (one warp, result in every lane).
template <typename Rows>
__device__ __forceinline__ int64_t total_live_blocks(const Rows& rows, int B, int* dev_status) {
  int64_t s = 0;
  for (int b = threadIdx.x & 31; b < B; b += 32) {
    const int raw = rows.raw(b);
    if (clamp_len(raw, rows.cap) != raw && blockIdx.x == 0) flag_status(dev_status, PKV_DEV_BAD_LENGTH);
    s += rows.blocks(rows.len(b)).n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Position the cursor at global tile t (a single thread's scan).
template <typename Rows>
__device__ inline void cursor_seek(TileCursor& c, const Rows& rows, int B, int Hkv, int64_t t,
                                   int64_t t_end) {
  c = TileCursor{B, 0, 0, 0, 0, 0, 0, t, t_end};
  if (t >= t_end) return;
  int64_t base = 0;
  for (int b = 0; b < B; ++b) {
    const int len = rows.len(b);
    const SeqRange r = rows.blocks(len);
    const int64_t seg = (int64_t)r.n * Hkv;
    if (t < base + seg) {
      const int64_t off = t - base;
      c.b = b;
      c.g = (int)(off / r.n);
      c.j = (int)(off % r.n);
      c.jlo = r.jlo;
      c.n = r.n;
      c.len = len;
      c.seg_base = base + (int64_t)c.g * r.n;
      return;
    }
    base += seg;
  }
}

// The same by a whole warp, 32 rows at a time: for calls whose rows are many (query rows).
// Every lane gets the cursor.
template <typename Rows>
__device__ inline void cursor_seek_warp(TileCursor& c, const Rows& rows, int B, int Hkv, int64_t t,
                                        int64_t t_end) {
  c = TileCursor{B, 0, 0, 0, 0, 0, 0, t, t_end};
  if (t >= t_end) return;
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int len = b0 + lane < B ? rows.len(b0 + lane) : 0;
    const SeqRange r = rows.blocks(len);
    const int64_t seg = (int64_t)r.n * Hkv;
    int64_t incl = seg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, t < base + incl);
    if (past) {
      const int owner = __ffs((int)past) - 1;
      const int64_t start = base + __shfl_sync(0xffffffffu, incl - seg, owner), off = t - start;
      c.b = b0 + owner;
      c.jlo = __shfl_sync(0xffffffffu, r.jlo, owner);
      c.n = __shfl_sync(0xffffffffu, r.n, owner);
      c.len = __shfl_sync(0xffffffffu, len, owner);
      c.g = (int)(off / c.n);
      c.j = (int)(off % c.n);
      c.seg_base = start + (int64_t)c.g * c.n;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Advance to the next tile; returns false when the CTA's range is exhausted.
template <typename Rows>
__device__ inline bool cursor_next(TileCursor& c, const Rows& rows, int B, int Hkv) {
  ++c.t;
  if (c.t >= c.t_end) return false;
  if (++c.j < c.n) return true;
  c.j = 0;
  c.seg_base += c.n;
  if (++c.g < Hkv) return true;
  c.g = 0;
  for (;;) {
    if (++c.b >= B) return false;
    c.len = rows.len(c.b);
    const SeqRange r = rows.blocks(c.len);
    c.jlo = r.jlo;
    c.n = r.n;
    if (r.n > 0) return true;
  }
}

}  // namespace pkv
