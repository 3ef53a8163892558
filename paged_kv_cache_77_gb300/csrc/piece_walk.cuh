// Runs of pieces of 32 tokens, one for every warp of a CTA, out of the CTA's share of the blocks that a
// decode call reads; and where a warp's lanes find a piece's tokens.
#pragma once

#include "row_cursor.cuh"

namespace pkv {

constexpr int TILE = 128, SUB = 32;  // tokens of a block, and of a piece of it

// Rows 2c and 2c + 1 of a product's 8 rows are tokens 0 3, 1 2, 4 7, 5 6 (and 8 further on): K's
// 16-byte loads, 8 lanes at a time, then meet two rows of different banks, V's 8-byte loads rows
// that share them by twos only.
__device__ __forceinline__ int even_row(int c) { return (c & 1) | (c & 2) << 1; }
__device__ __forceinline__ int token_of(int r) { return even_row(r >> 1) ^ ((r & 1) ? 3 : 0); }

// A warp's walk over its run, segment by segment (a segment is the blocks that the rows of one
// sequence and kv head see). The run is counted in pieces of 32 tokens of whole blocks; of the last
// block only the pieces that hold tokens are visited.
struct Walk {
  int b, g, len;
  int pos, stop;   // next position, and where the run leaves the segment or the tokens end
  int todo;        // pieces of the run from this segment's first visit on
  int padded;      // of them in this segment
  bool ends;       // whether the segment's last token is in the run
  __device__ __forceinline__ void enter(int at) {
    const int end = (len + TILE - 1) & ~(TILE - 1);
    pos = at;
    padded = min((end - at) / SUB, todo);
    ends = padded * SUB == end - at;
    stop = min(at + padded * SUB, (len + SUB - 1) & ~(SUB - 1));
  }
  // The first of the pieces of warp w of `warps`, in a CTA's share of `tiles` blocks.
  static __device__ __forceinline__ int64_t run(int64_t tiles, int w, int warps) {
    return tiles * (TILE / SUB) * w / warps;
  }
  // Enters the run of pieces [u0, u1) of the CTA's share [t0, t1) (all lanes of a warp); whether it
  // begins with a segment's first piece.
  __device__ __forceinline__ bool seek(const DenseRows& rows, int B, int Hkv, int64_t t0, int64_t t1, int64_t u0,
                                       int64_t u1) {
    constexpr int PER = TILE / SUB;
    TileCursor t;
    cursor_seek_warp(t, rows, B, Hkv, t0 + u0 / PER, t1);
    b = t.b;
    g = t.g;
    len = t.len;
    todo = (int)(u1 - u0);
    enter((t.jlo + t.j) * TILE + (int)(u0 % PER) * SUB);
    return t.j == 0 && u0 % PER == 0;
  }
  // Enters pieces [u0, u1) of one segment, of kv head kv of sequence seq (len > 0), whose first block is jlo.
  __device__ __forceinline__ void start(int seq, int kv, int length, int jlo, int u0, int u1) {
    b = seq;
    g = kv;
    len = length;
    todo = u1 - u0;
    enter(jlo * TILE + u0 * SUB);
  }
  // The next segment of the run; false behind its end.
  __device__ __forceinline__ bool next(const DenseRows& rows, int B, int Hkv) {
    todo -= padded;
    if (todo <= 0) return false;
    if (++g == Hkv) {
      g = 0;
      do {
        if (++b >= B) return false;
        len = rows.len(b);
      } while (len == 0);
    }
    enter(rows.blocks(len).jlo * TILE);
    return true;
  }
};

}  // namespace pkv
