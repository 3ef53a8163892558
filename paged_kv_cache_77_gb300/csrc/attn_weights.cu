// accumulate_attention_weights: the attention that a step's query rows pay to every cached row
// of their sequence, summed over the query heads of its kv head and added to the row's running
// sum. With the log-sum-exp that the step's attention returned, a weight is
// exp(scale q . k - lse): one pass over the keys, no second pass for a normaliser, no values.
//
// The keys may be bf16, FP8 (E4M3 with a scale per row) or 4-bit (fp4.cuh). bf16 enters the
// product as it is; the others are exact in fp16, with q scaled by a power of two per row.
// Scores, exponentials and sums are fp32. A warp owns a token: no atomics, the sum's order is
// fixed. Two kernels, by what bounds them:
//   - bf16 keys, or more than 16 query rows per kv head: a CTA walks its share of the (sequence, kv
//     head, block) tiles; each of its 8 warps takes 16 tokens of a tile straight from global memory
//     into the registers of the A operand (the next tile's while it works on this one), 8 query rows
//     at a time are the columns of B, from shared memory. bf16 keys of one decode step run at the
//     memory's rate (64 sequences of up to 32,768 tokens, 64 / 8 heads: 324 to 332 us, 95 to 98 % of the
//     copy rate). Those of an observation window are bound by latency: 4 x 8,192 tokens, 32 rows of 8
//     heads, two launches of 128 rows each, 69 us where the keys' bytes take 10; 16 warps an SM wait for
//     their products, for B operands (shared memory 59 % busy) and for exponentials in turn (tensor pipe
//     34 %, issue slots 34 %, exponential unit 9 %);
//   - FP8 and 4-bit keys with up to 16 rows, which are bound by instructions: every warp has a run
//     of its own, in pieces of 32 tokens through a ring in shared memory, the queries in registers
//     (the same batch over FP8 keys 239 us with the first kernel and 187 to 206 with this one, 82 to 89 %
//     of the copy rate; over 4-bit keys 253 and 108 us, 89 %).
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "mma_f16.cuh"
#include "pdl.cuh"
#include "piece_walk.cuh"
#include "query_f16.cuh"
#include "row_cursor.cuh"

namespace pkv {
namespace {

constexpr int BS = 128, D = 128, WARPS = 8;

// How a lane's share of a 16-token tile lies in its cache. Lane 4 i + c holds tokens i and i + 8:
// 16-byte chunk x of the row's channels first(c, x) .. + 7 (as the query operand holds them).
template <int FMT>
struct Keys;
template <>
struct Keys<kKeysBf16> {
  static constexpr int LOADS = 4;  // 16-byte loads of a token
  static constexpr int ROW = 256;  // bytes of a row
  static __device__ __forceinline__ int at(int c, int x) { return 16 * (c + 4 * x); }
  static __device__ __forceinline__ int first(int c, int x) { return 8 * (c + 4 * x); }
};
template <>
struct Keys<kKeysFp8> {
  static constexpr int LOADS = 2;
  static constexpr int ROW = 128;
  static __device__ __forceinline__ int at(int c, int x) { return 16 * (c + 4 * x); }
  static __device__ __forceinline__ int first(int c, int x) { return 16 * (c + 4 * (x >> 1)) + 8 * (x & 1); }
};
template <>
struct Keys<kKeysFp4> {
  static constexpr int LOADS = 1;
  static constexpr int ROW = fp4::kCodeBytes;
  static __device__ __forceinline__ int at(int c, int x) { return 16 * c; }
  static __device__ __forceinline__ int first(int c, int x) { return 32 * c + 8 * x; }
};

// One tile's data of a lane, as it comes from memory.
template <int FMT>
struct Fetched {
  uint4 k[2][Keys<FMT>::LOADS];
  uint32_t scale[2];  // FP8: the row's fp32 scale; 4-bit: scale bytes 2c and 2c + 1
  float old;          // the running sum of the token that this lane writes
};

__device__ __forceinline__ void widen_e4m3(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

template <int FMT>
__global__ void __launch_bounds__(32 * WARPS, 2)
    attn_weights_kernel(const __grid_constant__ WeightsArgs a) {
  using K = Keys<FMT>;
  __shared__ uint4 sq[kWeightsMaxRows / 8][4][32];           // B operands
  __shared__ float sf[kWeightsMaxRows], sl[kWeightsMaxRows];  // score factor, lse (both for log2)
  __shared__ int si[kWeightsMaxRows];                         // last position that a row sees
  __shared__ int64_t total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const DenseRows rows = {a.seq_lens, BS, 0, a.max_blocks * BS};
  pdl_wait_then_launch();
  if (warp == 0) {
    const int64_t tot = total_live_blocks(rows, a.B, a.dev_status);
    if (lane == 0) total = tot * a.Hkv;
  }
  __syncthreads();
  const int64_t T = total, G = gridDim.x;
  const int64_t t0 = cta_tile_start(blockIdx.x, T, G), t1 = cta_tile_start(blockIdx.x + 1, T, G);
  if (t0 >= t1) return;
  const int R = a.rows * a.n_rep, tiles = (R + 7) / 8;

  TileCursor cur, nxt;
  cursor_seek_warp(cur, rows, a.B, a.Hkv, t0, t1);
  nxt = cur;
  bool more = true;
  auto block_of = [&](const TileCursor& t) {
    return __ldg(a.block_table + (int64_t)t.b * a.max_blocks + t.j);
  };
  // Loads of this warp's tokens of tile `t` in block `blk`; tokens behind the sequence's end are
  // left out (the caches may hold anything there, and the block's rows are all in bounds).
  auto fetch = [&](const TileCursor& t, int blk, Fetched<FMT>& f) {
    if (blk < 0 || (int64_t)blk >= a.num_blocks) return;
    const int p0 = t.j * BS + warp * 16;
    if (p0 >= t.len) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = warp * 16 + g + 8 * h;
      const int64_t hrow = ((int64_t)blk * a.Hkv + t.g) * BS + tok;  // head-major
      const int64_t trow = ((int64_t)blk * BS + tok) * a.Hkv + t.g;  // token-major
      const uint8_t* src = a.k_cache + (FMT == kKeysFp4 ? hrow : trow) * K::ROW;
#pragma unroll
      for (int x = 0; x < K::LOADS; ++x) f.k[h][x] = ld_nc_v4(src + K::at(c, x));
      if constexpr (FMT == kKeysFp8) f.scale[h] = __ldg(reinterpret_cast<const uint32_t*>(a.k_scale) + hrow);
      if constexpr (FMT == kKeysFp4)
        f.scale[h] = __ldg(reinterpret_cast<const uint16_t*>(a.k_scale + hrow * fp4::kScaleBytes) + c);
      if (c == h) f.old = a.weights[hrow];
    }
  };
  Fetched<FMT> now, then;
  int blk = block_of(cur), blk1 = 0;
  fetch(cur, blk, now);
  more = cursor_next(nxt, rows, a.B, a.Hkv);
  if (more) blk1 = block_of(nxt);
  int seg_b = -1, seg_g = -1, fresh = 0;
  for (;;) {
    const TileCursor ahead = nxt;
    const int blk_ahead = blk1;
    const bool go_on = more;
    if (go_on) {
      fetch(ahead, blk_ahead, then);
      more = cursor_next(nxt, rows, a.B, a.Hkv);
      if (more) blk1 = block_of(nxt);
    }
    if (cur.b != seg_b || cur.g != seg_g) {
      __syncthreads();  // nobody reads the last segment's rows any more
      seg_b = cur.b;
      seg_g = cur.g;
      const int first = cur.len - a.q_len + a.row0;  // position of the launch's first query token
      const int n = __ldg(a.num_fresh + cur.b);
      fresh = cur.len - (n < 0 ? 0 : n > cur.len ? cur.len : n);
      for (int n8 = warp; n8 < tiles; n8 += WARPS) {
        const int r = n8 * 8 + g;
        const int64_t row = ((int64_t)cur.b * a.q_len + a.row0 + r / a.n_rep) * a.H +
                            (int64_t)cur.g * a.n_rep + r % a.n_rep;
        const uint16_t* src = r < R ? a.q + row * D : nullptr;
        uint4 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = src ? __ldg(reinterpret_cast<const uint4*>(src + K::first(c, x))) : make_uint4(0, 0, 0, 0);
        float factor = a.scale_log2;
        if constexpr (FMT != kKeysBf16) factor *= query_to_f16(w);
#pragma unroll
        for (int x = 0; x < 4; ++x) sq[n8][x][lane] = w[x];
        if (c == 0) {
          sf[r] = factor;
          sl[r] = r < R ? __ldg(a.lse + row) * kLog2e : 0.f;
          si[r] = r < R ? first + r / a.n_rep : INT32_MIN;  // (a column without a row sees none)
        }
      }
      __syncthreads();
    }
    const int p0 = cur.j * BS + warp * 16;
    const bool ok = blk >= 0 && (int64_t)blk < a.num_blocks;
    if (!ok && tid == 0) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
    if (ok && p0 < cur.len) {
      uint32_t k0[16], k1[16];  // tokens g and g + 8: register 4x + h pairs with the query's chunk x
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t(&k)[16] = h ? k1 : k0;
        if constexpr (FMT == kKeysBf16) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            k[4 * x] = now.k[h][x].x;
            k[4 * x + 1] = now.k[h][x].y;
            k[4 * x + 2] = now.k[h][x].z;
            k[4 * x + 3] = now.k[h][x].w;
          }
        } else if constexpr (FMT == kKeysFp8) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            widen_e4m3(now.k[h][x].x, k[8 * x], k[8 * x + 1]);
            widen_e4m3(now.k[h][x].y, k[8 * x + 2], k[8 * x + 3]);
            widen_e4m3(now.k[h][x].z, k[8 * x + 4], k[8 * x + 5]);
            widen_e4m3(now.k[h][x].w, k[8 * x + 6], k[8 * x + 7]);
          }
        } else {
          const uint32_t w[4] = {now.k[h][0].x, now.k[h][0].y, now.k[h][0].z, now.k[h][0].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t s = x < 2 ? fp4::scale_dup0(now.scale[h]) : fp4::scale_dup1(now.scale[h]);
            uint32_t y[4];
            fp4::widen(w[x], y);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[4 * x + i] = fp4::mul2(y[i], s);
          }
        }
      }
      const int pa = p0 + g, pb = pa + 8;
      float wa = 0.f, wb = 0.f;
      for (int n = 0; n < tiles; ++n) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 b = sq[n][x][lane];
          if constexpr (FMT == kKeysBf16) {
            mma_bf16(s, k0[4 * x], k1[4 * x], k0[4 * x + 1], k1[4 * x + 1], b.x, b.y);
            mma_bf16(s, k0[4 * x + 2], k1[4 * x + 2], k0[4 * x + 3], k1[4 * x + 3], b.z, b.w);
          } else {
            mma_f16(s, k0[4 * x], k1[4 * x], k0[4 * x + 1], k1[4 * x + 1], b.x, b.y);
            mma_f16(s, k0[4 * x + 2], k1[4 * x + 2], k0[4 * x + 3], k1[4 * x + 3], b.z, b.w);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = n * 8 + 2 * c + (i & 1);
          float f = sf[r];
          if constexpr (FMT == kKeysFp8) f *= __uint_as_float(now.scale[i >> 1]);
          const float p = exp2f(fmaf(s[i], f, -sl[r]));
          const bool seen = (i < 2 ? pa : pb) <= si[r];
          if (i < 2)
            wa += seen ? p : 0.f;
          else
            wb += seen ? p : 0.f;
        }
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        wa += __shfl_xor_sync(0xffffffffu, wa, d);
        wb += __shfl_xor_sync(0xffffffffu, wb, d);
      }
      const int pos = c ? pb : pa;
      if (c < 2 && pos < cur.len) {
        const float added = c ? wb : wa;
        a.weights[((int64_t)blk * a.Hkv + cur.g) * BS + warp * 16 + g + 8 * c] =
            pos >= fresh && a.start ? added : fmaf(now.old, a.decay, added);
      }
    }
    if (!go_on) break;
    cur = ahead;
    blk = blk_ahead;
    now = then;
  }
}

// ------------------------------------------------------------------- runs: FP8 and 4-bit keys
constexpr int RUN_WARPS = 16, RUN_STAGES = 3;

// A piece in shared memory: 32 rows of codes, their scales, their running sums.
template <int FMT>
struct Piece;
template <>
struct __align__(128) Piece<kKeysFp8> {
  uint8_t codes[SUB * 128];  // 16-byte chunk i of row r at chunk i ^ 4 (r & 1): other banks for odd rows
  float scales[SUB];
  float sums[SUB];
  int64_t row;  // of the first token, head-major; -1: the block does not exist
};
template <>
struct __align__(128) Piece<kKeysFp4> {
  uint8_t codes[SUB * fp4::kCodeBytes];
  uint8_t scales[SUB * fp4::kScaleBytes];
  float sums[SUB];
  int64_t row;
};

template <int FMT, int NT>
__global__ void __launch_bounds__(32 * RUN_WARPS, 1) attn_weights_runs_kernel(const __grid_constant__ WeightsArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ int64_t total;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, and known to be)
  Piece<FMT>* ring = reinterpret_cast<Piece<FMT>*>(smem_raw) + warp * RUN_STAGES;
  const DenseRows rows = {a.seq_lens, TILE, 0, a.max_blocks * TILE};
  pdl_wait_then_launch();
  if (warp == 0) {
    const int64_t tot = total_live_blocks(rows, a.B, a.dev_status);
    if (lane == 0) total = tot * a.Hkv;
  }
  __syncthreads();
  const int64_t T = total, G = gridDim.x;
  const int64_t t0 = cta_tile_start(blockIdx.x, T, G), t1 = cta_tile_start(blockIdx.x + 1, T, G);
  const int64_t u0 = Walk::run(t1 - t0, warp, RUN_WARPS), u1 = Walk::run(t1 - t0, warp + 1, RUN_WARPS);
  if (u0 >= u1) return;
  Walk cur = {};
  cur.seek(rows, a.B, a.Hkv, t0, t1, u0, u1);
  const int R = a.rows * a.n_rep;

  // ---- the ring: one group of asynchronous copies a piece
  Walk ahead = cur;
  bool more = true;
  int ids = 0, ids_j = -64;  // 32 table entries of the sequence, from block ids_j on
  bool enter = true;         // whether the piece's block has to be looked up
  int64_t row = -1;          // of the next piece's first token, head-major (-1: its block does not exist)
  auto issue = [&](int st) {
    while (more && ahead.pos >= ahead.stop) {
      const int b = ahead.b;
      more = ahead.next(rows, a.B, a.Hkv);
      if (ahead.b != b) ids_j = -64;
      enter = true;
    }
    if (more) {
      if (enter || ahead.pos % TILE == 0) {
        enter = false;
        const int j = ahead.pos / TILE;
        if ((unsigned)(j - ids_j) >= 32u) {
          ids_j = j;
          // (Counted in blocks: the last positions lie just below 2^31.)
          ids = j + lane <= (ahead.len - 1) / TILE ? __ldg(a.block_table + (int64_t)ahead.b * a.max_blocks + j + lane) : 0;
        }
        const int blk = __shfl_sync(0xffffffffu, ids, j - ids_j);
        row = -1;
        if (blk >= 0 && (int64_t)blk < a.num_blocks)
          row = ((int64_t)blk * a.Hkv + ahead.g) * TILE + ahead.pos % TILE;
        else if (lane == 0)
          flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
      }
      Piece<FMT>& p = ring[st];
      if (lane == 0) p.row = row;
      if (row >= 0) {
        // Zeros instead of the rows behind the sequence's end.
        const int live = ahead.len - ahead.pos;
        if constexpr (FMT == kKeysFp4) {
          const uint8_t* src = a.k_cache + row * fp4::kCodeBytes + 16 * lane;
          const uint32_t dst = smem_u32(p.codes) + 16 * lane;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cp_async_16(dst + 512 * i, src + 512 * i, 8 * i + (lane >> 2) < live ? 16 : 0);
          if (lane < 16)
            cp_async_16(smem_u32(p.scales) + 16 * lane, a.k_scale + row * fp4::kScaleBytes + 16 * lane,
                        2 * lane < live ? 16 : 0);
        } else {
          // Token-major codes: row (block, token, head).
          const int64_t token = row / TILE / a.Hkv * TILE + row % TILE;
          const int r = lane >> 3, chunk = lane & 7;
          const uint8_t* src = a.k_cache + ((token + r) * a.Hkv + ahead.g) * 128 + 16 * chunk;
          const uint32_t dst = smem_u32(p.codes) + 128 * r + 16 * (chunk ^ (r & 1) * 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            cp_async_16(dst + 512 * i, src + (int64_t)512 * i * a.Hkv, 4 * i + r < live ? 16 : 0);
          if (lane < 8) cp_async_16(smem_u32(p.scales) + 16 * lane, a.k_scale + row * 4 + 16 * lane, 16);
        }
        if (lane >= 16 && lane < 24)
          cp_async_16(smem_u32(p.sums) + 16 * (lane - 16), a.weights + row + 4 * (lane - 16), 16);
        row += SUB;
      }
      ahead.pos += SUB;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < RUN_STAGES; ++st) issue(st);

  // Of a piece, lane 4 g + c writes the sum of row g + 8 (c & 1) of the (c >> 1)-th 16 tokens.
  const int mine = 16 * (c >> 1) + 8 * (c & 1) + token_of(g);
  int st = 0;
  do {
    uint4 qf[NT][4];
    float f[NT][2], minus[NT][2];  // of this lane's rows: score factor, negated lse (both for log2)
    int limit[NT][2];              // last position that they see
    const int first = cur.len - a.q_len + a.row0;
    const int n_fresh = __ldg(a.num_fresh + cur.b);
    const int fresh = cur.len - (n_fresh < 0 ? 0 : n_fresh > cur.len ? cur.len : n_fresh);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      auto query = [&](int r) {
        return ((int64_t)cur.b * a.q_len + a.row0 + r / a.n_rep) * a.H + (int64_t)cur.g * a.n_rep + r % a.n_rep;
      };
      const int r0 = 8 * n + g;
      const uint16_t* src = a.q + query(r0) * D;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        qf[n][x] = r0 < R ? __ldg(reinterpret_cast<const uint4*>(src + Keys<FMT>::first(c, x))) : make_uint4(0, 0, 0, 0);
      const float down = query_to_f16(qf[n]) * a.scale_log2;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * n + 2 * c + x;
        f[n][x] = __shfl_sync(0xffffffffu, down, 8 * c + 4 * x);
        minus[n][x] = r < R ? -__ldg(a.lse + query(r)) * kLog2e : -INFINITY;
        limit[n][x] = r < R ? first + r / a.n_rep : INT32_MIN;
      }
    }
    for (; cur.pos < cur.stop; cur.pos += SUB) {
      cp_async_wait<RUN_STAGES - 1>();
      __syncwarp();  // every lane's copies are there
      const Piece<FMT>& p = ring[st];
      const int64_t at = p.row;
      if (at >= 0) {
        const bool inside = cur.pos + SUB - 1 <= first;
        float sum[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 16 * h + token_of(g);
          uint32_t k0[16], k1[16];
          float by[2] = {1.f, 1.f};
          if constexpr (FMT == kKeysFp4) {
            const uint4 w0 = *reinterpret_cast<const uint4*>(p.codes + t * fp4::kCodeBytes + 16 * c);
            const uint4 w1 = *reinterpret_cast<const uint4*>(p.codes + (t + 8) * fp4::kCodeBytes + 16 * c);
            const uint32_t e0 = *reinterpret_cast<const uint16_t*>(p.scales + t * fp4::kScaleBytes + 2 * c);
            const uint32_t e1 = *reinterpret_cast<const uint16_t*>(p.scales + (t + 8) * fp4::kScaleBytes + 2 * c);
            const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t y0[4], y1[4];
              fp4::widen(x0[x], y0);
              fp4::widen(x1[x], y1);
              const uint32_t s0 = x < 2 ? fp4::scale_dup0(e0) : fp4::scale_dup1(e0);
              const uint32_t s1 = x < 2 ? fp4::scale_dup0(e1) : fp4::scale_dup1(e1);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                k0[4 * x + i] = fp4::mul2(y0[i], s0);
                k1[4 * x + i] = fp4::mul2(y1[i], s1);
              }
            }
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int chunk = (c + 4 * x) ^ (t & 1) * 4;
              const uint4 w0 = *reinterpret_cast<const uint4*>(p.codes + t * 128 + 16 * chunk);
              const uint4 w1 = *reinterpret_cast<const uint4*>(p.codes + (t + 8) * 128 + 16 * chunk);
              widen_e4m3(w0.x, k0[8 * x], k0[8 * x + 1]);
              widen_e4m3(w0.y, k0[8 * x + 2], k0[8 * x + 3]);
              widen_e4m3(w0.z, k0[8 * x + 4], k0[8 * x + 5]);
              widen_e4m3(w0.w, k0[8 * x + 6], k0[8 * x + 7]);
              widen_e4m3(w1.x, k1[8 * x], k1[8 * x + 1]);
              widen_e4m3(w1.y, k1[8 * x + 2], k1[8 * x + 3]);
              widen_e4m3(w1.z, k1[8 * x + 4], k1[8 * x + 5]);
              widen_e4m3(w1.w, k1[8 * x + 6], k1[8 * x + 7]);
            }
            by[0] = p.scales[t];
            by[1] = p.scales[t + 8];
          }
          sum[h][0] = sum[h][1] = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              mma_f16(s, k0[4 * x], k1[4 * x], k0[4 * x + 1], k1[4 * x + 1], qf[n][x].x, qf[n][x].y);
              mma_f16(s, k0[4 * x + 2], k1[4 * x + 2], k0[4 * x + 3], k1[4 * x + 3], qf[n][x].z, qf[n][x].w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z = FMT == kKeysFp8 ? s[i] * by[i >> 1] : s[i];
              float e = exp2f(fmaf(z, f[n][i & 1], minus[n][i & 1]));
              if (!inside && cur.pos + t + 8 * (i >> 1) > limit[n][i & 1]) e = 0.f;
              sum[h][i >> 1] += e;
            }
          }
        }
        // The quad's lanes hold the rows' sums of four tokens: a lane gets one token's.
        float a0 = c & 1 ? sum[0][1] : sum[0][0], b0 = c & 1 ? sum[0][0] : sum[0][1];
        float a1 = c & 1 ? sum[1][1] : sum[1][0], b1 = c & 1 ? sum[1][0] : sum[1][1];
        a0 += __shfl_xor_sync(0xffffffffu, b0, 1);
        a1 += __shfl_xor_sync(0xffffffffu, b1, 1);
        const float keep = c & 2 ? a1 : a0, give = c & 2 ? a0 : a1;
        const float added = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        const int pos = cur.pos + mine;
        if (pos < cur.len)
          a.weights[at + mine] = pos >= fresh && a.start ? added : fmaf(p.sums[mine], a.decay, added);
      }
      __syncwarp();  // every lane has read the stage
      issue(st);
      st = (st + 1) % RUN_STAGES;
    }
  } while (cur.next(rows, a.B, a.Hkv));
  cp_async_wait<0>();
}

template <int FMT>
cudaError_t launch_tiles(const WeightsArgs& a, cudaStream_t stream, int num_sms) {
  return launch_dependent(attn_weights_kernel<FMT>, dim3(2 * num_sms), dim3(32 * WARPS), 0, stream, a);
}

template <int FMT, int NT>
cudaError_t launch_runs(const WeightsArgs& a, cudaStream_t stream, int num_sms) {
  const size_t smem = sizeof(Piece<FMT>) * RUN_STAGES * RUN_WARPS;
  static_assert(sizeof(Piece<FMT>) * RUN_STAGES * RUN_WARPS <= 220 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(attn_weights_runs_kernel<FMT, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(attn_weights_runs_kernel<FMT, NT>, dim3(num_sms), dim3(32 * RUN_WARPS), smem, stream, a);
}

template <int FMT>
cudaError_t launch_fmt(const WeightsArgs& a, cudaStream_t stream, int num_sms) {
  if constexpr (FMT != kKeysBf16) {
    const int rows = a.rows * a.n_rep;
    if (rows <= 8) return launch_runs<FMT, 1>(a, stream, num_sms);
    if (rows <= 16) return launch_runs<FMT, 2>(a, stream, num_sms);
  }
  return launch_tiles<FMT>(a, stream, num_sms);
}

}  // namespace

// Query tokens in pieces of at most kWeightsMaxRows rows: the first piece applies the decay and
// starts the new rows over, the others add to what it left.
cudaError_t launch_attn_weights(WeightsArgs a, int format, cudaStream_t stream, int num_sms) {
  const int per = kWeightsMaxRows / a.n_rep;
  for (int row0 = 0; row0 < a.q_len; row0 += per) {
    a.row0 = row0;
    a.rows = a.q_len - row0 < per ? a.q_len - row0 : per;
    a.start = row0 == 0;
    if (row0) a.decay = 1.f;
    const cudaError_t e = format == kKeysBf16  ? launch_fmt<kKeysBf16>(a, stream, num_sms)
                          : format == kKeysFp8 ? launch_fmt<kKeysFp8>(a, stream, num_sms)
                                               : launch_fmt<kKeysFp4>(a, stream, num_sms);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
