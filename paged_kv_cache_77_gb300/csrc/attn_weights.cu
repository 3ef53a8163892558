// accumulate_attention_weights: the attention that a step's query rows pay to every cached row
// of their sequence, summed over the query heads of its kv head and added to the row's running
// sum. With the log-sum-exp that the step's attention returned, a weight is
// exp(scale q . k - lse): one pass over the keys, no second pass for a normaliser, no values.
//
// A CTA walks its share of the (sequence, kv head, block) tiles; each of its 8 warps takes 16
// tokens of a tile straight from global memory into the registers of the A operand (the next
// tile's while it works on this one), 8 query rows at a time are the columns of B. One warp
// owns a token: no atomics, the sum's order is fixed.
//
// The keys may be bf16, FP8 (E4M3 with a scale per row) or 4-bit (fp4.cuh). bf16 enters the
// product as it is; the others are exact in fp16, with q scaled by a power of two per row.
// Scores, exponentials and sums are fp32.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "mma_f16.cuh"
#include "pdl.cuh"
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
  __shared__ int si[kWeightsMaxRows];                         // query token of a row
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
  int seg_b = -1, seg_g = -1, first = 0, fresh = 0;
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
      first = cur.len - a.q_len + a.row0;  // position of the launch's first query token
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
          si[r] = r < R ? r / a.n_rep : -(1 << 30);  // no position is that early
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
          const bool seen = (i < 2 ? pa : pb) <= first + si[r];
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

template <int FMT>
cudaError_t launch_fmt(const WeightsArgs& a, cudaStream_t stream, int num_sms) {
  return launch_dependent(attn_weights_kernel<FMT>, dim3(2 * num_sms), dim3(32 * WARPS), 0, stream, a);
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
