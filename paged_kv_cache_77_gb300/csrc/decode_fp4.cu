// Split-KV decode over the 4-bit cache (fp4.cuh has the format).
//
// For each query row, o = softmax(scale q K^T) V over the row's visible positions. A CTA has a
// share of the (sequence, kv head, block) tiles, equal for all CTAs (or, where sequences are few and
// short, all tiles of one sequence and kv head), and every warp of it an
// equal run of that share in pieces of 32 tokens. A warp works alone: it brings its pieces into a
// ring of its own in shared memory with asynchronous copies, keeps a running maximum, sum and
// output in registers, and writes what it finishes. Only the segments that cross from warp to warp are joined, once, when the CTA's share
// is done: the warp in which a segment starts adds up what the later ones left in shared memory.
//
// Both products run on mma.sync with the tokens (K) and the channels (V) as the 16 rows of A
// and the query rows of the kv head as the 8 columns of B, so a group of 8 heads fills the
// instruction. The codes become fp16 in the registers that the product takes them from: a lane
// holds 32 channels of two tokens of K (two 16-byte loads) and 16 channels of four tokens of V
// (four 8-byte loads, their nibbles interleaved so that a byte holds two tokens of a channel).
// A tile in tensor memory would have to pass through shared memory once more, widened to four
// times its size.
//
// Arithmetic. Code times scale is exact in fp16 (6 bits). q is scaled by a power of two per
// row into fp16's range, which keeps its 8 bits but for elements 2^22 times smaller than the
// row's largest. Scores, maxima, sums and outputs are fp32. The weights exp(s - m) enter the
// value product as fp16 (off by at most 2^-11 of themselves), scaled by 2^7 so that a weight keeps
// its 11 bits down to 2^-21 of the largest and counts down to 2^-32; the same rounded weights
// are summed (a row of ones as one more A operand) and divide the output, so that a row of equal
// values keeps its value. The log-sum-exp takes the sum of the unrounded ones.
//
// Roofline: HBM; 144 bytes per token and kv head. Measured on GB300: 64 sequences of up to 32,768
// tokens, 64 / 8 heads (1.16 GB) 192 us, 89 % of the copy rate, 301 warp instructions per 16 tokens and
// kv head, issue slots 68 % busy. Before: the warps of a CTA on one tile, joined at each segment's end
// through shared memory, 368 us (a segment's end cost 6 us, and 64 sequences of up to 2,048 tokens 78 us
// instead of 25); warps with runs of their own 267; an unmasked path 216; copies that need no barrier
// 194. More than 8 query rows per kv head are bound by instructions: 16 rows 56 % of the copy rate.
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

constexpr int D = 128;
constexpr int CODES = SUB * fp4::kCodeBytes;     // 2048
constexpr int SCALES = SUB * fp4::kScaleBytes;   // 256
constexpr int STAGE = 2 * (CODES + SCALES);      // K codes, V codes, K scales, V scales
constexpr float kShift = 7.f;                    // weights are 2^kShift exp(s - m)
constexpr float kLazy = 8.f;                     // a maximum may be passed by this much (log2)

// NT: 8-row tiles of query rows.
template <int NT>
struct Shape {
  static constexpr int WARPS = NT == 1 ? 16 : 8;
  static constexpr int STAGES = NT == 1 ? 2 : 4;
};

enum : int { kNothing = 0, kGoesOn = 1, kEnds = 2 };  // what a warp left of its first segment

template <int NT>
struct Smem {
  uint8_t stage[Shape<NT>::WARPS][Shape<NT>::STAGES][STAGE];
  float4 o[Shape<NT>::WARPS][NT][8][32];      // a warp's part of a segment that an earlier one began
  float stat[Shape<NT>::WARPS][NT][3][8];     // its maxima, sums, sums of the unrounded weights
  int left[Shape<NT>::WARPS];
  int64_t total;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// A running softmax over part of a segment, spread over the lanes of a warp: lane 4 g + c has the
// query rows 8 n + 2 c and 8 n + 2 c + 1 (x = 0, 1), of their outputs channels 16 g .. + 15
// (o[n][d][x] and o[n][d][x + 2]: channels 16 g + 2 d and 16 g + 2 d + 1).
template <int NT>
struct Running {
  float m[NT][2];        // maximum, log2
  float l[NT][4];        // sum of the rounded weights ([2], [3]: copies)
  float sum[NT][2];      // this lane's sum of the unrounded ones
  float o[NT][8][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) l[n][i] = 0.f;
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
    }
  }
  __device__ __forceinline__ void scale_row(int n, int x, float by) {
    l[n][x] *= by;
    sum[n][x] *= by;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      o[n][d][x] *= by;
      o[n][d][x + 2] *= by;
    }
  }
  __device__ __forceinline__ void sum_lanes() {  // every lane of a row gets the row's whole sum
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[n][x] += __shfl_xor_sync(0xffffffffu, sum[n][x], d);
  }
};

template <int NT>
__device__ __forceinline__ void leave(Smem<NT>& sm, int warp, int lane, const Running<NT>& r) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int d = 0; d < 8; ++d) sm.o[warp][n][d][lane] = make_float4(r.o[n][d][0], r.o[n][d][1], r.o[n][d][2], r.o[n][d][3]);
    if (lane < 4) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sm.stat[warp][n][0][2 * lane + x] = r.m[n][x];
        sm.stat[warp][n][1][2 * lane + x] = r.l[n][x];
        sm.stat[warp][n][2][2 * lane + x] = r.sum[n][x];
      }
    }
  }
}

template <int NT>
__device__ __forceinline__ void take(const Smem<NT>& sm, int warp, int lane, Running<NT>& r) {
  const int c = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float by[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float other = sm.stat[warp][n][0][2 * c + x];
      const float top = fmaxf(r.m[n][x], other);
      // (A part without a finite score has sums of 0, or NaN, which any factor keeps.)
      r.scale_row(n, x, r.m[n][x] == -INFINITY ? 1.f : exp2_approx(r.m[n][x] - top));
      by[x] = other == -INFINITY ? 1.f : exp2_approx(other - top);
      r.m[n][x] = top;
      r.l[n][x] += sm.stat[warp][n][1][2 * c + x] * by[x];
      r.sum[n][x] += sm.stat[warp][n][2][2 * c + x] * by[x];
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const float4 v = sm.o[warp][n][d][lane];
      r.o[n][d][0] += v.x * by[0];
      r.o[n][d][1] += v.y * by[1];
      r.o[n][d][2] += v.z * by[0];
      r.o[n][d][3] += v.w * by[1];
    }
  }
}

// Writes a segment's rows, or a part of them (slot >= 0) to the workspace.
template <int NT>
__device__ __forceinline__ void put(const DecodeFp4Args& a, const Running<NT>& r, int lane, int b, int kv, int64_t slot) {
  const int g = lane >> 2, c = lane & 3, R = a.n_rep * a.q_len;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 8 * n + 2 * c + x;
      if (row >= R) continue;
      // A sum that is not a number (a NaN score) makes the row's output and lse NaN.
      const bool none = r.l[n][x] == 0.f;
      const float inv = none ? 0.f : 1.f / r.l[n][x];
      const float lse2 = none ? -INFINITY : r.m[n][x] + log2f(r.sum[n][x]) - kShift;
      float v[16];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        v[2 * d] = r.o[n][d][x] * inv;
        v[2 * d + 1] = r.o[n][d][x + 2] * inv;
      }
      const int64_t at = slot >= 0 ? slot * R + row
                                   : ((int64_t)b * a.q_total + a.row0 + row / a.n_rep) * a.H +
                                         (int64_t)kv * a.n_rep + row % a.n_rep;
      if (slot >= 0 || a.out_f32) {
        float4* dst = reinterpret_cast<float4*>((slot >= 0 ? a.ws_o : reinterpret_cast<float*>(a.out)) + at * D + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + at * D + 16 * g);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if (g == 0) {
        if (slot >= 0)
          a.ws_lse[at] = lse2;
        else if (a.lse)
          a.lse[at] = lse2 * kLn2;
      }
    }
}

// All warps' parts of the CTA's one segment, summed by all threads, two channels of two rows each.
template <int NT>
__device__ __forceinline__ void join(const DecodeFp4Args& a, const Smem<NT>& sm, int b, int kv) {
  constexpr int WARPS = Shape<NT>::WARPS;
  const int R = a.n_rep * a.q_len;
  for (int item = threadIdx.x; item < NT * 256; item += 32 * WARPS) {
    const int n = item >> 8, d = item >> 5 & 7, lane = item & 31, g = lane >> 2, c = lane & 3;
    float top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (sm.left[w] != kNothing) {
        const float2 m = *reinterpret_cast<const float2*>(&sm.stat[w][n][0][2 * c]);
        top[0] = fmaxf(top[0], m.x);
        top[1] = fmaxf(top[1], m.y);
      }
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (sm.left[w] != kNothing) {
        const float2 m = *reinterpret_cast<const float2*>(&sm.stat[w][n][0][2 * c]);
        const float2 part = *reinterpret_cast<const float2*>(&sm.stat[w][n][1][2 * c]);
        const float2 exact = *reinterpret_cast<const float2*>(&sm.stat[w][n][2][2 * c]);
        const float4 v = sm.o[w][n][d][lane];
        // (A part without a finite score has sums of 0, or NaN, which any factor keeps.)
        const float by0 = m.x == -INFINITY ? 1.f : exp2_approx(m.x - top[0]);
        const float by1 = m.y == -INFINITY ? 1.f : exp2_approx(m.y - top[1]);
        l[0] += part.x * by0;
        l[1] += part.y * by1;
        sum[0] += exact.x * by0;
        sum[1] += exact.y * by1;
        o[0] += v.x * by0;
        o[1] += v.y * by1;
        o[2] += v.z * by0;
        o[3] += v.w * by1;
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 8 * n + 2 * c + x;
      if (row >= R) continue;
      const bool none = l[x] == 0.f;
      const float inv = none ? 0.f : 1.f / l[x];
      const int64_t at = ((int64_t)b * a.q_total + a.row0 + row / a.n_rep) * a.H + (int64_t)kv * a.n_rep + row % a.n_rep;
      const int64_t to = at * D + 16 * g + 2 * d;
      if (a.out_f32)
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + to) = make_float2(o[x] * inv, o[x + 2] * inv);
      else
        *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<uint16_t*>(a.out) + to) =
            __floats2bfloat162_rn(o[x] * inv, o[x + 2] * inv);
      if (a.lse && d == 0 && g == 0) a.lse[at] = none ? -INFINITY : (top[x] + log2f(sum[x]) - kShift) * kLn2;
    }
  }
}

// What the query rows of a launch see of a sequence: row i (of the call's) the positions in
// (first + i - window, first + i].
struct Sight {
  int first, window, row0, rows;
  __device__ __forceinline__ bool sees(int pos, int i) const {
    return pos <= first + i && (window <= 0 || pos > first + i - window);
  }
  __device__ __forceinline__ bool any(int pos) const {  // of the launch's rows
    return pos <= first + row0 + rows - 1 && (window <= 0 || pos > first + row0 - window);
  }
  __device__ __forceinline__ bool all(int lo, int hi) const {  // every row every position of [lo, hi]
    return hi <= first + row0 && (window <= 0 || lo > first + row0 + rows - 1 - window);
  }
};

// N times 16 tokens, from position p0 on, whose codes and scales lie at kc, vc, ks and vs in shared
// memory. kMask: some row may not see some of them.
template <int NT, int N, bool kMask>
__device__ __forceinline__ void attend(Running<NT>& r, const uint4 (&qf)[NT][4], const float (&f)[NT][2],
                                       float (&limit)[NT][2], float (&shift)[NT][2],
                                       const int (&row_i)[NT][2], const uint8_t* kc, const uint8_t* vc,
                                       const uint8_t* ks, const uint8_t* vs, int p0, const Sight& sight,
                                       int g, int c) {
  // ---- scores: 16 tokens x 8 NT query rows at a time
  float s[N][NT][4];
#pragma unroll
  for (int h = 0; h < N; ++h) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[h][n][i] = 0.f;
    const int r0 = 16 * h + token_of(g);
    const uint4 w0 = *reinterpret_cast<const uint4*>(kc + r0 * fp4::kCodeBytes + 16 * c);
    const uint4 w1 = *reinterpret_cast<const uint4*>(kc + (r0 + 8) * fp4::kCodeBytes + 16 * c);
    const uint32_t e0 = *reinterpret_cast<const uint16_t*>(ks + r0 * fp4::kScaleBytes + 2 * c);
    const uint32_t e1 = *reinterpret_cast<const uint16_t*>(ks + (r0 + 8) * fp4::kScaleBytes + 2 * c);
    const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t sc0 = i < 2 ? fp4::scale_dup0(e0) : fp4::scale_dup1(e0);
      const uint32_t sc1 = i < 2 ? fp4::scale_dup0(e1) : fp4::scale_dup1(e1);
      uint32_t y0[4], y1[4];
      fp4::widen(x0[i], y0);
      fp4::widen(x1[i], y1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y0[k] = fp4::mul2(y0[k], sc0);
        y1[k] = fp4::mul2(y1[k], sc1);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_f16(s[h][n], y0[0], y1[0], y0[1], y1[1], qf[n][i].x, qf[n][i].y);
        mma_f16(s[h][n], y0[2], y1[2], y0[3], y1[3], qf[n][i].z, qf[n][i].w);
      }
    }
  }
  // ---- running maxima, raised only when a score passes one by 2^kLazy (limit: that score)
  bool past = false;
  bool seen[N][NT][4];
  float top[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      top[n][x] = -INFINITY;
#pragma unroll
      for (int h = 0; h < N; ++h)
#pragma unroll
        for (int i = x; i < 4; i += 2) {
          seen[h][n][i] = !kMask || sight.sees(p0 + 16 * h + token_of(g) + (i >> 1) * 8, row_i[n][x]);
          top[n][x] = fmaxf(top[n][x], seen[h][n][i] ? s[h][n][i] : -INFINITY);
        }
      past = past || top[n][x] > limit[n][x];
    }
  if (__any_sync(0xffffffffu, past)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float t = top[n][x] == -INFINITY ? -INFINITY : top[n][x] * f[n][x];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
        t = fmaxf(r.m[n][x], t);
        r.scale_row(n, x, r.m[n][x] == -INFINITY ? 1.f : exp2_approx(r.m[n][x] - t));
        r.m[n][x] = t;
        if (t > -INFINITY) {
          limit[n][x] = (t + kLazy) / f[n][x];
          shift[n][x] = kShift - t;
        }
      }
  }
  // ---- weights, transposed into the B operand of the value product
  uint32_t pb[N][NT][2];
#pragma unroll
  for (int h = 0; h < N; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = seen[h][n][i] ? exp2_approx(fmaf(s[h][n][i], f[n][i & 1], shift[n][i & 1])) : 0.f;
        r.sum[n][i & 1] += p[i];
      }
      pb[h][n][0] = transpose8(pack_f16(p[0], p[1]));
      pb[h][n][1] = transpose8(pack_f16(p[2], p[3]));
    }
  // ---- values: of each 16 tokens the four of rows 2c, 2c + 1, 2c + 8, 2c + 9; channels 16 g .. + 15
  const int even = even_row(c);
#pragma unroll
  for (int h = 0; h < N; ++h) {
    uint2 w[4];
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * h + (even ^ (i & 1 ? 3 : 0)) + (i & 2) * 4;
      w[i] = *reinterpret_cast<const uint2*>(vc + t * fp4::kCodeBytes + 8 * g);
      e[i] = vs[t * fp4::kScaleBytes + g];
    }
    uint32_t poison = 0;
    if (kMask) {
      // A token that no row sees may hold any bytes, and 0 times NaN is NaN: its scales become zero.
      // So do those past the largest of a token that some rows see; the rows that do see it get their
      // NaN below.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = (even ^ (i & 1 ? 3 : 0)) + (i & 2) * 4;
        const bool by_some = sight.any(p0 + 16 * h + t);
        if (by_some && e[i] > (uint32_t)fp4::kMaxScale) poison |= 1u << t;
        if (!by_some || e[i] > (uint32_t)fp4::kMaxScale) e[i] = 0;
      }
    }
    const uint32_t sa = fp4::scale_pair(e[0], e[1]), sb = fp4::scale_pair(e[2], e[3]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x0 = k ? w[0].y : w[0].x, x1 = k ? w[1].y : w[1].x;
      const uint32_t x2 = k ? w[2].y : w[2].x, x3 = k ? w[3].y : w[3].x;
      constexpr uint32_t lo = 0x0f0f0f0fu, hi = 0xf0f0f0f0u;
      uint32_t a0[4], a1[4], a2[4], a3[4];
      fp4::widen((x0 & lo) | (x1 << 4 & hi), a0);  // even channels
      fp4::widen((x0 >> 4 & lo) | (x1 & hi), a1);  // odd ones
      fp4::widen((x2 & lo) | (x3 << 4 & hi), a2);
      fp4::widen((x2 >> 4 & lo) | (x3 & hi), a3);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t y0 = fp4::mul2(a0[d], sa), y1 = fp4::mul2(a1[d], sa);
        const uint32_t y2 = fp4::mul2(a2[d], sb), y3 = fp4::mul2(a3[d], sb);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16(r.o[n][4 * k + d], y0, y1, y2, y3, pb[h][n][0], pb[h][n][1]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      mma_f16(r.l[n], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pb[h][n][0], pb[h][n][1]);
    if (kMask) {
      poison |= __shfl_xor_sync(0xffffffffu, poison, 1);
      poison |= __shfl_xor_sync(0xffffffffu, poison, 2);
      for (; poison; poison &= poison - 1) {
        const int pos = p0 + 16 * h + __ffs((int)poison) - 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!sight.sees(pos, row_i[n][x])) continue;
#pragma unroll
            for (int d = 0; d < 8; ++d) r.o[n][d][x] = r.o[n][d][x + 2] = __uint_as_float(0x7fc00000u);
          }
      }
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(32 * Shape<NT>::WARPS, 1) decode_fp4_kernel(const __grid_constant__ DecodeFp4Args a) {
  constexpr int WARPS = Shape<NT>::WARPS, STAGES = Shape<NT>::STAGES;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<NT>& sm = *reinterpret_cast<Smem<NT>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, and known to be)
  const DenseRows rows = {a.seq_lens, TILE, a.window, a.max_blocks * TILE};
  pdl_wait_then_launch();
  int64_t t0 = 0, t1;  // the CTA's blocks
  int seg_b = 0, seg_g = 0, seg_len = 0, seg_lo = 0;
  if (a.whole) {
    seg_b = blockIdx.x / a.Hkv;
    seg_g = blockIdx.x % a.Hkv;
    const int raw = rows.raw(seg_b);
    seg_len = clamp_len(raw, rows.cap);
    if (raw != seg_len && seg_g == 0 && tid == 0) flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
    const SeqRange range = rows.blocks(seg_len);
    seg_lo = range.jlo;
    t1 = range.n;
    if (range.n == 0) {
      if (warp == 0) {
        Running<NT> none;
        none.clear();
        put(a, none, lane, seg_b, seg_g, -1);
      }
      return;
    }
  } else {
    if (warp == 0) {
      const int64_t tot = total_live_blocks(rows, a.B, a.dev_status);
      if (lane == 0) sm.total = tot * a.Hkv;
    }
    __syncthreads();
    const int64_t T = sm.total, G = min((int64_t)gridDim.x, T);
    if (blockIdx.x >= G) return;
    t0 = cta_tile_start(blockIdx.x, T, G);
    t1 = cta_tile_start(blockIdx.x + 1, T, G);
  }

  // This warp's run: pieces u0 .. u1 - 1 of the CTA's.
  const int64_t u0 = Walk::run(t1 - t0, warp, WARPS), u1 = Walk::run(t1 - t0, warp + 1, WARPS);
  const int g = lane >> 2, c = lane & 3, R = a.n_rep * a.q_len;
  Running<NT> r;
  Walk cur = {};
  bool begun = false;  // whether the segment that the warp is in began in its run
  bool open = false;   // whether it goes on behind the run, and is this warp's to finish
  int left = kNothing;
  if (u0 < u1) {
    if (a.whole) {
      cur.start(seg_b, seg_g, seg_len, seg_lo, (int)u0, (int)u1);
      begun = u0 == 0;
    } else {
      begun = cur.seek(rows, a.B, a.Hkv, t0, t1, u0, u1);
    }
    // ---- the ring: the run's it-th visited piece is in stage it % STAGES, one group of
    // asynchronous copies each. A lane copies 16 bytes of every eighth row of the codes, and 16 bytes
    // of the scales of K (lanes 0 to 15) or V.
    Walk ahead = cur;
    bool more = true;
    int ids = 0, ids_j = -64;  // 32 table entries of the sequence, from block ids_j on
    bool enter = true;         // whether the piece's block has to be looked up
    const uint8_t *k_src = nullptr, *v_src = nullptr, *s_src = nullptr;
    unsigned bad = 0;          // stages whose block does not exist
    const uint32_t ring = smem_u32(sm.stage[warp]) + 16 * lane;
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
          const bool ok = blk >= 0 && (int64_t)blk < a.num_blocks;
          if (!ok && lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
          const int64_t row = ((int64_t)(ok ? blk : 0) * a.Hkv + ahead.g) * TILE + ahead.pos % TILE;
          k_src = ok ? a.k_cache + row * fp4::kCodeBytes + 16 * lane : nullptr;
          v_src = a.v_cache + row * fp4::kCodeBytes + 16 * lane;
          s_src = (lane < 16 ? a.k_scale4 : a.v_scale4) + row * fp4::kScaleBytes + 16 * (lane & 15);
        }
        const uint32_t dst = ring + st * STAGE;
        if (k_src != nullptr) {
          bad &= ~(1u << st);
          if (ahead.len - ahead.pos >= SUB) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              cp_async_16(dst + 512 * i, k_src + 512 * i, 16);
              cp_async_16(dst + CODES + 512 * i, v_src + 512 * i, 16);
            }
            cp_async_16(dst + 2 * CODES, s_src, 16);
          } else {
            // Zeros instead of the rows behind the sequence's end (two rows of scales at a time).
            const int live = ahead.len - ahead.pos;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t bytes = 8 * i + (lane >> 2) < live ? 16 : 0;
              cp_async_16(dst + 512 * i, k_src + 512 * i, bytes);
              cp_async_16(dst + CODES + 512 * i, v_src + 512 * i, bytes);
            }
            cp_async_16(dst + 2 * CODES, s_src, 2 * (lane & 15) < live ? 16 : 0);
          }
          k_src += CODES;
        } else {
          bad |= 1u << st;
        }
        v_src += CODES;
        s_src += SCALES;
        ahead.pos += SUB;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < STAGES; ++st) issue(st);

    int row_i[NT][2];  // query tokens of this lane's rows
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) row_i[n][x] = a.row0 + min(n * 8 + 2 * c + x, R - 1) / a.n_rep;
    const bool reaches_in = u0 == 0 && !begun;  // the run starts with a segment of the CTA before
    for (int st = 0, seg = 0;; ++seg) {
      if (seg) begun = true;
      r.clear();
      uint4 qf[NT][4];              // B operands of the scores
      // Factors of this lane's rows, scores that raise their maxima, kShift less their maxima.
      float f[NT][2], limit[NT][2], shift[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g;
        const uint16_t* src = a.q + (((int64_t)cur.b * a.q_total + a.row0 + row / a.n_rep) * a.H +
                                     (int64_t)cur.g * a.n_rep + row % a.n_rep) * D + 32 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[n][i] = row < R ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        const float down = query_to_f16(qf[n]) * a.scale_log2;
        f[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);
        f[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
        limit[n][0] = limit[n][1] = -INFINITY;
        shift[n][0] = shift[n][1] = kShift;
      }
      const Sight sight = {cur.len - a.q_total, a.row_window, a.row0, a.q_len};
      for (; cur.pos < cur.stop; cur.pos += SUB) {
        cp_async_wait<STAGES - 1>();
        __syncwarp();  // every lane's copies are there
        if (!(bad >> st & 1)) {
          const uint8_t* tile = sm.stage[warp][st];
          const uint8_t *k = tile, *v = tile + CODES, *ks = tile + 2 * CODES, *vs = ks + SCALES;
          constexpr int C16 = 16 * fp4::kCodeBytes, S16 = 16 * fp4::kScaleBytes;
          if (sight.all(cur.pos, cur.pos + SUB - 1)) {
            attend<NT, 2, false>(r, qf, f, limit, shift, row_i, k, v, ks, vs, cur.pos, sight, g, c);
          } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
              attend<NT, 1, true>(r, qf, f, limit, shift, row_i, k + h * C16, v + h * C16, ks + h * S16,
                                  vs + h * S16, cur.pos + 16 * h, sight, g, c);
          }
        }
        __syncwarp();  // every lane has read the stage
        issue(st);
        st = (st + 1) % STAGES;
      }
      r.sum_lanes();
      const bool own = !a.whole && (begun || reaches_in);
      if (cur.ends && own) {
        put(a, r, lane, cur.b, cur.g, begun ? (int64_t)-1 : (int64_t)a.B * a.Hkv + blockIdx.x);
      } else if (own) {
        open = true;
      } else {
        leave(sm, warp, lane, r);
        left = cur.ends ? kEnds : kGoesOn;
      }
      if (!cur.ends || !cur.next(rows, a.B, a.Hkv)) break;
    }
    cp_async_wait<0>();
  }
  if (lane == 0) sm.left[warp] = left;
  __syncthreads();
  if (a.whole) {
    join(a, sm, seg_b, seg_g);
    return;
  }
  if (!open) return;
  // The segment that this warp began (or that reaches into the CTA's share from the one before)
  // goes on in the next warps.
  bool ended = false;
  for (int x = warp + 1; x < WARPS && !ended; ++x) {
    if (sm.left[x] == kNothing) continue;
    take(sm, x, lane, r);
    ended = sm.left[x] == kEnds;
  }
  put(a, r, lane, cur.b, cur.g,
      begun ? (ended ? (int64_t)-1 : (int64_t)cur.b * a.Hkv + cur.g) : (int64_t)a.B * a.Hkv + blockIdx.x);
}

template <int NT>
cudaError_t launch_n(const DecodeFp4Args& a, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<NT>);
  static_assert(sizeof(Smem<NT>) <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(decode_fp4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_fp4_kernel<NT>, dim3(a.whole ? a.B * a.Hkv : a.num_ctas), dim3(32 * Shape<NT>::WARPS), smem, stream, a);
}

}  // namespace

// Query tokens in pieces of at most 16 rows per kv head, each with a pass over the cache of its own.
cudaError_t launch_decode_fp4(DecodeFp4Args a, cudaStream_t stream) {
  const int per = 16 / a.n_rep;
  // Short sequences, no more (sequence, kv head) pairs than SMs: a CTA each. The second launch and the
  // joins in memory cost more than the SMs left idle. Measured on GB300 (us shared out, and a CTA each):
  // 64 pairs of up to 512 tokens 10.5, 7.1, 2,048 11.4, 9.5, 4,096 13.4, 13.6, all of 4,096 17.2, 19.8; 128 of
  // 2,048 17.7, 13.2; 8 of up to 2,048 10.6, 8.9; 1 of 2,048 10.9, 12.5; 256 of up to 128 9.5, 12.7. With 16
  // rows: 64 pairs of up to 1,024 tokens 13.8, 11.2, 2,048 13.9, 16.6. The host knows the table's width, not the
  // lengths: behind a wider table short sequences are shared out.
  const int most = a.q_total < per ? a.q_total : per;
  a.whole = a.max_blocks <= (most * a.n_rep <= 8 ? 16 : 8) && a.B * a.Hkv <= a.num_ctas;
  for (a.row0 = 0; a.row0 < a.q_total; a.row0 += per) {
    a.q_len = a.q_total - a.row0 < per ? a.q_total - a.row0 : per;
    cudaError_t e = a.n_rep * a.q_len <= 8 ? launch_n<1>(a, stream) : launch_n<2>(a, stream);
    if (e == cudaSuccess && !a.whole) e = launch_decode_merge(a, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
