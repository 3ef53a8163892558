// Split-KV decode over the 4-bit cache (fp4.cuh has the format).
//
// For each query row, o = softmax(scale q K^T) V over the row's visible positions. A CTA walks
// its share of the (sequence, kv head, block) tiles; a tile is 18 KB in four contiguous pieces
// (K codes, V codes, their scales) that one warp brings into a ring in shared memory with bulk
// copies. Every consumer warp takes 16 tokens of a tile and keeps its own running maximum, sum
// and output in registers; the warps meet once per segment.
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
// are summed (a row of ones as one more A operand) and divide the output.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "mma_f16.cuh"
#include "pdl.cuh"
#include "query_f16.cuh"
#include "row_cursor.cuh"
#include "tc_ptx.cuh"

namespace pkv {
namespace {

constexpr int BS = 128, D = 128;
constexpr int CODES = BS * fp4::kCodeBytes;    // 8192
constexpr int SCALES = BS * fp4::kScaleBytes;  // 1024
constexpr int STAGE = 2 * (CODES + SCALES);    // K codes, V codes, K scales, V scales
constexpr int OPAD = 132;                      // floats per output row of a warp's partial
constexpr float kShift = 7.f;                  // weights are 2^kShift exp(s - m)
constexpr float kLazy = 8.f;                   // a maximum may be passed by this much (log2)

template <int NT>
struct Shape {
  static constexpr int WARPS = NT == 1 ? 16 : 8;  // consumer warps
  static constexpr int GROUPS = WARPS / 8;        // tiles worked on at once
  static constexpr int STAGES = 8;
  static constexpr int THREADS = 32 * (WARPS + 1);
};

template <int NT>
struct Smem {
  uint8_t stage[Shape<NT>::STAGES][STAGE];
  float o[Shape<NT>::WARPS][8][OPAD];
  float m[NT][Shape<NT>::WARPS][8], l[Shape<NT>::WARPS][8];
  uint4 q[NT == 1 ? 1 : NT][4][32];     // B operands of the scores, for more than 8 rows
  float f[NT][8];                       // score factor of each row
  uint64_t full[Shape<NT>::STAGES], empty[Shape<NT>::STAGES];
  int ok[Shape<NT>::STAGES];            // whether the tile's block exists
  int64_t total;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// Row r (0..7) of a product's 8 rows is token token_of(r): lanes c and c + 4 of a quad's V
// loads then take four consecutive tokens, which lie in different banks.
__device__ __forceinline__ int token_of(int r) { return (r >> 1) + ((r & 1) << 2); }

// A lane's 32 consecutive channels of a query row (null: a row of zeros) as fp16, and the power
// of two that was taken out of the row.
__device__ __forceinline__ float load_query(const uint16_t* x, uint4 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = x ? __ldg(reinterpret_cast<const uint4*>(x) + i) : make_uint4(0, 0, 0, 0);
  return query_to_f16(w);
}

template <int NT>
__global__ void __launch_bounds__(Shape<NT>::THREADS, 1) decode_fp4_kernel(const __grid_constant__ DecodeArgs a) {
  using S = Shape<NT>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<NT>& sm = *reinterpret_cast<Smem<NT>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const DenseRows rows = {a.seq_lens, BS, a.window, a.max_blocks * BS};
  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      tc::mbar_init(smem_u32(&sm.full[i]), 1);
      tc::mbar_init(smem_u32(&sm.empty[i]), 8);
    }
    tc::fence_mbar_init();
  }
  pdl_wait_then_launch();
  if (warp == 0) {
    const int64_t tot = total_live_blocks(rows, a.B, a.dev_status);
    if (lane == 0) sm.total = tot * a.Hkv;
  }
  __syncthreads();
  const int64_t T = sm.total, G = gridDim.x;
  const int64_t t0 = cta_tile_start(blockIdx.x, T, G), t1 = cta_tile_start(blockIdx.x + 1, T, G);
  if (t0 >= t1) return;
  TileCursor cur;
  cursor_seek_warp(cur, rows, a.B, a.Hkv, t0, t1);

  if (warp == S::WARPS) {
    // ---------------------------------------------------------------- producer
    int ids = 0, ids_b = -1, ids_j = 0;  // 32 table entries of sequence ids_b, from ids_j on
    int it = 0;
    bool alive = true;
    do {
      const int st = it % S::STAGES;
      if (cur.b != ids_b || cur.j < ids_j || cur.j >= ids_j + 32) {
        ids_b = cur.b;
        ids_j = cur.j;
        ids = cur.j + lane < cur.n
                  ? __ldg(a.block_table + (int64_t)cur.b * a.max_blocks + cur.jlo + cur.j + lane)
                  : 0;
      }
      const int blk = __shfl_sync(0xffffffffu, ids, cur.j - ids_j);
      const bool ok = blk >= 0 && (int64_t)blk < a.num_blocks;
      if (!ok && lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
      if (it >= S::STAGES) alive = tc::mbar_wait_sleepy(smem_u32(&sm.empty[st]), (it / S::STAGES - 1) & 1);
      if (!__all_sync(0xffffffffu, alive)) break;
      const uint32_t full = smem_u32(&sm.full[st]);
      // Rows behind the sequence's end stay where they are (an even number is copied: 16 bytes
      // of scales are two rows).
      const int live = min(BS, (cur.len - (cur.jlo + cur.j) * BS + 1) & ~1);
      if (lane == 0) {
        sm.ok[st] = ok;
        tc::mbar_expect_tx(full, ok ? (uint32_t)live * 2 * (fp4::kCodeBytes + fp4::kScaleBytes) : 0u);
      }
      __syncwarp();
      if (ok && lane < 4) {
        const int64_t row = ((int64_t)blk * a.Hkv + cur.g) * BS;
        const uint32_t dst = smem_u32(sm.stage[st]);
        if (lane < 2)
          bulk_load(dst + lane * CODES, (lane ? a.v_cache : a.k_cache) + row * fp4::kCodeBytes,
                    live * fp4::kCodeBytes, full);
        else
          bulk_load(dst + 2 * CODES + (lane - 2) * SCALES,
                    (lane == 3 ? a.v_scale4 : a.k_scale4) + row * fp4::kScaleBytes,
                    live * fp4::kScaleBytes, full);
      }
      ++it;
    } while (cursor_next(cur, rows, a.B, a.Hkv));
    if (!__all_sync(0xffffffffu, alive)) {
      if (lane == 0) flag_status(a.dev_status, PKV_DEV_TIMEOUT);
      // Nothing may land in shared memory after the block has gone.
      for (int i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i)
        tc::mbar_wait_sleepy(smem_u32(&sm.full[i % S::STAGES]), (i / S::STAGES) & 1);
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, c = lane & 3;
  const int tb = (warp & 7) * 16;  // this warp's tokens of a tile
  const int R = a.n_rep * a.q_len;
  uint4 qf[4];                     // NT == 1 only
  float f[NT][2], m[NT][2], o[NT][8][4], l[NT][4];
  int row_i[NT][2];                // query token of this lane's rows
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) row_i[n][x] = min(n * 8 + 2 * c + x, R - 1) / a.n_rep;
  int64_t piece_first = t0;
  int it = 0;
  bool dead = false;
  for (;;) {
    if (cur.t == t0 || cur.j == 0) {
      piece_first = cur.t;
      auto query = [&](int r) {
        return r < R ? a.q + (((int64_t)cur.b * a.q_len + r / a.n_rep) * a.H + (int64_t)cur.g * a.n_rep +
                              r % a.n_rep) * D + 32 * c
                     : nullptr;
      };
      if constexpr (NT == 1) {
        const float down = load_query(query(g), qf) * a.scale_log2;
        f[0][0] = __shfl_sync(0xffffffffu, down, 8 * c);
        f[0][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      } else {
        if (warp < NT) {
          const float down = load_query(query(warp * 8 + g), qf);
#pragma unroll
          for (int i = 0; i < 4; ++i) sm.q[warp][i][lane] = qf[i];
          if (c == 0) sm.f[warp][g] = down * a.scale_log2;
        }
        tc::named_bar_sync(1, S::WARPS * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f[n][0] = sm.f[n][2 * c];
          f[n][1] = sm.f[n][2 * c + 1];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) l[n][i] = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][x][i] = 0.f;
      }
    }

    if (S::GROUPS == 1 || (it % S::GROUPS) == (warp >> 3)) {
      const int st = it % S::STAGES;
      if (!dead && !tc::mbar_wait(smem_u32(&sm.full[st]), (it / S::STAGES) & 1)) {
        dead = true;
        flag_status(a.dev_status, PKV_DEV_TIMEOUT);
      }
      dead = __any_sync(0xffffffffu, dead);
      const int p0 = (cur.jlo + cur.j) * BS + tb;  // position of this warp's first token
      // Positions that the query rows see: row i those in (first + i - window, first + i].
      const int first = cur.len - a.q_len;
      const int low = a.row_window > 0 ? max(first - a.row_window + 1, 0) : 0;  // of row 0
      if (!dead && sm.ok[st] && p0 < cur.len && p0 + 15 >= low) {
        const uint8_t* kc = sm.stage[st] + tb * fp4::kCodeBytes;
        const uint8_t* vc = kc + CODES;
        const uint8_t* ks = sm.stage[st] + 2 * CODES + tb * fp4::kScaleBytes;
        const uint8_t* vs = ks + SCALES;
        // Whether every query row sees all 16 tokens.
        const bool inside = p0 + 15 <= first && (a.row_window <= 0 || p0 >= cur.len - a.row_window);

        // ---- scores: 16 tokens x 8 NT query rows
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
        {
          const int r0 = token_of(g);
          const uint4 w0 = *reinterpret_cast<const uint4*>(kc + r0 * fp4::kCodeBytes + 16 * c);
          const uint4 w1 = *reinterpret_cast<const uint4*>(kc + (r0 + 8) * fp4::kCodeBytes + 16 * c);
          const uint32_t u0 = *reinterpret_cast<const uint16_t*>(ks + r0 * fp4::kScaleBytes + 2 * c);
          const uint32_t u1 = *reinterpret_cast<const uint16_t*>(ks + (r0 + 8) * fp4::kScaleBytes + 2 * c);
          const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sc0 = i < 2 ? fp4::scale_dup0(u0) : fp4::scale_dup1(u0);
            const uint32_t sc1 = i < 2 ? fp4::scale_dup0(u1) : fp4::scale_dup1(u1);
            uint32_t y0[4], y1[4];
            fp4::widen(x0[i], y0);
            fp4::widen(x1[i], y1);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              y0[h] = fp4::mul2(y0[h], sc0);
              y1[h] = fp4::mul2(y1[h], sc1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 b;
              if constexpr (NT == 1)
                b = qf[i];
              else
                b = sm.q[n][i][lane];
              mma_f16(s[n], y0[0], y1[0], y0[1], y1[1], b.x, b.y);
              mma_f16(s[n], y0[2], y1[2], y0[3], y1[3], b.z, b.w);
            }
          }
        }
        const int pa = p0 + token_of(g);  // position of s[.][0..1]; s[.][2..3] is 8 further
        bool past = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[n][i];
            x *= f[n][i & 1];
            if (!inside) {
              const int pos = pa + (i >> 1) * 8, at = first + row_i[n][i & 1];
              if (pos > at || (a.row_window > 0 && pos <= at - a.row_window)) x = -INFINITY;
            }
            past |= x > m[n][i & 1] + kLazy;
          }
        // ---- running maxima, raised only when a score passes one by 2^kLazy
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float t = fmaxf(s[n][x], s[n][x + 2]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
              const float top = fmaxf(m[n][x], t);
              const float scale = m[n][x] == -INFINITY ? 0.f : exp2_approx(m[n][x] - top);
              m[n][x] = top;
              l[n][x] *= scale;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[n][d][x] *= scale;
                o[n][d][x + 2] *= scale;
              }
            }
        }
        // ---- weights, transposed into the B operand of the value product
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float base[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) base[x] = m[n][x] == -INFINITY ? 0.f : m[n][x] - kShift;
          pb[n][0] = transpose8(pack_f16(exp2_approx(s[n][0] - base[0]), exp2_approx(s[n][1] - base[1])));
          pb[n][1] = transpose8(pack_f16(exp2_approx(s[n][2] - base[0]), exp2_approx(s[n][3] - base[1])));
        }
        // ---- values: tokens c, c + 4, c + 8, c + 12; channels 16 g .. 16 g + 15
        uint2 w[4];
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = *reinterpret_cast<const uint2*>(vc + (c + 4 * i) * fp4::kCodeBytes + 8 * g);
          u[i] = vs[(c + 4 * i) * fp4::kScaleBytes + g];
        }
        uint32_t poison = 0;
        if (!inside) {
          // A token that no row sees may hold any bytes, and 0 times NaN is NaN: its scales become
          // zero. So do those past the largest of a token that some rows see; the rows that do see
          // it get their NaN below.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = p0 + c + 4 * i;
            const bool seen = pos < cur.len && pos >= low;
            if (seen && u[i] > (uint32_t)fp4::kMaxScale) poison |= 1u << (c + 4 * i);
            if (!seen || u[i] > (uint32_t)fp4::kMaxScale) u[i] = 0;
          }
        }
        const uint32_t sa = fp4::scale_pair(u[0], u[1]), sb = fp4::scale_pair(u[2], u[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x0 = h ? w[0].y : w[0].x, x1 = h ? w[1].y : w[1].x;
          const uint32_t x2 = h ? w[2].y : w[2].x, x3 = h ? w[3].y : w[3].x;
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
            for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * h + d], y0, y1, y2, y3, pb[n][0], pb[n][1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma_f16(l[n], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, pb[n][0], pb[n][1]);
        if (!inside) {
          poison |= __shfl_xor_sync(0xffffffffu, poison, 1);
          poison |= __shfl_xor_sync(0xffffffffu, poison, 2);
          for (; poison; poison &= poison - 1) {
            const int pos = p0 + __ffs((int)poison) - 1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int at = first + row_i[n][x];
                if (pos > at || (a.row_window > 0 && pos <= at - a.row_window)) continue;
#pragma unroll
                for (int d = 0; d < 8; ++d) o[n][d][x] = o[n][d][x + 2] = __uint_as_float(0x7fc00000u);
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(smem_u32(&sm.empty[st]));
    }
    ++it;

    const bool piece_end = cur.t + 1 == t1 || cur.j + 1 == cur.n;
    if (piece_end) {
      // ---- join the warps: maxima, then the outputs relative to the largest
      const bool whole = piece_first == cur.seg_base && cur.j + 1 == cur.n;
      const int64_t slot =
          piece_first == cur.seg_base ? (int64_t)cur.b * a.Hkv + cur.g : (int64_t)a.B * a.Hkv + blockIdx.x;
      if (g == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sm.m[n][warp][2 * c] = m[n][0];
          sm.m[n][warp][2 * c + 1] = m[n][1];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n && n * 8 >= R) break;
        tc::named_bar_sync(1, S::WARPS * 32);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < S::WARPS; ++i) top = fmaxf(top, sm.m[n][i][2 * c + x]);
          const float scale = m[n][x] == -INFINITY ? (l[n][x] == 0.f ? 0.f : 1.f) : exp2_approx(m[n][x] - top);
          float4* dst = reinterpret_cast<float4*>(&sm.o[warp][2 * c + x][16 * g]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_float4(o[n][2 * i][x] * scale, o[n][2 * i][x + 2] * scale,
                                 o[n][2 * i + 1][x] * scale, o[n][2 * i + 1][x + 2] * scale);
          if (g == 0) sm.l[warp][2 * c + x] = l[n][x] * scale;
        }
        tc::named_bar_sync(1, S::WARPS * 32);
        // Eight rows of 128 outputs over the consumer threads.
        constexpr int PER = 8 * D / (32 * S::WARPS);
        const int h = tid * PER / D, d = tid * PER % D, row = n * 8 + h;
        if (row < R) {
          float sum = 0.f, top = -INFINITY, acc[PER];
#pragma unroll
          for (int x = 0; x < PER; ++x) acc[x] = 0.f;
#pragma unroll
          for (int i = 0; i < S::WARPS; ++i) {
            sum += sm.l[i][h];
            top = fmaxf(top, sm.m[n][i][h]);
#pragma unroll
            for (int x = 0; x < PER; ++x) acc[x] += sm.o[i][h][d + x];
          }
          // A sum that is not a number (a NaN score) makes the row's output and lse NaN.
          const bool none = sum == 0.f;
          const float inv = none ? 0.f : 1.f / sum;
          const float lse2 = none ? -INFINITY : top + log2f(sum) - kShift;
          if (whole) {
            const int64_t at = ((int64_t)cur.b * a.q_len + row / a.n_rep) * a.H + (int64_t)cur.g * a.n_rep +
                               row % a.n_rep;
#pragma unroll
            for (int x = 0; x < PER; x += 2) {
              if (a.out_f32) {
                *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at * D + d + x) =
                    make_float2(acc[x] * inv, acc[x + 1] * inv);
              } else {
                *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at * D + d + x) =
                    __floats2bfloat162_rn(acc[x] * inv, acc[x + 1] * inv);
              }
            }
            if (a.lse && d == 0) a.lse[at] = lse2 * kLn2;
          } else {
            const int64_t at = slot * R + row;
#pragma unroll
            for (int x = 0; x < PER; x += 2)
              *reinterpret_cast<float2*>(a.ws_o + at * D + d + x) = make_float2(acc[x] * inv, acc[x + 1] * inv);
            if (d == 0) a.ws_lse[at] = lse2;
          }
        }
      }
    }
    if (!cursor_next(cur, rows, a.B, a.Hkv)) break;
  }
}

template <int NT>
cudaError_t launch_n(const DecodeArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(Smem<NT>);
  static_assert(sizeof(Smem<NT>) <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(decode_fp4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_fp4_kernel<NT>, dim3(a.num_ctas), dim3(Shape<NT>::THREADS), smem, stream, a);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeArgs& a, cudaStream_t stream) {
  const int rows = a.n_rep * a.q_len;
  if (rows <= 8) return launch_n<1>(a, stream);
  if (rows <= 16) return launch_n<2>(a, stream);
  return launch_n<4>(a, stream);
}

}  // namespace pkv
