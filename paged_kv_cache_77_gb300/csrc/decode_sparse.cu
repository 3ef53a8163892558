// Decode over selected blocks on the tcgen05 decode kernel (decode_tc.cuh): every query row
// and kv head brings a list of blocks of its sequence and attends to the visible tokens in
// them. Rows are independent, so q_len rows of a sequence are q_len rows of the kernel. With
// rows in the thousands the merge cannot search the whole tile list once per row, as the dense
// one does: it starts from the cuts instead.
//
// Bound by HBM, as the dense kernel: 64 KB per listed (block, kv head). Measured on GB300: 512
// rows x 32 blocks of 64 long sequences (0.99 GB) 159.7 us, 92 % of the copy rate; 64 rows x 4
// blocks (17 MB) 16 us a call, host time and latency; 8,192 query rows x 8 kv heads x 2 blocks
// 1.5 ms (6.5 ms with the dense merge and a seek by one thread).
#include "decode_tc.cuh"

namespace pkv {

// Joins the pieces of the segments that the split cut, one block per CTA of the attention
// kernel: block i looks at the tile its CTA's range starts with, and if that is the first cut
// of a segment, merges all of the segment's pieces, a warp per query head (log-sum-exp
// weights, a lane 4 consecutive output elements). Rows without a block get o = 0, lse = -inf,
// spread over the blocks. The search reads only the call's inputs and overlaps the attention.
// Roofline: HBM (latency); the cut segments' partials.
__global__ void __launch_bounds__(512) sparse_merge_kernel(const __grid_constant__ DecodeArgs a) {
  using tcd::BS;
  using tcd::D;
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SparseRows rows = {a.seq_lens, BS, a.rows_per_seq, a.num_selected, a.max_blocks * BS};
  const int64_t G = a.num_ctas, i = blockIdx.x;
  const int64_t T = total_live_blocks(rows, a.B, nullptr) * a.Hkv;
  const int64_t t0 = cta_tile_start(i, T, G);
  TileCursor c;
  cursor_seek_warp(c, rows, a.B, a.Hkv, t0, cta_tile_start(i + 1, T, G));
  // The first CTA of the segment, which ends at this cut if the cut is the segment's first.
  const bool cut = c.b < a.B && c.seg_base < t0;  // (no tile at all: c.b = B)
  const int64_t i0 = cut ? cta_of_tile(c.seg_base, T, G) : 0;
  const bool first_cut = cut && cta_tile_start(i0 + 1, T, G) == t0;
  const int64_t i1 = first_cut ? cta_of_tile(c.seg_base + c.n - 1, T, G) : 0;
  auto put = [&](int64_t row, float4 v, float lse) {
    if (a.out_f32) {
      reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * D)[lane] = v;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * D)[lane] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (a.lse && lane == 0) a.lse[row] = lse;
  };
  pdl_wait_primary();
  for (int64_t r = i; r < a.B; r += G) {
    if (rows.len((int)r)) continue;
    for (int x = h; x < a.H; x += a.n_rep) put(r * a.H + x, make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY);
  }
  if (!first_cut) return;
  // Weights relative to the largest of all pieces' log-sum-exps, added in the pieces' order:
  // the same sums as the dense merge's.
  auto partial = [&](int64_t p) -> int64_t {  // row of the workspace, -1: a CTA without a tile
    if (p > i1 || (p > i0 && cta_tile_start(p + 1, T, G) == cta_tile_start(p, T, G))) return -1;
    return (p == i0 ? (int64_t)c.b * a.Hkv + c.g : (int64_t)a.B * a.Hkv + p) * a.n_rep + h;
  };
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAtOnce = 8;  // pieces whose loads are in flight together
  if (i1 - i0 >= kAtOnce)
    for (int64_t p = i0; p <= i1; ++p)
      if (partial(p) >= 0) top = fmaxf(top, a.ws_lse[partial(p)]);
  for (int64_t p0 = i0; p0 <= i1; p0 += kAtOnce) {
    float l2[kAtOnce];
    float4 x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t at = partial(p0 + u);
      l2[u] = at >= 0 ? a.ws_lse[at] : -INFINITY;
      x[u] = at >= 0 ? reinterpret_cast<const float4*>(a.ws_o + at * D)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, l2[u]);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const float w = l2[u] == -INFINITY ? 0.f : exp2f(l2[u] - top);
      acc.x += w * x[u].x;
      acc.y += w * x[u].y;
      acc.z += w * x[u].z;
      acc.w += w * x[u].w;
      sum += w;
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;  // (a NaN piece makes the row NaN)
  put((int64_t)c.b * a.H + (int64_t)c.g * a.n_rep + h,
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv),
      sum != 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY);
}

static cudaError_t launch_attention(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.n_rep) {
    case 1: return launch_tc_n<1, 1, true>(a, stream);
    case 2: return launch_tc_n<2, 1, true>(a, stream);
    case 4: return launch_tc_n<4, 1, true>(a, stream);
    case 8: return launch_tc_n<8, 1, true>(a, stream);
    case 16: return launch_tc_n<16, 1, true>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode_sparse(const DecodeArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_attention(a, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(sparse_merge_kernel, dim3(a.num_ctas), dim3(32 * a.n_rep), 0, stream, a);
}

}  // namespace pkv
