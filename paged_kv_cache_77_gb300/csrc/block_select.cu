// Block selection for sparse decode: a summary of each block's keys, kept up to date as rows
// are written, and the choice of the blocks that a query row attends to.
//
// Summary of a block, per kv head: the smallest and the largest key value of each of the 128
// channels, [num_blocks, H_kv, 2, 128] bf16 (exact: a minimum needs no rounding). For any key
// x of the block and any query q,
//
//   q . x = sum_d q_d x_d <= sum_d (max(q_d, 0) max_d + min(q_d, 0) min_d),
//
// so the sum over the n_rep query heads h of a kv head,
//
//   score = sum_d (P_d max_d + N_d min_d),  P = sum_h max(q_h, 0), N = sum_h min(q_h, 0),
//
// bounds the sum of the group's scaled-by-nothing dot products with any key of the block, at
// 512 bytes per block and kv head in place of 32 KB of keys.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {

namespace cg = cooperative_groups;

namespace {

constexpr int kBs = 128;    // tokens per block
constexpr int kDim = 128;   // head_dim
constexpr int kSumBytes = 2 * kDim * 2;  // one (block, kv head) summary

// Minimum / maximum of two packed bf16; NaN if either is.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

// ------------------------------------------------------------------ summaries
// One group of kWarps warps per (sequence, touched block, kv head). Half a warp holds a row of
// 256 bytes (16 bytes a lane), so a warp takes two rows at a time; all of a lane's rows are
// loaded before the first comparison. The halves meet by a shuffle, the warps through shared
// memory, and the old summary joins in where the block held rows before this step.
// Roofline: HBM; 256 B per new key and kv head read, 512 B per touched block and kv head
// written, and read where the block was begun earlier.
template <int kWarps>
__global__ void __launch_bounds__(256) block_summary_kernel(const __grid_constant__ SummaryArgs a) {
  constexpr int kGroups = 8 / kWarps;            // groups of a 256-thread CTA
  constexpr int kRowsAtOnce = kWarps == 1 ? 4 : 8;  // row pairs a lane holds at a time
  __shared__ uint4 part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / kWarps, w = warp % kWarps;
  const int64_t item = (int64_t)blockIdx.x * kGroups + group;
  const int64_t items = (int64_t)a.B * a.span * a.Hkv;
  // A warp of a group past the end has no work; with several warps a group is the CTA, whose
  // grid is exact.
  if (item >= items) return;
  const int g = (int)(item % a.Hkv);
  const int64_t bs = item / a.Hkv;
  const int s = (int)(bs % a.span), b = (int)(bs / a.span);
  const int len = __ldg(a.seq_lens + b), fresh = __ldg(a.num_new + b);
  if (fresh == 0) return;
  if (fresh < 0 || fresh > a.max_new || len < fresh || (int64_t)len > (int64_t)a.max_blocks * kBs) {
    if (s == 0 && g == 0 && w == 0 && lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
    return;
  }
  const int first = len - fresh;
  const int j = first / kBs + s;
  if ((int64_t)j * kBs >= len) return;  // the step touches fewer blocks than `span`
  const int blk = __ldg(a.block_table + (int64_t)b * a.max_blocks + j);
  if (blk < 0 || (int64_t)blk >= a.num_blocks) {
    if (g == 0 && w == 0 && lane == 0) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
    return;
  }
  const int r0 = first > j * kBs ? first - j * kBs : 0;
  const int r1 = len - j * kBs < kBs ? len - j * kBs : kBs;
  const int half = lane >> 4, c = lane & 15;
  const uint8_t* base = a.k_cache + ((int64_t)blk * kBs * a.Hkv + g) * (kDim * 2) + c * 16;
  const int64_t row_bytes = (int64_t)a.Hkv * kDim * 2;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) lo[i] = 0x7f807f80u, hi[i] = 0xff80ff80u;  // +inf, -inf
  for (int r = r0 + 2 * w + half; r < r1; r += 2 * kWarps * kRowsAtOnce) {
    uint4 x[kRowsAtOnce];
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u)
      if (r + 2 * kWarps * u < r1) x[u] = ld_nc_v4(base + (int64_t)(r + 2 * kWarps * u) * row_bytes);
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u) {
      if (r + 2 * kWarps * u >= r1) continue;
      const uint32_t v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = min2(lo[i], v[i]);
        hi[i] = max2(hi[i], v[i]);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = min2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], 16));
    hi[i] = max2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], 16));
  }
  // Lanes 0-15 go on with the minima of channels 8c..8c+7, lanes 16-31 with the maxima.
  uint4 acc = half ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
  auto merge = [&](const uint4& y) {
    acc.x = half ? max2(acc.x, y.x) : min2(acc.x, y.x);
    acc.y = half ? max2(acc.y, y.y) : min2(acc.y, y.y);
    acc.z = half ? max2(acc.z, y.z) : min2(acc.z, y.z);
    acc.w = half ? max2(acc.w, y.w) : min2(acc.w, y.w);
  };
  if (kWarps > 1) {
    part[warp][lane] = acc;
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int i = 1; i < kWarps; ++i) merge(part[i][lane]);
  }
  uint4* dst = reinterpret_cast<uint4*>(a.summaries + ((int64_t)blk * a.Hkv + g) * kSumBytes) + lane;
  if (r0 > 0) merge(*dst);
  *dst = acc;
}

cudaError_t launch_block_summaries(const SummaryArgs& a, cudaStream_t stream) {
  const int64_t items = (int64_t)a.B * a.span * a.Hkv;
  if (items == 0) return cudaSuccess;
  // Few new rows per block: a warp per (block, head) reads them in one go. From 16 rows on a
  // whole CTA shares a block's rows.
  if (a.max_new <= 16)
    block_summary_kernel<1><<<(unsigned)((items + 7) / 8), 256, 0, stream>>>(a);
  else
    block_summary_kernel<8><<<(unsigned)items, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ selection
// One cluster of C CTAs per (query row, kv head): all of them score blocks, the first keeps
// the scores in its shared memory (the others store into it) and selects.
//
// Scores are taken in fp32, 512 coalesced bytes per block (lanes 0-15 hold the minima and N,
// lanes 16-31 the maxima and P, 8 channels each), 8 blocks per warp at a time whose sums are
// reduced across the lanes together. Selection needs exact order only at the border, so the
// kernel bounds the fp32 error,
//
//   |score32 - score| <= eps = 2^-18 (sum_d P_d + |N_d|) max |summary|,
//
// (at most 15 roundings in P and N, one per product and sum, 5 in the reduction: 29 of 2^-24,
// of terms whose magnitudes add up to no more than the product), takes every block above
// tau + 2 eps and none below tau - 2 eps, tau being the K-th largest fp32 score, and scores
// the blocks between again in fp64. Usually there is one, tau's own, and then nothing is left
// to decide. The result is that of fp64 scores, ties to the lower block, whatever the order of
// the fp32 sums.
//
// A block whose score is NaN (a NaN key, or infinite keys that cancel) ranks above all others.
namespace {

constexpr int kSelWarps = 8;
constexpr int kSelThreads = 32 * kSelWarps;
constexpr uint32_t kNanKey = 0xfffffffeu;

// Order-preserving whole numbers for scores; -0 and +0 are equal, NaN is the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return kNanKey;
  const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const unsigned long long u = x == 0.0 ? 0ull : (unsigned long long)__double_as_longlong(x);
  return (u >> 63) ? ~u : u | (1ull << 63);
}

struct SelShared {
  int hist[256];
  int count[kSelWarps];
  int total, digit, above, above2;
  unsigned long long prefix;
  unsigned int amax[64];  // per warp of the cluster: largest |summary| seen, bf16 bits
};

// The k-th largest of keys[0, n) (1 <= k <= n), by 8 bits at a time from the top; *greater is
// the number of keys above it. Called by the whole CTA.
template <typename Key>
__device__ Key kth_largest(const Key* keys, int n, int k, SelShared& sh, int* greater) {
  constexpr int kBits = 8 * sizeof(Key);
  Key prefix = 0;
  int rest = k;
  for (int shift = kBits - 8; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      const Key key = keys[i];
      const bool in = shift == kBits - 8 || (key >> ((shift + 8) & (kBits - 1))) == prefix;
      if (in) atomicAdd(&sh.hist[(int)(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // Lane l sums digits 8l..8l+7; the lanes above it hold the larger digits.
      const int lane = threadIdx.x;
      int own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += sh.hist[8 * lane + i];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, incl, o);
        if (lane + o < 32) incl += y;
      }
      int above = incl - own;
      if (above < rest && rest <= incl) {
        for (int d = 8 * lane + 7;; --d) {
          if (above + sh.hist[d] >= rest) {
            sh.digit = d;
            sh.above = above;
            break;
          }
          above += sh.hist[d];
        }
      }
    }
    __syncthreads();
    prefix = (Key)((prefix << 8) | (Key)sh.digit);
    rest -= sh.above;
  }
  *greater = k - rest;
  return prefix;
}

// Calls put(rank, i) for every i in [0, n) with pick(i), rank counting them in ascending
// order; returns their number. Called by the whole CTA; each warp takes one run of indices.
template <typename Pick, typename Put>
__device__ int compact(int n, SelShared& sh, Pick pick, Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i0 = warp * run, i1 = min(n, i0 + run);
  int mine = 0;
  for (int i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && pick(i + lane)));
  if (lane == 0) sh.count[warp] = mine;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int v = 0; v < kSelWarps; ++v) {
    if (v < warp) at += sh.count[v];
    all += sh.count[v];
  }
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1 && pick(i + lane);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) put(at + __popc(m & ((1u << lane) - 1)), i + lane);
    at += __popc(m);
  }
  __syncthreads();
  return all;
}

}  // namespace

__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ unsigned long long sel_smem[];
  __shared__ SelShared sh;
  __shared__ double coef64[2 * kDim];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = blockIdx.x / C;  // (query row, kv head)
  const int g = (int)(seg % a.Hkv);
  const int64_t row = seg / a.Hkv;
  const int b = (int)(row / a.q_len), qi = (int)(row % a.q_len);
  const int cap = a.max_blocks * kBs;
  const int raw = __ldg(a.seq_lens + b);
  const int len = clamp_len(raw, cap);
  if (len != raw && g == 0 && qi == 0 && rank == 0 && threadIdx.x == 0)
    flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  const int row_len = len - a.q_len + 1 + qi;
  const int n = row_len > 0 ? (row_len + kBs - 1) / kBs : 0;
  const int K = a.num_selected;
  int32_t* out = a.out + seg * K;
  // Blocks [0, e0) and [e1, n) are always taken; the others compete for `want` places.
  const int e0 = a.num_sink, e1 = n - a.num_recent;
  const int want = K - a.num_sink - a.num_recent;
  if (n <= K || want == 0) {
    if (rank == 0)
      for (int i = threadIdx.x; i < K; i += kSelThreads)
        out[i] = n <= K ? (i < n ? i : -1) : (i < e0 ? i : e1 + (i - e0));
    return;  // the whole cluster takes this way
  }
  const int m = e1 - e0;  // > want
  unsigned long long* key64 = sel_smem;                                  // [max_blocks]
  uint32_t* key32 = reinterpret_cast<uint32_t*>(sel_smem + a.max_blocks);  // [max_blocks]
  uint32_t* key32_0 = cluster.map_shared_rank(key32, 0);
  unsigned int* amax_0 = cluster.map_shared_rank(sh.amax, 0);
  cluster.sync();  // the first CTA's shared memory may be stored into from here on

  // ---- fp32 scores
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  const int half = lane >> 4, c = lane & 15;
  const uint16_t* q = a.q + (row * a.H + (int64_t)g * a.n_rep) * kDim;
  float coef[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint32_t q_bits = 0;
  for (int h = 0; h < a.n_rep; ++h) {
    const uint4 x = ld_nc_v4(q + h * kDim + 8 * c);
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q_bits |= v[i] & 0x7fff7fffu;
      const float lo = bf16lo(v[i]), hi = bf16hi(v[i]);
      // A NaN goes into both sums (a maximum or minimum would drop it).
      coef[2 * i] = add_ieee(coef[2 * i], lo != lo ? lo : half ? max_ieee(lo, 0.f) : min_ieee(lo, 0.f));
      coef[2 * i + 1] =
          add_ieee(coef[2 * i + 1], hi != hi ? hi : half ? max_ieee(hi, 0.f) : min_ieee(hi, 0.f));
    }
  }
  uint32_t vmax = 0;  // two 16-bit maxima of |summary| as bits: NaN above infinity above all
  const uint8_t* sum0 = a.summaries + (int64_t)g * kSumBytes + lane * 16;
  const int64_t sum_stride = (int64_t)a.Hkv * kSumBytes;
  for (int j0 = (rank * kSelWarps + warp) * 8; j0 < m; j0 += C * kSelWarps * 8) {
    int blk = -1;
    if (lane < 8 && j0 + lane < m) {
      blk = __ldg(table + e0 + j0 + lane);
      if (blk < 0 || (int64_t)blk >= a.num_blocks) {
        blk = -1;
        flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
      }
    }
    uint4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int p = __shfl_sync(0xffffffffu, blk, u);
      x[u] = p >= 0 ? ld_nc_v4(sum0 + p * sum_stride) : make_uint4(0, 0, 0, 0);
    }
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fma_ieee(coef[2 * i], bf16lo(w[i]), s);
        s = fma_ieee(coef[2 * i + 1], bf16hi(w[i]), s);
        vmax = __vmaxu2(vmax, w[i] & 0x7fff7fffu);
      }
      v[u] = s;
    }
    // Sums over the 32 lanes of all 8 at once: each step halves the blocks a lane holds.
#pragma unroll
    for (int o = 16, k = 4; o >= 4; o >>= 1, k >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= k) continue;
        const float send = up ? v[i] : v[i + k];
        const float keep = up ? v[i + k] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
    const int u = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
    const bool bad = __shfl_sync(0xffffffffu, blk, u) < 0;
    if ((lane & 3) == 0 && j0 + u < m) key32_0[j0 + u] = bad ? 0u : order_key(v[0]);
  }
  {
    const uint32_t one = max(vmax & 0xffffu, vmax >> 16);
    const uint32_t all = __reduce_max_sync(0xffffffffu, one);
    if (lane == 0) amax_0[rank * kSelWarps + warp] = all;
  }
  cluster.sync();
  if (rank) return;

  // ---- the border
  // sum_d P_d + |N_d| over the warp's 32 lanes, the same in every warp.
  float size = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) size = add_ieee(size, fabsf(coef[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) size = add_ieee(size, __shfl_xor_sync(0xffffffffu, size, o));
  uint32_t top = 0;
  for (int i = lane; i < C * kSelWarps; i += 32) top = max(top, sh.amax[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  const float reach = mul_ieee(size, __uint_as_float(top << 16));  // bounds |score|, partial sums
  const bool q_zero = __reduce_or_sync(0xffffffffu, q_bits) == 0;
  int greater;
  const uint32_t tau = kth_largest(key32, m, want, sh, &greater);
  // Keys above `sure` are in, keys below `maybe` are out.
  uint32_t maybe = 0, sure = kNanKey;
  if (q_zero && reach == 0.f) {
    maybe = sure = tau;  // every finite score is an exact zero
  } else if (reach < 1e37f && tau != 0) {
    // The added constant covers sums flushed to zero. (A reach that is not finite bounds
    // nothing, and a tau of 0 is a bad block's key, not a score: every block is scored again.)
    const float eps = reach * 0x1p-18f + 1e-35f;
    const float x = __uint_as_float((tau & 0x80000000u) ? tau & 0x7fffffffu : ~tau);
    // Rounded outward: one more unit of 2^-23 of the larger operand.
    const float pad = 2.f * eps + (fabsf(x) + 2.f * eps) * 0x1p-22f;
    maybe = order_key(x - pad);
    sure = order_key(x + pad);
  }
  __shared__ int n_sure, n_maybe;
  if (threadIdx.x == 0) n_sure = n_maybe = 0;
  __syncthreads();
  {
    int s = 0, t = 0;
    for (int i = threadIdx.x; i < m; i += kSelThreads) {
      s += key32[i] > sure;
      t += key32[i] >= maybe;
    }
    s = __reduce_add_sync(0xffffffffu, s);
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) {
      atomicAdd(&n_sure, s);
      atomicAdd(&n_maybe, t);
    }
  }
  __syncthreads();
  uint32_t pass = maybe;  // keys from here on are taken
  if (n_maybe > want) {
    // More blocks in reach of the border than places: score them in fp64.
    const int need = want - n_sure;
    uint32_t* cand = reinterpret_cast<uint32_t*>(key64 + a.max_blocks) + a.max_blocks;
    const int nc = compact(
        m, sh, [&](int i) { return key32[i] >= maybe && key32[i] <= sure; },
        [&](int r, int i) { cand[r] = i; });
    for (int d = threadIdx.x; d < 2 * kDim; d += kSelThreads) {
      double s = 0.0;
      for (int h = 0; h < a.n_rep; ++h) {
        const uint32_t bits = q[h * kDim + d % kDim];
        const double x = widen_ieee(__uint_as_float(bits << 16));
        s += x != x ? x : d < kDim ? (x < 0.0 ? x : 0.0) : (x > 0.0 ? x : 0.0);
      }
      coef64[d] = s;
    }
    __syncthreads();
    for (int r = warp; r < nc; r += kSelWarps) {
      const int blk = __ldg(table + e0 + cand[r]);
      unsigned long long key = 0;  // a bad block's
      if (blk >= 0 && (int64_t)blk < a.num_blocks) {
        const uint4 x = ld_nc_v4(sum0 + blk * sum_stride);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = fma(coef64[8 * lane + 2 * i], widen_ieee(bf16lo(w[i])), s);
          s = fma(coef64[8 * lane + 2 * i + 1], widen_ieee(bf16hi(w[i])), s);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        key = order_key(s);
      }
      if (lane == 0) key64[r] = key;
    }
    __syncthreads();
    int above;
    const unsigned long long edge = kth_largest(key64, nc, need, sh, &above);
    // Above the edge: in. At the edge: the lower blocks, as many as there are places.
    for (int r = threadIdx.x; r < nc; r += kSelThreads) key32[cand[r]] = key64[r] > edge ? 0xffffffffu : 0u;
    __syncthreads();
    compact(
        nc, sh, [&](int r) { return key64[r] == edge; },
        [&](int k, int r) { if (k < need - above) key32[cand[r]] = 0xffffffffu; });
    pass = sure + 1;
  }
  for (int i = threadIdx.x; i < e0; i += kSelThreads) out[i] = i;
  compact(
      m, sh, [&](int i) { return key32[i] >= pass; }, [&](int r, int i) { out[e0 + r] = e0 + i; });
  for (int i = threadIdx.x; i < a.num_recent; i += kSelThreads) out[e0 + want + i] = e1 + i;
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t segs = (int64_t)a.B * a.q_len * a.Hkv;
  if (segs == 0) return cudaSuccess;
  // A cluster is as wide as it takes to give every SM two CTAs, as long as each of its CTAs
  // has a round of 64 blocks to score.
  int C = 1;
  while (C < 8 && segs * C < 2 * num_sms && a.max_blocks > C * kSelWarps * 8) C *= 2;
  const size_t smem = (size_t)a.max_blocks * 16;  // fp64 keys, fp32 keys, candidates
  cudaError_t e = cudaFuncSetAttribute(select_blocks_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_blocks_kernel, a);
}

}  // namespace pkv
