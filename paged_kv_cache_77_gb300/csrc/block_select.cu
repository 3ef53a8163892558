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
#include "ieee_math.cuh"
#include "launch.h"
#include "pdl.cuh"

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

// Largest magnitudes, NaN if either is; the sign bits of the result mean nothing.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

// ------------------------------------------------------------------ summaries
// One group of kWarps warps per (sequence, touched block, kv head). Half a warp holds a row of
// 256 bytes (16 bytes a lane), so a warp takes two rows at a time, and a lane has several loads
// in flight. The halves meet by a shuffle, the warps through shared memory, and the old summary
// joins in where the block held rows before this step.
// Roofline: HBM; 256 B per new key and kv head read, 512 B per touched block and kv head
// written, and read where the block was begun earlier.
template <int kWarps>
__global__ void __launch_bounds__(256, kWarps == 1 ? 4 : 8)
    block_summary_kernel(const __grid_constant__ SummaryArgs a) {
  constexpr int kGroups = 8 / kWarps;            // groups of a 256-thread CTA
  // Rows a lane holds at a time. Prefill chunks of 16 sequences (127 MB), a warp per item: 8 rows
  // and four resident CTAs per SM 20.2 us (GB300, 93 % of the copy rate), 8 and three 22.6, 4 and
  // four 20.5, 4 and six 23.2. A CTA per item: 4 and eight 22.0, 4 and six 23.3, 8 and five 23.5,
  // 2 and eight 23.7.
  constexpr int kRowsAtOnce = kWarps == 1 ? 8 : 4;
  __shared__ uint4 part[8][32];
  pdl_wait_then_launch();
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
    // A row past the end repeats the last one: it changes neither bound, and without a branch
    // around them the loads are in flight together.
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u)
      x[u] = ld_nc_v4(base + (int64_t)min(r + 2 * kWarps * u, r1 - 1) * row_bytes);
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u) {
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

cudaError_t launch_block_summaries(const SummaryArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t items = (int64_t)a.B * a.span * a.Hkv;
  if (items == 0) return cudaSuccess;
  // A warp per item, unless whole blocks come in fewer than 4 items per SM: then the eight warps
  // of a CTA share one. Measured with 8 kv heads (us, warp and CTA): one sequence of 1,024 new
  // rows (72 items) 4.1 and 2.9, of 8,192 (520 items) 4.3 and 3.9; 64 sequences of 64 (1,024
  // items) 3.5 and 4.9, 512 of 64 11.0 and 19.3, 16 of 8,192 37.5 and 39.1; 16 sequences of 16,
  // which leave most of a CTA's warps without a row, 2.6 and 3.0.
  if (a.max_new <= 16 || items >= 4 * (int64_t)num_sms)
    return launch_dependent(block_summary_kernel<1>, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, a);
  return launch_dependent(block_summary_kernel<8>, dim3((unsigned)items), dim3(256), 0, stream, a);
}

// ------------------------------------------------------------------ selection
// One cluster of C CTAs per (query row, kv head). Each CTA scores one run of the row's blocks
// and keeps their keys (order-preserving whole numbers) in its shared memory. A row of at most
// 256 competing blocks is one CTA's, and is selected by one warp with the keys in registers;
// of longer ones all keys go to the shared memory of the cluster's first CTA, which selects with
// the keys in registers. Only where many blocks are at the border the CTAs select together,
// exchanging histograms and counts through distributed shared memory.
//
// Scores are taken in fp32, 512 coalesced bytes per block (lanes 0-15 hold the minima and N,
// lanes 16-31 the maxima and P, 8 channels each), 8 blocks per warp at a time whose sums are
// reduced across the lanes together. Selection needs exact order only at the border, so the
// kernel bounds the fp32 error,
//
//   |score32 - score| <= eps = 14 2^-24 (sum_d P_d + |N_d|) max |summary|
//
// (one rounding in P and N, 5 in a lane's sum of products, 5 in the reduction, and room for
// the bound's own), finds the K-th largest fp32 score tau to within a bin narrower
// than eps, takes every block above the bin by more than 2 eps and none below it by more, and
// scores the blocks between again where they are more than the places left: few of them in pairs
// of fp32 numbers, and in fp64 where those do not tell them apart. The result is that of fp64
// scores, ties to the lower block, whatever the order of the fp32 sums.
//
// A block whose score is NaN (a NaN key, or infinite keys that cancel) ranks above all others.
namespace {

constexpr int kSelWarps = 8;
constexpr int kSelThreads = 32 * kSelWarps;
constexpr int kMaxCluster = 8;
constexpr int kMaxChunk = 4096;           // blocks whose keys a CTA holds, 64 KB
static_assert(kSelectMaxBlocks <= kMaxCluster * kMaxChunk, "a row's keys fit its cluster");
constexpr int kDigitBits = 9;             // two digits of this size decide most 32-bit searches
constexpr int kDigits = 1 << kDigitBits;  // two per thread
constexpr int kWarpKeys = 8;              // keys of a lane where one warp selects
constexpr uint32_t kNanKey = 0xfffffffeu;
constexpr uint32_t kTaken = 0xffffffffu;  // above every score's key
constexpr uint32_t kEdge = kNanKey;       // candidates at the border, once no key is a NaN's

// Order-preserving whole numbers for scores; -0 and +0 are equal, NaN is the largest. Key 0
// stands for a block whose table entry is bad.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return kNanKey;
  const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return ~0ull;
  const unsigned long long u = x == 0.0 ? 0ull : (unsigned long long)__double_as_longlong(x);
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What decides a row: keys above `sure` are in, keys below `maybe` are out, and of those between
// the `need` best by more exact scores.
struct Border {
  uint32_t maybe, sure;
  int need, settled;
};

// Digit counts: 4 passes over 32-bit keys, 8 over 64.
using Hist = int[4 + 8][kDigits];

// Shared memory of one CTA. What other CTAs of the cluster read (counts, pub, the keys) is
// written once per kernel and place, so one cluster barrier between the writes and the reads
// is enough.
struct SelShared {
  float coef[2 * kDim], coef_low[2 * kDim];  // N, then P: their fp32 sums and what those left out
  unsigned long long pub[4][2];          // a pair of numbers per exchange
  unsigned long long lo[kSelWarps], hi[kSelWarps];
  float size[kSelWarps];
  uint32_t any_q[kSelWarps], amax[kSelWarps];
  int warp_sum[kSelWarps], warp_sum2[kSelWarps];
  int digit, above, inside, candidates, done;
  uint32_t few[32], best;                // a single CTA's candidates, and which are taken
  unsigned long long few64[32];          // their keys
  Border border;
  uint32_t range[kMaxCluster][3];        // smallest and largest key and largest |summary| of each CTA
};

struct Cluster {
  int size, rank;
  __device__ __forceinline__ void sync() const {
    if (size > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  }
  template <typename T>
  __device__ __forceinline__ T read(T* mine, int r) const {
    return r == rank ? *mine : *cg::this_cluster().map_shared_rank(mine, r);
  }
};

// Where a row's blocks lie and what bounds their scores.
struct Row {
  const int32_t* table;  // of the CTA's first block
  const uint8_t* sum;    // the lane's 16 bytes of block 0's summary
  int64_t sum_stride, num_blocks;
  float eps;             // bound of a score's fp32 error
  bool bounded;          // eps is one
  bool exact;            // every good block's score is exactly zero
};

// An fp32 value as a double from its bits (conversions run at the rate of the fp64 units): the
// exponent's bias moves from 127 to 1023. Subnormals, infinities and NaN are converted.
__device__ __forceinline__ double widen_bits(uint32_t bits) {
  if ((bits & 0x7f800000u) - 0x00800000u < 0x7f000000u)
    return __hiloint2double((int)((bits & 0x80000000u) | (((bits & 0x7fffffffu) >> 3) + (896u << 20))),
                            (int)(bits << 29));
  return (bits & 0x7fffffffu) ? widen_ieee(__uint_as_float(bits)) : 0.0;
}

// Keys of up to 4 candidates in fp64, by a warp; key64[r] for the blocks cand[r]. An fp64
// operation of a warp costs some 70 to 90 cycles here, so there are few: 8 additions for the
// coefficients and 16 operations a candidate, no conversions (a smaller version with
// conversions, always four candidates, took 9.7k cycles instead of 6k).
__device__ void score64(const Row& row, const SelShared& sh, const uint32_t* cand,
                        unsigned long long* key64, int n) {
  const int lane = threadIdx.x & 31;
  uint4 x[4];
  bool good[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int blk = r < n ? __ldg(row.table + cand[r]) : -1;
    good[r] = blk >= 0 && (int64_t)blk < row.num_blocks;
    x[r] = good[r] ? ld_nc_v4(row.sum + blk * row.sum_stride) : make_uint4(0, 0, 0, 0);
  }
  double k[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    k[i] = widen_bits(__float_as_uint(sh.coef[8 * lane + i])) +
           widen_bits(__float_as_uint(sh.coef_low[8 * lane + i]));
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r >= n) break;
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    double s[4];  // short chains: an fp64 operation takes long
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s[i] = fma(k[2 * i], widen_bits(w[i] << 16), k[2 * i + 1] * widen_bits(w[i] & 0xffff0000u));
    s[0] = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    if (lane == 0) key64[r] = good[r] ? order_key(s[0]) : 0ull;
  }
}

// The same in pairs of fp32 numbers: a sum and, beside it, what its roundings left out (Knuth's
// two-sum, and a product's error by a fused multiply-add). With `reach` what bounds a score and
// its partial sums, the second numbers of a level of the 13 additions are below 15 2^-24 reach in
// all and rounded twice a level: the result is off by less than 2^-39 reach. In fp32 arithmetic
// four candidates take a tenth of the time that they take in fp64.
// A key is the order key of the rounded sum, then that of the rest.
__device__ void score_pairs(const Row& row, const SelShared& sh, const uint32_t* cand,
                            unsigned long long* keys, int n) {
  // Eight lanes a candidate, 32 channels a lane. One loop of 8 channels: unrolled over all of
  // them the code's fetch costs more than the loop.
  const int lane = threadIdx.x & 31, r = lane >> 3, sub = lane & 7;
  const int blk = r < n ? __ldg(row.table + cand[r]) : -1;
  const bool good = blk >= 0 && (int64_t)blk < row.num_blocks;
  const uint8_t* at = row.sum + (good ? blk : 0) * row.sum_stride + (sub - lane) * 16;
  uint4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = ld_nc_v4(at + k * 128);
  float s = 0.f, rest = 0.f;
  auto add = [](float& s, float& rest, float p, float e) {
    const float sum = add_ieee(s, p);
    const float back = sub_ieee(sum, s);
    const float lost = add_ieee(sub_ieee(s, sub_ieee(sum, back)), sub_ieee(p, back));
    rest = add_ieee(rest, add_ieee(lost, e));
    s = sum;
  };
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const float* c = sh.coef + 8 * (sub + 8 * k);
    const float* low = sh.coef_low + 8 * (sub + 8 * k);
    const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      const float p = mul_ieee(c[i], v);
      add(s, rest, p, fma_ieee(low[i], v, fma_ieee(c[i], v, neg_ieee(p))));
    }
    x[0] = x[1], x[1] = x[2], x[2] = x[3];
  }
#pragma unroll
  for (int o = 4; o; o >>= 1)
    add(s, rest, __shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, rest, o));
  float low = 0.f;
  add(s, low, rest, 0.f);
  if (sub == 0 && r < n)
    keys[r] = good ? (unsigned long long)order_key(s) << 32 | order_key(low) : 0ull;
}

// Keys that decide: exact zeros as they are, the others in fp64.
__device__ __forceinline__ void exact_keys(const Row& row, const SelShared& sh, const uint32_t* key32,
                                           const uint32_t* cand, unsigned long long* key64, int n) {
  const int lane = threadIdx.x & 31;
  if (!row.exact)
    score64(row, sh, cand, key64, n);
  else if (lane < n)
    key64[lane] = key32[cand[lane]];
}

// Up to 32 candidates, those of lanes [0, n): the rank of a lane's, those above it and those equal
// to it at lower places counted; 32 in the other lanes.
__device__ int rank_in_warp(unsigned long long mine, uint32_t place, int n) {
  int rank = (threadIdx.x & 31) < n ? 0 : 32;
  for (int s = 0; s < n; ++s) {
    const unsigned long long other = __shfl_sync(0xffffffffu, mine, s);
    const uint32_t where = __shfl_sync(0xffffffffu, place, s);
    rank += other > mine || (other == mine && where < place);
  }
  return rank;
}

// Whether the best `need` of the lanes' candidates are theirs by more than the pairs' errors.
// (A bad block's key 0 is a NaN here, and decides nothing; nor do sums near the subnormals,
// which order_key takes for zero.)
__device__ bool decided(const Row& row, unsigned long long mine, int rank, int need) {
  const unsigned last = __ballot_sync(0xffffffffu, rank == need - 1);
  const unsigned next = __ballot_sync(0xffffffffu, rank == need);
  const unsigned long long a = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1);
  const unsigned long long b = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
  const float gap = (key_score((uint32_t)(a >> 32)) - key_score((uint32_t)(b >> 32))) +
                    (key_score((uint32_t)a) - key_score((uint32_t)b));
  return gap > row.eps * 0x1p-13f + 1e-37f;  // eps is 14 2^-24 of the bound
}

// Low bits of the keys that need not be decided: a bin of 2^bits keys in [kmin, kmax] is
// narrower than eps, for its scores are at most the largest magnitude's 2^-23 apart.
__device__ __forceinline__ int spare_bits(const Row& row, uint32_t kmin, uint32_t kmax) {
  if (kmin == 0 || row.exact) return 0;  // bad blocks among them
  const uint32_t top = __float_as_uint(fmaxf(fabsf(key_score(kmin)), fabsf(key_score(kmax)))) >> 23;
  const int bits = (int)(__float_as_uint(row.eps) >> 23) - ((int)top - 23);
  return min(max(bits, 0), 31);
}

// [maybe, sure] from the bin [lo, hi] that holds the K-th largest key.
__device__ __forceinline__ void border(const Row& row, uint32_t lo, uint32_t hi, uint32_t* maybe,
                                       uint32_t* sure) {
  *maybe = 0;
  *sure = kNanKey;
  if (row.exact) {
    *maybe = *sure = lo;
  } else if (row.bounded && lo != 0) {  // lo = 0: bad blocks are at the border
    const float a = key_score(lo), b = key_score(hi);
    // Rounded outward: a few units of 2^-24 of the operands.
    *maybe = order_key(a - (2.f * row.eps + (fabsf(a) + row.eps) * 0x1p-22f));
    *sure = order_key(b + (2.f * row.eps + (fabsf(b) + row.eps) * 0x1p-22f));
  }
}

// Selection by one warp: the `want` best of the m <= 256 blocks with keys key32[0, m), in
// ascending order, to out[i] = first + block. Lane l holds blocks l, l + 32, ...: counting the
// keys from a threshold on takes 8 comparisons and a warp sum, so the K-th largest is found two
// bits at a time, from the highest in which the keys differ down to a bin narrower than eps.
__device__ void select_by_warp(const Row& row, SelShared& sh, const uint32_t* key32,
                               unsigned long long* key64, uint32_t* cand, int m, int want, int first,
                               int32_t* out) {
  const int lane = threadIdx.x & 31;
  uint32_t k[kWarpKeys];
  uint32_t kmin = 0xffffffffu, kmax = 0;
#pragma unroll
  for (int u = 0; u < kWarpKeys; ++u) {
    const int i = lane + 32 * u;
    k[u] = i < m ? key32[i] : 0u;
    kmin = min(kmin, i < m ? k[u] : 0xffffffffu);
    kmax = max(kmax, k[u]);
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  uint32_t lo = kmin, hi = kmin, maybe, sure;
  if (kmin != kmax && row.bounded) {
    // Two bits a step: keys from each of three thresholds on are counted in the fields of one
    // word (a count is at most 256).
    const int spare = spare_bits(row, kmin, kmax);
    int bits = 32 - __clz((int)(kmin ^ kmax));  // undecided bits
    bits += bits & 1;
    lo = bits < 32 ? kmin & ~((1u << bits) - 1) : 0u;
    do {
      bits -= 2;
      uint32_t c = 0;
#pragma unroll
      for (int u = 0; u < kWarpKeys; ++u)
        c += (k[u] >= (lo | (1u << bits))) + ((k[u] >= (lo | (2u << bits))) << 10) +
             ((k[u] >= (lo | (3u << bits))) << 20);
      c = __reduce_add_sync(0xffffffffu, c);
      const uint32_t digit = (c >> 20) >= (uint32_t)want             ? 3
                             : ((c >> 10) & 1023u) >= (uint32_t)want ? 2
                             : (c & 1023u) >= (uint32_t)want         ? 1
                                                                     : 0;
      lo |= digit << bits;
      if (digit && (c >> (10 * digit - 10) & 1023u) == (uint32_t)want) {
        // The keys from lo on are as many as wanted: the least of them is the one looked for.
        uint32_t least = 0xffffffffu;
#pragma unroll
        for (int u = 0; u < kWarpKeys; ++u) least = k[u] >= lo ? min(least, k[u]) : least;
        lo = __reduce_min_sync(0xffffffffu, least);
        bits = 0;
        break;
      }
    } while (bits > spare);
    hi = lo | ((1u << bits) - 1);
  }
  border(row, lo, hi, &maybe, &sure);
  uint32_t pass = maybe;
  // (Keys behind the row's end are 0: they count only where bad blocks do.)
  int in = 0, surely = 0;
#pragma unroll
  for (int u = 0; u < kWarpKeys; ++u) {
    in += lane + 32 * u < m && k[u] >= maybe;
    surely += k[u] > sure;
  }
  in = __reduce_add_sync(0xffffffffu, in);
  if (in > want) {
    const int need = want - (int)__reduce_add_sync(0xffffffffu, surely);
    int nc = 0;
#pragma unroll
    for (int u = 0; u < kWarpKeys; ++u) {
      const bool c = lane + 32 * u < m && k[u] >= maybe && k[u] <= sure;
      const unsigned mask = __ballot_sync(0xffffffffu, c);
      if (c) cand[nc + __popc(mask & ((1u << lane) - 1))] = lane + 32 * u;
      nc += __popc(mask);
    }
    __syncwarp();
    bool done = false;
    if (nc <= 32 && row.bounded && !row.exact) {
      for (int r = 0; r < nc; r += 4) score_pairs(row, sh, cand + r, key64 + r, min(4, nc - r));
      __syncwarp();
      const unsigned long long mine = lane < nc ? key64[lane] : 0;
      const int rank = rank_in_warp(mine, lane, nc);
      done = decided(row, mine, rank, need);
      if (done && lane < nc) cand[lane] |= rank < need ? 0x80000000u : 0u;
      __syncwarp();
    }
    if (!done) {
      for (int r = 0; r < nc; r += 4) exact_keys(row, sh, key32, cand + r, key64 + r, min(4, nc - r));
      __syncwarp();
      // A candidate's rank: those above it, and those equal to it in lower blocks.
#pragma unroll 1
      for (int u = 0; u < kWarpKeys; ++u) {
        if (32 * u >= nc) break;
        const int r = lane + 32 * u;
        const unsigned long long mine = r < nc ? key64[r] : 0;
        int rank = 0;
        for (int s = 0; s < nc; ++s) {
          const unsigned long long other = key64[s];
          rank += other > mine || (other == mine && s < r);
        }
        if (r < nc) cand[r] |= rank < need ? 0x80000000u : 0u;
      }
    }
    __syncwarp();
    // Back to the lanes that hold the keys; the r-th candidate in ascending order is cand[r].
    int at = 0;
#pragma unroll
    for (int u = 0; u < kWarpKeys; ++u) {
      const bool c = lane + 32 * u < m && k[u] >= maybe && k[u] <= sure;
      const unsigned mask = __ballot_sync(0xffffffffu, c);
      if (c) k[u] = (cand[at + __popc(mask & ((1u << lane) - 1))] >> 31) ? kTaken : 0u;
      at += __popc(mask);
    }
    pass = sure + 1;
  }
  int at = 0;
#pragma unroll
  for (int u = 0; u < kWarpKeys; ++u) {
    const bool c = lane + 32 * u < m && k[u] >= pass;
    const unsigned mask = __ballot_sync(0xffffffffu, c);
    if (c) out[at + __popc(mask & ((1u << lane) - 1))] = first + lane + 32 * u;
    at += __popc(mask);
  }
}

// What a search for the k-th largest key found: it lies in [lo, hi], a bin of `inside` keys,
// below `above` others.
template <typename Key>
struct Bin {
  Key lo, hi;
  int above, inside;
};

// The k-th largest of the cluster's keys (each(f) calls f for this thread's; all are in [kmin,
// kmax]) to within a bin of 2^spare values, or one that `done` accepts, by 9 bits at a time below
// the bits they share. Every pass counts digits in its own histogram hist[pass], zero beforehand.
template <typename Key, typename Each, typename Done>
__device__ Bin<Key> kth_largest(Each each, int k, Key kmin, Key kmax, int spare, int (*hist)[kDigits],
                                SelShared& sh, const Cluster& cl, Done done) {
  Bin<Key> b = {kmin, kmax, 0, 0};
  if (kmin == kmax) return b;
  const int top = 8 * (int)sizeof(Key) - 1 -
                  (sizeof(Key) == 8 ? __clzll((long long)(kmin ^ kmax)) : __clz((int)(kmin ^ kmax)));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int pass = 0, high = top;; ++pass) {
    const int shift = high >= kDigitBits ? high - kDigitBits + 1 : 0;  // digit: bits [shift, high]
    const Key mask = (Key)((1u << (high - shift + 1)) - 1);
    each([&](Key key) {
      if (key >= b.lo && key <= b.hi) atomicAdd(&hist[pass][(int)((key >> shift) & mask)], 1);
    });
    cl.sync();
    // Thread t holds digits 511 - 2t and 510 - 2t, so that a prefix sum counts the larger ones.
    int upper = 0, lower = 0;
    const int d = kDigits - 2 - 2 * threadIdx.x;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {  // all reads at once
      if (r >= cl.size) continue;
      const int2 two = cl.read(reinterpret_cast<int2*>(&hist[pass][d]), r);
      lower += two.x;
      upper += two.y;
    }
    const int own = upper + lower;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    int before = b.above + incl - own;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) before += w < warp ? sh.warp_sum[w] : 0;
    if (before < k && k <= before + own) {  // one thread
      const bool up = k <= before + upper;
      sh.digit = d + up;
      sh.above = up ? before : before + upper;
      sh.inside = up ? upper : lower;
    }
    __syncthreads();
    const Key base = (b.lo & ~((mask << shift) | (((Key)1 << shift) - 1))) | ((Key)sh.digit << shift);
    b.lo = base;
    b.hi = base | (((Key)1 << shift) - 1);
    b.above = sh.above;
    b.inside = sh.inside;
    if (shift <= spare || done(b)) return b;
    high = shift - 1;
  }
}

// Sums of a and c over the CTA's threads and, for the CTAs of the cluster, the sums of a over
// those before this one and of both over all. `slot`: this exchange's place in sh.pub.
struct Counted {
  int before_a, all_a, all_c;
};
__device__ Counted count_cluster(int a, int c, int slot, SelShared& sh, const Cluster& cl) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  a = __reduce_add_sync(0xffffffffu, a);
  c = __reduce_add_sync(0xffffffffu, c);
  if (lane == 0) {
    sh.warp_sum[warp] = a;
    sh.warp_sum2[warp] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long sa = 0, sc = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      sa += sh.warp_sum[w];
      sc += sh.warp_sum2[w];
    }
    sh.pub[slot][0] = sa;
    sh.pub[slot][1] = sc;
  }
  cl.sync();
  // Lane r reads CTA r's pair.
  const int x = lane < cl.size ? (int)cl.read(&sh.pub[slot][0], lane) : 0;
  const int y = lane < cl.size ? (int)cl.read(&sh.pub[slot][1], lane) : 0;
  Counted t;
  t.before_a = __reduce_add_sync(0xffffffffu, lane < cl.rank ? x : 0);
  t.all_a = __reduce_add_sync(0xffffffffu, x);
  t.all_c = __reduce_add_sync(0xffffffffu, y);
  return t;
}

// Calls put(rank, i) for every i in [0, n) with pick(i), rank counting them in ascending
// order. Called by the whole CTA; each warp takes one run of indices.
template <typename Pick, typename Put>
__device__ void compact(int n, SelShared& sh, Pick pick, Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i0 = warp * run, i1 = min(n, i0 + run);
  int mine = 0;
  for (int i = i0; i < i1; i += 32)
    mine += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && pick(i + lane)));
  if (lane == 0) sh.warp_sum[warp] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += sh.warp_sum[w];
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1 && pick(i + lane);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) put(at + __popc(m & ((1u << lane) - 1)), i + lane);
    at += __popc(m);
  }
  __syncthreads();
}

// Selection by one CTA of the `want` best of n blocks, to out in ascending order, where at most 32
// blocks are at the border. Otherwise it writes nothing and returns what is known of the border.
// Warp w has one run of the keys, in registers: elements 128 u + 4 lane + c of the run in k[4 u + c].
__device__ Border select_few(const Row& row, SelShared& sh, Hist& hist, const uint32_t* keys, int n,
                             int want, int first, uint32_t kmin, uint32_t kmax, int32_t* out) {
  constexpr int kQuads = kSelectMaxBlocks / (4 * kSelThreads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (n + 4 * kSelThreads - 1) / (4 * kSelThreads);
  const int base = warp * quads * 128 + 4 * lane;
  uint32_t k[4 * kQuads];  // 0 behind the row's end: no larger than any key
#pragma unroll
  for (int u = 0; u < kQuads; ++u) {
    const int i = base + 128 * u;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (u < quads && i < n) x = *reinterpret_cast<const uint4*>(keys + i);
    k[4 * u] = x.x;
    k[4 * u + 1] = i + 1 < n ? x.y : 0;
    k[4 * u + 2] = i + 2 < n ? x.z : 0;
    k[4 * u + 3] = i + 3 < n ? x.w : 0;
  }
  const Cluster alone = {1, 0};
  uint32_t lo = 0, hi = 0;
  if (row.bounded) {
    const Bin<uint32_t> bin = kth_largest<uint32_t>(
        [&](auto f) {
#pragma unroll
          for (int j = 0; j < 4 * kQuads; ++j)
            if (j < 4 * quads) f(k[j]);
        },
        want, kmin, kmax, spare_bits(row, kmin, kmax), hist, sh, alone,
        [](const Bin<uint32_t>&) { return false; });
    lo = bin.lo;
    hi = bin.hi;
  }
  Border b = {0, 0, want, 0};
  border(row, lo, hi, &b.maybe, &b.sure);
  if (lo == 0) return b;
  uint32_t picks = 0, edge = 0;  // a bit per key
#pragma unroll
  for (int j = 0; j < 4 * kQuads; ++j) {
    picks |= (uint32_t)(k[j] > b.sure) << j;
    edge |= (uint32_t)(k[j] >= b.maybe && k[j] <= b.sure) << j;
  }
  const Counted t = count_cluster(__popc(picks), __popc(edge), 0, sh, alone);
  b.need = want - t.all_a;
  if (t.all_c > 32 && t.all_c > b.need) return b;
  b.settled = 1;
  if (t.all_c == b.need) {
    picks |= edge;
  } else {
    // More blocks at the border than places: score them again, and rank them, one a lane.
    const int nc = t.all_c;
    for (uint32_t e = edge; e; e &= e - 1) {
      const int j = __ffs(e) - 1;
      sh.few[atomicAdd(&sh.candidates, 1)] = base + 32 * (j & ~3) + (j & 3);
    }
    __syncthreads();
    for (bool pairs = !row.exact;; pairs = false) {
      if (4 * warp < nc) {
        if (pairs)
          score_pairs(row, sh, sh.few + 4 * warp, sh.few64 + 4 * warp, min(4, nc - 4 * warp));
        else
          exact_keys(row, sh, keys, sh.few + 4 * warp, sh.few64 + 4 * warp, min(4, nc - 4 * warp));
      }
      __syncthreads();
      if (warp == 0) {
        const unsigned long long mine = lane < nc ? sh.few64[lane] : 0;
        const int rank = rank_in_warp(mine, lane < nc ? sh.few[lane] : 0, nc);
        const bool done = !pairs || decided(row, mine, rank, b.need);
        const unsigned best = __ballot_sync(0xffffffffu, rank < b.need);
        if (lane == 0) {
          sh.done = done;
          sh.best = best;
        }
      }
      __syncthreads();
      if (sh.done) break;
    }
    for (uint32_t e = edge; e; e &= e - 1) {
      const int j = __ffs(e) - 1;
      const uint32_t i = base + 32 * (j & ~3) + (j & 3);
      for (uint32_t x = sh.best; x; x &= x - 1)
        if (sh.few[__ffs(x) - 1] == i) picks |= 1u << j;
    }
  }
  const int mine = (int)__reduce_add_sync(0xffffffffu, __popc(picks));
  if (lane == 0) sh.warp_sum[warp] = mine;
  __syncthreads();
  for (int w = 0; w < warp; ++w) out += sh.warp_sum[w];
#pragma unroll 1
  for (int u = 0; u < quads; ++u, picks >>= 4) {
    const uint32_t own = picks & 15u;
    if (!__any_sync(0xffffffffu, own)) continue;
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const unsigned mask = __ballot_sync(0xffffffffu, own >> c & 1);
      before += __popc(mask & ((1u << lane) - 1));
      all += __popc(mask);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (own >> c & 1) out[before++] = first + base + 128 * u + c;
    out += all;
  }
  return b;
}

// Selection by a cluster, whose CTA `rank` holds the keys of m blocks from `first` on, with more
// than 32 blocks at the border: those are scored in fp64.
__device__ void select_many(const Row& row, SelShared& sh, Hist& hist, const Cluster& cl, uint32_t* key32,
                            unsigned long long* key64, uint32_t* cand, int m, int first, const Border& b,
                            int32_t* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 8 * kDigits; i += kSelThreads) (&hist[4][0])[i] = 0;
  for (int i = threadIdx.x; i < m; i += kSelThreads)
    if (key32[i] >= b.maybe && key32[i] <= b.sure) cand[atomicAdd(&sh.candidates, 1)] = i;
  __syncthreads();
  const int nc = sh.candidates;
  unsigned long long lo64 = ~0ull, hi64 = 0;
  for (int r = warp * 4; r < nc; r += kSelWarps * 4) {
    exact_keys(row, sh, key32, cand + r, key64 + r, min(4, nc - r));
    __syncwarp();
    for (int s = r; s < min(nc, r + 4); ++s) {
      lo64 = min(lo64, key64[s]);
      hi64 = max(hi64, key64[s]);
    }
  }
  if (lane == 0) {
    sh.lo[warp] = lo64;
    sh.hi[warp] = hi64;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSelWarps; ++w) {
      sh.lo[0] = min(sh.lo[0], sh.lo[w]);
      sh.hi[0] = max(sh.hi[0], sh.hi[w]);
    }
    sh.pub[1][0] = sh.lo[0];
    sh.pub[1][1] = sh.hi[0];
  }
  cl.sync();
  for (int r = 0; r < cl.size; ++r) {
    lo64 = min(lo64, cl.read(&sh.pub[1][0], r));
    hi64 = max(hi64, cl.read(&sh.pub[1][1], r));
  }
  // All keys of the bin are taken, or (one value) as many of the lowest blocks as it takes.
  const Bin<unsigned long long> bin = kth_largest<unsigned long long>(
      [&](auto f) {
        for (int i = threadIdx.x; i < nc; i += kSelThreads) f(key64[i]);
      },
      b.need, lo64, hi64, 0, hist + 4, sh, cl,
      [&](const Bin<unsigned long long>& x) { return x.above + x.inside == b.need; });
  int at_edge = 0;
  for (int r = threadIdx.x; r < nc; r += kSelThreads) {
    const bool edge = key64[r] >= bin.lo && key64[r] <= bin.hi;
    at_edge += edge;
    key32[cand[r]] = key64[r] > bin.hi ? kTaken : edge ? kEdge : 0u;
  }
  const int rest = b.need - bin.above - count_cluster(at_edge, 0, 2, sh, cl).before_a;
  compact(
      m, sh, [&](int i) { return key32[i] == kEdge; },
      [&](int k, int i) { key32[i] = k < rest ? kTaken : 0u; });
  int in = 0;
  for (int i = threadIdx.x; i < m; i += kSelThreads) in += key32[i] > b.sure;
  const int before = count_cluster(in, 0, 3, sh, cl).before_a;
  compact(
      m, sh, [&](int i) { return key32[i] > b.sure; },
      [&](int r, int i) { out[before + r] = first + i; });
  if (cl.size > 1) cl.sync();  // the others may still be reading this CTA's shared memory
}

}  // namespace

// kWide: for tables of more blocks than one warp selects, or (to be narrow) a CTA. A warp has two
// groups of 8 blocks' summaries in flight, which takes 512 rows of 600 blocks 39.5 us, 45.8 with
// one. Narrow, the registers of a second group buy resident CTAs: 512 rows of 256 blocks take 14.0
// us with one group and four CTAs per SM, 17.2 with three, 19.5 with five (whose registers spill);
// two groups took 18.3 where one took 15.2.
template <bool kWide>
__global__ void __launch_bounds__(kSelThreads, kWide ? 2 : 4)
    select_blocks_kernel(const __grid_constant__ SelectArgs a, int chunk_cap) {
  extern __shared__ __align__(16) unsigned long long sel_smem[];
  __shared__ SelShared sh;
  __shared__ int hist[kWide ? 12 : 1][kDigits];
  pdl_wait_then_launch();
  const Cluster cl = {kWide ? (int)cg::this_cluster().num_blocks() : 1,
                      kWide ? (int)cg::this_cluster().block_rank() : 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = blockIdx.x / cl.size;  // (query row, kv head)
  const int g = (int)(seg % a.Hkv);
  const int64_t qrow = seg / a.Hkv;
  const int b = (int)(qrow / a.q_len), qi = (int)(qrow % a.q_len);
  const int cap = a.max_blocks * kBs;
  const int raw = __ldg(a.seq_lens + b);

  const int len = clamp_len(raw, cap);
  if (len != raw && g == 0 && qi == 0 && cl.rank == 0 && threadIdx.x == 0)
    flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  const int row_len = len - a.q_len + 1 + qi;
  const int n = row_len > 0 ? (row_len + kBs - 1) / kBs : 0;
  const int K = a.num_selected;
  int32_t* out = a.out + seg * K;
  // Blocks [0, e0) and [e1, n) are always taken; the others compete for `want` places.
  const int e0 = a.num_sink, e1 = n - a.num_recent;
  const int want = K - a.num_sink - a.num_recent;
  if (cl.rank == 0) {
    if (n <= K) {
      for (int i = threadIdx.x; i < K; i += kSelThreads) out[i] = i < n ? i : -1;
    } else {
      for (int i = threadIdx.x; i < e0; i += kSelThreads) out[i] = i;
      for (int i = threadIdx.x; i < a.num_recent; i += kSelThreads) out[e0 + want + i] = e1 + i;
    }
  }
  if (n <= K || want == 0) return;  // the whole cluster takes this way
  out += e0;
  const int total = e1 - e0;  // > want
  // Few blocks are one CTA's work, however wide the table and with it the cluster.
  const bool by_warp = !kWide || total <= 32 * kWarpKeys;
  if (by_warp && cl.rank) return;
  // This CTA's run of competing blocks: [first, first + m).
  const int chunk = by_warp ? total : ((total + cl.size - 1) / cl.size + 7) & ~7;
  const int first = e0 + cl.rank * chunk;
  const int m = max(0, min(chunk, e1 - first));
  // [chunk_cap], and [max_blocks] in the same place: the keys of the whole row, which the first
  // CTA of a cluster has for as long as it selects by itself.
  unsigned long long* key64 = sel_smem;
  uint32_t* gathered = reinterpret_cast<uint32_t*>(sel_smem);
  const bool many = kWide && !by_warp && cl.size > 1;
  uint32_t* key32 = gathered + (kWide && cl.size > 1 ? max(2 * chunk_cap, a.max_blocks) : 2 * chunk_cap);
  uint32_t* cand = key32 + chunk_cap;  // [chunk_cap] each
  Row row;
  row.table = a.block_table + (int64_t)b * a.max_blocks + first;
  row.sum = a.summaries + (int64_t)g * kSumBytes + lane * 16;
  row.sum_stride = (int64_t)a.Hkv * kSumBytes;
  row.num_blocks = a.num_blocks;
  constexpr int kGroup = kWide ? 16 : 8;
  // Table entries of a group, one per lane; a group that ends the run repeats its last block,
  // so that every load below is unconditional and all of them are in flight together.
  auto entry = [&](int j) { return j < m ? __ldg(row.table + min(j + (lane & (kGroup - 1)), m - 1)) : 0; };
  int next = entry(warp * kGroup);

  if (many) cg::this_cluster().barrier_arrive();

  // ---- coefficients: thread d sums N (d < 128) or P of its channel over the heads, and what
  // the fp32 sums leave out (the error of each addition, found exactly)
  {
    const int d = threadIdx.x;
    const uint16_t* q = a.q + (qrow * a.H + (int64_t)g * a.n_rep) * kDim + d % kDim;
    float sum = 0.f, low = 0.f;
    uint32_t any = 0;
    for (int h0 = 0; h0 < a.n_rep; h0 += 8) {
      uint32_t bits[8];
#pragma unroll
      for (int h = 0; h < 8; ++h) bits[h] = h0 + h < a.n_rep ? __ldg(q + (h0 + h) * kDim) : 0u;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        any |= bits[h] & 0x7fffu;
        const float v = __uint_as_float(bits[h] << 16);
        const float x = d < kDim ? min_nan(v, 0.f) : max_nan(v, 0.f);
        const float s = add_ieee(sum, x);
        const float back = sub_ieee(s, sum);
        low = add_ieee(low, add_ieee(sub_ieee(sum, sub_ieee(s, back)), sub_ieee(x, back)));
        sum = s;
      }
    }
    const float all = add_ieee(sum, low);
    const bool finite = abs_ieee(all) < INFINITY;
    low = finite ? add_ieee(low, sub_ieee(sum, all)) : 0.f;
    sum = finite ? all : sum;
    sh.coef[d] = sum;
    sh.coef_low[d] = low;
    float size = abs_ieee(sum);
#pragma unroll
    for (int o = 16; o; o >>= 1) size = add_ieee(size, __shfl_xor_sync(0xffffffffu, size, o));
    any = __reduce_or_sync(0xffffffffu, any);
    if (lane == 0) {
      sh.size[warp] = size;
      sh.any_q[warp] = any;
    }
    if (threadIdx.x == 0) sh.candidates = 0;
  }
  if (!by_warp)
    for (int i = threadIdx.x; i < 4 * kDigits; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();

  // ---- fp32 scores
  uint64_t coef[4];  // of channels 2i and 2i + 1
#pragma unroll
  for (int i = 0; i < 4; ++i) coef[i] = f2pack(sh.coef[8 * lane + 2 * i], sh.coef[8 * lane + 2 * i + 1]);
  uint32_t* far = nullptr;
  if (many) {
    cg::this_cluster().barrier_wait();  // every CTA runs: its shared memory can be written
    far = cg::this_cluster().map_shared_rank(gathered, 0) + (first - e0);
  }
  uint32_t vmax = 0;  // the largest |summary| of the even and the odd channels (NaN: the largest bits)
  uint32_t kmin = 0xffffffffu, kmax = 0;
  for (int j0 = warp * kGroup; j0 < m; j0 += kSelWarps * kGroup) {
    const int blk = next;
    next = entry(j0 + kSelWarps * kGroup);
    const bool bad = blk < 0 || (int64_t)blk >= a.num_blocks;
    const int from = bad ? 0 : blk;
    uint4 x[kGroup];
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
      x[u] = ld_nc_v4(row.sum + __shfl_sync(0xffffffffu, from, u) * row.sum_stride);
    const unsigned bad_mask = __ballot_sync(0xffffffffu, bad);
    if (bad_mask) {  // block 0 stood in for them: it must not count in vmax
      if (bad) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
        if (bad_mask >> u & 1) x[u] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u0 = 0; u0 < kGroup; u0 += 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t w[4] = {x[u0 + u].x, x[u0 + u].y, x[u0 + u].z, x[u0 + u].w};
        uint64_t s = 0;  // two sums of four products
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = ffma2(coef[i], f2pack(bf16lo(w[i]), bf16hi(w[i])), s);
          vmax = max_abs2(vmax, w[i]);
        }
        const float2 both = f2unpack(s);
        v[u] = both.x + both.y;
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
      const int u = u0 + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
      if ((lane & 3) == 0 && j0 + u < m) {
        const uint32_t key = bad_mask >> u & 1 ? 0u : order_key(v[0]);
        key32[j0 + u] = key;
        if (many) far[j0 + u] = key;
        kmin = min(kmin, key);
        kmax = max(kmax, key);
      }
    }
  }

  // ---- range of the keys and of the summaries, over the cluster
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  uint32_t top = __reduce_max_sync(0xffffffffu, max(vmax & 0x7fffu, vmax >> 16 & 0x7fffu));
  if (lane == 0) {
    sh.lo[warp] = kmin;
    sh.hi[warp] = kmax;
    sh.amax[warp] = top;
  }
  __syncthreads();
  if (by_warp && warp) return;
  top = __reduce_max_sync(0xffffffffu, sh.amax[lane & 7]);
  if (!by_warp) {
    if (threadIdx.x < cl.size) {  // thread r tells CTA r
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int w = 0; w < kSelWarps; ++w) {
        lo = min(lo, (uint32_t)sh.lo[w]);
        hi = max(hi, (uint32_t)sh.hi[w]);
      }
      uint32_t* to = sh.range[cl.rank];
      if (cl.size > 1) to = cg::this_cluster().map_shared_rank(to, threadIdx.x);
      to[0] = lo;
      to[1] = hi;
      to[2] = top;
    }
    cl.sync();
    const int r = lane < cl.size ? lane : 0;
    kmin = __reduce_min_sync(0xffffffffu, sh.range[r][0]);
    kmax = __reduce_max_sync(0xffffffffu, sh.range[r][1]);
    top = __reduce_max_sync(0xffffffffu, sh.range[r][2]);
  }
  float size = 0.f;
  uint32_t any = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    size = add_ieee(size, sh.size[w]);
    any |= sh.any_q[w];
  }
  const float reach = mul_ieee(size, __uint_as_float(top << 16));  // bounds |score|, partial sums
  // A reach that is not finite bounds nothing. The added constant covers sums flushed to zero.
  row.bounded = reach < 1e37f;
  row.exact = row.bounded && (any == 0 || top == 0);
  row.eps = row.exact ? 0.f : reach * (14.f * 0x1p-24f) + 1e-35f;
  if constexpr (kWide) {
    if (!by_warp) {
      // One CTA selects where few blocks are at the border: a barrier of the cluster with a read of
      // another CTA's shared memory takes about a microsecond, and a selection by all CTAs six.
      Border b;
      if (cl.rank == 0) b = select_few(row, sh, hist, many ? gathered : key32, total, want, e0, kmin, kmax, out);
      if (many) {
        if (cl.rank == 0 && threadIdx.x < cl.size)
          *cg::this_cluster().map_shared_rank(&sh.border, threadIdx.x) = b;
        cl.sync();
        b = sh.border;
      }
      if (!b.settled) select_many(row, sh, hist, cl, key32, key64, cand, m, first, b, out);
      return;
    }
  }
  select_by_warp(row, sh, key32, key64, cand, m, want, first, out);
}

template <bool kWide>
static cudaError_t launch_select_n(const SelectArgs& a, int C, int64_t segs, cudaStream_t stream) {
  const int alone = a.max_blocks < 32 * kWarpKeys ? a.max_blocks : 32 * kWarpKeys;
  int chunk_cap = ((a.max_blocks + C - 1) / C + 7) & ~7;
  if (chunk_cap < alone) chunk_cap = alone;
  // fp64 keys (or all fp32 keys of a cluster's row), fp32 keys, candidates
  const size_t shared = C > 1 && a.max_blocks > 2 * chunk_cap ? a.max_blocks : 2 * chunk_cap;
  const size_t smem = (shared + 2 * chunk_cap) * 4;
  if (smem > 16 * 1024) {  // with the static part more than a kernel gets unasked
    const cudaError_t e = cudaFuncSetAttribute(select_blocks_kernel<kWide>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 16);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_blocks_kernel<kWide>, a, chunk_cap);
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t segs = (int64_t)a.B * a.q_len * a.Hkv;
  if (segs == 0) return cudaSuccess;
  // Cluster width: as wide as a grid of one CTA per SM allows, or two where the rows are long, and
  // enough that a CTA's keys stay within 64 KB. Measured on GB300 (us for 1, 2, 4, 8 CTAs a row): 8
  // rows of 600 blocks 11.6, 10.2, 8.7, 7.7; 32 of 280 9.1, 9.2, 8.3, 8.7; 32 of 1,000 15.4, 11.8,
  // 9.5, 9.4; 32 of 8,000 -, 67, 41, 32; 128 of 600 13.9, 14.5, 21, 33; 128 of 1,000 16.8, 15.9,
  // 22, 34; 128 of 8,000 -, 90, 103, 119; 512 of 1,000 56, 71, 89, 137.
  int C = 1;
  const int64_t most = (a.max_blocks >= 800 ? 2 : 1) * (int64_t)num_sms;
  while (C < kMaxCluster && (a.max_blocks > kMaxChunk * C || segs * 2 * C <= most)) C *= 2;
  if (a.max_blocks > 32 * kWarpKeys) return launch_select_n<true>(a, C, segs, stream);
  return launch_select_n<false>(a, 1, segs, stream);
}

}  // namespace pkv
