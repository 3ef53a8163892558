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
#include "mma_bf16.cuh"
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
// One cluster of C CTAs per kv head and query row, or two neighbouring query rows of a sequence
// (kRows). Each CTA scores one run of the rows' blocks and keeps their keys (order-preserving whole numbers) in its shared memory. A row of at most
// 256 competing blocks is one CTA's, and is selected by one warp with the keys in registers;
// of longer ones all keys go to the shared memory of the cluster's first CTA, which selects with
// the keys in registers. Only where many blocks are at the border the CTAs select together,
// exchanging histograms and counts through distributed shared memory.
//
// Scores are matrix products of bf16 numbers with fp32 sums: a fp32 coefficient is the sum of three
// bf16 numbers, so a row's coefficients are three columns of 256, and 16 summaries, as they lie in
// memory, the rows of the other factor. A warp multiplies them 16 channels at a time (mma.sync: the
// operands come straight from global memory to registers, once, and there are 3 or 6 columns), in
// an order of the channels that lets a lane load 16 bytes. Products with fused multiply-adds and
// sums over the lanes took 50 cycles a block and half the kernel's time: 8 rows of 8,000 blocks 18.6
// us, 14.7 so. Selection needs exact order only at the border, so the kernel bounds the error,
//
//   |score32 - score| <= eps = 56 2^-24 (sum_d P_d + |N_d|) max |summary|
//
// (the 16 sums of a product, each at least as good as a truncation to 24 bits: 32, of which 20,000
// products of random numbers with exponents up to 40 apart reached 4; pkv_selftest_bf16_products
// hands the products out, and a test holds them to this; the 16 products' sum 16; the columns' 3;
// the coefficients 1; room for the bound's own), and finds the K-th largest fp32 score tau to within
// a bin narrower than eps, takes every block above the bin by more than 2 eps and none below it by
// more, and scores the blocks between again where they are more than the places left: few of them in
// pairs of fp32 numbers, and in fp64 where those do not tell them apart. The result is that of fp64
// scores, ties to the lower block, whatever the order of the fp32 sums.
//
// A block whose score is NaN (a NaN key, or infinite keys that cancel) ranks above all others.
namespace {

constexpr int kSelWarps = 8;
constexpr int kSelThreads = 32 * kSelWarps;
constexpr int kMaxCluster = 8;
constexpr int kMaxChunk = 2048;           // blocks whose keys a CTA holds
constexpr int kMaxKeys = kSelectMaxBlocks > 2 * kMaxChunk ? kSelectMaxBlocks : 2 * kMaxChunk;
static_assert(kSelectMaxBlocks <= kMaxCluster * kMaxChunk, "a row's keys fit its cluster");
constexpr int kDigitBits = 9;             // two digits of this size decide most 32-bit searches
constexpr int kDigits = 1 << kDigitBits;  // two per thread
constexpr int kWarpKeys = 8;              // keys of a lane where one warp selects
constexpr uint32_t kNanKey = 0xfffffffeu;
constexpr uint32_t kTaken = 0xffffffffu;  // above every score's key
constexpr uint32_t kBad = 0xffffffffu;    // half a score of a bad block: no sum's NaN has these bits
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

// What decides a row: keys above `sure` are in, keys below `maybe` are out, and of those between
// the `need` best by more exact scores.
struct Border {
  uint32_t maybe, sure;
  int need, settled;
};

// Digit counts: 4 passes over 32-bit keys, 8 over 64.
using Hist = int[4 + 8][kDigits];

// Shared memory of one CTA. What other CTAs of the cluster read (counts, pub, the keys) is
// written once per row and place, so one cluster barrier between the writes and the reads is
// enough; another ends a row.
struct SelShared {
  unsigned long long pub[4][2];          // a pair of numbers per exchange
  unsigned long long lo[kSelWarps], hi[kSelWarps];
  int warp_sum[kSelWarps], warp_sum2[kSelWarps];
  int digit, above, inside, candidates, done;
  uint32_t few[32], best;                // a single CTA's candidates, and which are taken
  unsigned long long few64[32];          // their keys
  uint32_t top[kSelWarps], tops[kMaxCluster];  // largest |summary| of each warp and each CTA
};

// The same for a query row.
struct RowShared {
  float coef[2 * kDim], coef_low[2 * kDim];  // N, then P: their fp32 sums and what those left out
  float size[kSelWarps];
  uint32_t any_q[kSelWarps];
  uint32_t lo[kSelWarps], hi[kSelWarps];     // smallest and largest key of each warp
  uint32_t los[kMaxCluster], his[kMaxCluster];  // and of each CTA
  Border border;
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

// A row's coefficients, where its blocks lie and what bounds their scores.
struct Row {
  const float *coef, *coef_low;
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
__device__ void score64(const Row& row, const uint32_t* cand,
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
    k[i] = widen_bits(__float_as_uint(row.coef[8 * lane + i])) +
           widen_bits(__float_as_uint(row.coef_low[8 * lane + i]));
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
__device__ void score_pairs(const Row& row, const uint32_t* cand,
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
    const float* c = row.coef + 8 * (sub + 8 * k);
    const float* low = row.coef_low + 8 * (sub + 8 * k);
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
__device__ __forceinline__ void exact_keys(const Row& row, const uint32_t* key32,
                                           const uint32_t* cand, unsigned long long* key64, int n) {
  const int lane = threadIdx.x & 31;
  if (!row.exact)
    score64(row, cand, key64, n);
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
  return gap > row.eps * 0x1p-15f + 1e-37f;  // eps is at least 56 2^-24 of the bound
}

// Low bits of the keys that need not be decided: a bin of 2^bits keys in [kmin, kmax] is
// narrower than eps, for its scores are at most the largest magnitude's 2^-23 apart.
__device__ __forceinline__ int spare_bits(const Row& row, uint32_t kmin, uint32_t kmax) {
  if (kmin == 0 || row.exact) return 0;  // bad blocks among them
  const uint32_t top = __float_as_uint(fmaxf(fabsf(key_score(kmin)), fabsf(key_score(kmax)))) >> 23;
  const int bits = (int)(__float_as_uint(row.eps) >> 23) - ((int)top - 23);
  return min(max(bits, 0), 31);
}

// [maybe, sure] from the bin [lo, hi] that holds the K-th largest key. With lo = 0 (bad blocks at
// the border, or no bound) every key is between them, whatever the scores: no block is in before
// the choice, so all of the row's places are the choice's.
__device__ __forceinline__ void border(const Row& row, uint32_t lo, uint32_t hi, uint32_t* maybe,
                                       uint32_t* sure) {
  *maybe = 0;
  *sure = kNanKey;
  if (lo == 0) return;
  if (row.exact) {
    *maybe = *sure = lo;
  } else if (row.bounded) {
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
__device__ void select_by_warp(const Row& row, const uint32_t* key32,
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
      for (int r = 0; r < nc; r += 4) score_pairs(row, cand + r, key64 + r, min(4, nc - r));
      __syncwarp();
      const unsigned long long mine = lane < nc ? key64[lane] : 0;
      const int rank = rank_in_warp(mine, lane, nc);
      done = decided(row, mine, rank, need);
      if (done && lane < nc) cand[lane] |= rank < need ? 0x80000000u : 0u;
      __syncwarp();
    }
    if (!done) {
      for (int r = 0; r < nc; r += 4) exact_keys(row, key32, cand + r, key64 + r, min(4, nc - r));
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
  for (int i = threadIdx.x; i < 4 * kDigits; i += kSelThreads) (&hist[0][0])[i] = 0;
  if (threadIdx.x == 0) sh.candidates = 0;
  __syncthreads();
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
          score_pairs(row, sh.few + 4 * warp, sh.few64 + 4 * warp, min(4, nc - 4 * warp));
        else
          exact_keys(row, keys, sh.few + 4 * warp, sh.few64 + 4 * warp, min(4, nc - 4 * warp));
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
  if (threadIdx.x == 0) sh.candidates = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < m; i += kSelThreads)
    if (key32[i] >= b.maybe && key32[i] <= b.sure) cand[atomicAdd(&sh.candidates, 1)] = i;
  __syncthreads();
  const int nc = sh.candidates;
  unsigned long long lo64 = ~0ull, hi64 = 0;
  for (int r = warp * 4; r < nc; r += kSelWarps * 4) {
    exact_keys(row, key32, cand + r, key64 + r, min(4, nc - r));
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

// kWide: for tables of more blocks than one warp selects, or (to be narrow) a CTA; kRows: query rows
// of a sequence that a cluster selects for. A wide kernel's warp has 16 whole summaries in flight;
// narrow, two warps share them, so that rows of 64 blocks keep all of them busy and 64 registers do,
// for four CTAs per SM: 512 rows of 256 blocks take 14.0 us (three CTAs 17.1, five, whose registers
// spill, 23.8), of 128 10.3 (12.7, 15.7), of random lengths up to 256 13.5 (12.5, 21).
template <bool kWide, int kRows>
__global__ void __launch_bounds__(kSelThreads, kWide ? 2 : 4)
    select_blocks_kernel(const __grid_constant__ SelectArgs a, int chunk_cap) {
  extern __shared__ __align__(16) unsigned long long sel_smem[];
  __shared__ SelShared sh;
  __shared__ RowShared rows[kRows];
  // Columns 0 to 2 (and 4 to 6 of a second row) hold a row's coefficients; what is in the others
  // does not count. The stride keeps two columns' 64 bytes in different banks.
  __shared__ __align__(16) uint16_t split[8][2 * kDim + 32];
  __shared__ int hist[kWide ? 12 : 1][kDigits];
  pdl_wait_then_launch();
  const Cluster cl = {kWide ? (int)cg::this_cluster().num_blocks() : 1,
                      kWide ? (int)cg::this_cluster().block_rank() : 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = blockIdx.x / cl.size;  // (kRows query rows, kv head)
  const int g = (int)(seg % a.Hkv);
  const int64_t group = seg / a.Hkv;
  const int groups = (a.q_len + kRows - 1) / kRows;
  const int b = (int)(group / groups), q0 = (int)(group % groups) * kRows;
  const int cap = a.max_blocks * kBs;
  const int raw = __ldg(a.seq_lens + b);
  const int len = clamp_len(raw, cap);
  if (len != raw && g == 0 && q0 == 0 && cl.rank == 0 && threadIdx.x == 0)
    flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  const int K = a.num_selected;
  // Blocks [0, e0) and the last num_recent are always taken; the others compete for `want` places.
  const int e0 = a.num_sink, want = K - a.num_sink - a.num_recent;
  int32_t* first_out = a.out + (((int64_t)b * a.q_len + q0) * a.Hkv + g) * K;
  auto out = [&](int r) { return first_out + (kRows == 1 ? 0 : r * (int64_t)a.Hkv * K); };
  int total[kRows];  // competing blocks (of the later row at least as many), 0: none to choose
  int most = 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    total[r] = 0;
    if (q0 + r >= a.q_len) continue;
    const int row_len = len - a.q_len + 1 + q0 + r;
    const int n = row_len > 0 ? (row_len + kBs - 1) / kBs : 0;
    if (cl.rank == 0) {
      if (n <= K) {
        for (int i = threadIdx.x; i < K; i += kSelThreads) out(r)[i] = i < n ? i : -1;
      } else {
        for (int i = threadIdx.x; i < e0; i += kSelThreads) out(r)[i] = i;
        for (int i = threadIdx.x; i < a.num_recent; i += kSelThreads)
          out(r)[e0 + want + i] = n - a.num_recent + i;
      }
    }
    if (n > K && want > 0) total[r] = n - a.num_recent - e0;  // > want
    most = max(most, total[r]);
  }
  if (most == 0) return;  // the whole cluster takes this way
  // Few blocks are one CTA's work, however wide the table and with it the cluster.
  const bool by_warp = !kWide || most <= 32 * kWarpKeys;
  if (by_warp && cl.rank) return;
  const bool many = kWide && !by_warp && cl.size > 1;
  if (many) cg::this_cluster().barrier_arrive();
  // This CTA's run of competing blocks: [start, start + m), of a row as many of them as it has.
  const int chunk = by_warp ? most : ((most + cl.size - 1) / cl.size + 7) & ~7;
  const int start = cl.rank * chunk;
  const int m = max(0, min(chunk, most - start));
  // [chunk_cap], and [max_blocks] in the same place: the keys of a whole row, in the CTA of a
  // cluster that selects for it, until it has.
  unsigned long long* key64 = sel_smem;
  uint32_t* gathered = reinterpret_cast<uint32_t*>(sel_smem);
  uint32_t* key32 = gathered + (kWide && cl.size > 1 ? max(2 * chunk_cap, a.max_blocks) : 2 * chunk_cap);
  uint32_t* cand = key32 + kRows * chunk_cap;  // [chunk_cap] per row; [chunk_cap]
  Row row;
  row.table = a.block_table + (int64_t)b * a.max_blocks + e0 + start;
  row.sum = a.summaries + (int64_t)g * kSumBytes + lane * 16;
  row.sum_stride = (int64_t)a.Hkv * kSumBytes;
  row.num_blocks = a.num_blocks;
  constexpr int kGroup = 16;  // blocks of a matrix product
  // Table entries of a group, one per lane; a group that ends the run repeats its last block,
  // so that every load below is unconditional and all of them are in flight together.
  auto entry = [&](int j) { return j < m ? __ldg(row.table + min(j + (lane & (kGroup - 1)), m - 1)) : 0; };
  // Narrow, two warps share a group, one on the minima and one on the maxima.
  constexpr int kShare = kWide ? 1 : 2;
  constexpr int kSweep = kSelWarps / kShare * kGroup;
  const int j00 = warp / kShare * kGroup;
  int next = entry(j00);

  // ---- coefficients: thread d sums N (d < 128) or P of its channel over the heads, and what
  // the fp32 sums leave out (the error of each addition, found exactly)
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (total[r] == 0) continue;
    const int d = threadIdx.x;
    const uint16_t* q =
        a.q + (((int64_t)b * a.q_len + q0 + r) * a.H + (int64_t)g * a.n_rep) * kDim + d % kDim;
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
    // Three bf16 numbers whose sum it is, one each 8 of its 24 bits.
    const float high = __bfloat162float(__float2bfloat16_rn(sum));
    const float rest = sub_ieee(sum, high);
    const float mid = __bfloat162float(__float2bfloat16_rn(rest));
    split[4 * r][d] = __float_as_uint(high) >> 16;
    split[4 * r + 1][d] = __float_as_uint(mid) >> 16;
    split[4 * r + 2][d] = __bfloat16_as_ushort(__float2bfloat16_rn(sub_ieee(rest, mid)));
    rows[r].coef[d] = sum;
    rows[r].coef_low[d] = low;
    float size = abs_ieee(sum);
#pragma unroll
    for (int o = 16; o; o >>= 1) size = add_ieee(size, __shfl_xor_sync(0xffffffffu, size, o));
    any = __reduce_or_sync(0xffffffffu, any);
    if (lane == 0) {
      rows[r].size[warp] = size;
      rows[r].any_q[warp] = any;
    }
  }
  __syncthreads();

  // ---- fp32 scores
  uint32_t kmin = 0xffffffffu, kmax = 0;  // of the row that the lane writes
  uint32_t* far = nullptr;
  const int at = lane >> 2, c = lane & 3;  // place in the fragments
  const int r = kRows == 1 ? 0 : c >> 1;
  if (many) {
    cg::this_cluster().barrier_wait();  // every CTA runs: its shared memory can be written
    far = cg::this_cluster().map_shared_rank(gathered, r) + start;
  }
  const int mine = c < 2 * kRows ? min(m, (kRows == 1 || r == 0 ? total[0] : total[kRows - 1]) - start) : 0;
  uint32_t vmax = 0;  // the largest |summary| of the even and the odd channels (NaN: the largest bits)
  constexpr int kPieces = 8 / kShare;  // 64-byte pieces of a summary
  const int t0 = kPieces * (warp % kShare);
  const uint8_t* sums = row.sum + (c - lane) * 16 + t0 * 64;
  for (int j0 = j00; j0 < m; j0 += kSweep) {
    const int blk = next;
    next = entry(j0 + kSweep);
    const bool bad = blk < 0 || (int64_t)blk >= a.num_blocks;
    const int from = bad ? 0 : blk;
    const uint8_t* p = sums + __shfl_sync(0xffffffffu, from, at) * row.sum_stride;
    const uint8_t* p8 = sums + __shfl_sync(0xffffffffu, from, at + 8) * row.sum_stride;
    const unsigned bad_mask = __ballot_sync(0xffffffffu, bad);
    if (bad) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint4 x[kPieces], y[kPieces];
#pragma unroll
    for (int t = 0; t < kPieces; ++t) {
      x[t] = ld_nc_v4(p + t * 64);
      y[t] = ld_nc_v4(p8 + t * 64);
    }
    if (bad_mask) {  // block 0 stood in for them: it must not count in vmax
#pragma unroll
      for (int t = 0; t < kPieces; ++t) {
        if (bad_mask >> at & 1) x[t] = make_uint4(0, 0, 0, 0);
        if (bad_mask >> (at + 8) & 1) y[t] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < kPieces; ++t) {
      const uint4 k = *reinterpret_cast<const uint4*>(&split[at][32 * (t0 + t) + 8 * c]);
      float d[4];
      mma16816(d, x[t].x, y[t].x, x[t].y, y[t].y, k.x, k.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += d[i];
      mma16816(d, x[t].z, y[t].z, x[t].w, y[t].w, k.z, k.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += d[i];
      vmax = max_abs2(max_abs2(max_abs2(vmax, x[t].x), x[t].y), max_abs2(x[t].z, x[t].w));
      vmax = max_abs2(max_abs2(max_abs2(vmax, y[t].x), y[t].y), max_abs2(y[t].z, y[t].w));
    }
    // A row's three columns are in two lanes: both sum them, and one takes block `at`, one at + 8.
    float v = c & 1 ? acc[0] : acc[0] + acc[1], v8 = c & 1 ? acc[2] : acc[2] + acc[3];
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v8 += __shfl_xor_sync(0xffffffffu, v8, 1);
    const int u = at + 8 * (c & 1);
    const float score = c & 1 ? v8 : v;
    if (!kWide) {
      if (j0 + u < mine) (t0 ? cand : key32)[j0 + u] = bad_mask >> u & 1 ? kBad : __float_as_uint(score);
    } else if (j0 + u < mine) {
      const uint32_t key = bad_mask >> u & 1 ? 0u : order_key(score);
      key32[r * chunk_cap + j0 + u] = key;
      if (many) far[j0 + u] = key;
      kmin = min(kmin, key);
      kmax = max(kmax, key);
    }
  }

  // ---- range of the keys and of the summaries
  uint32_t top = __reduce_max_sync(0xffffffffu, max(vmax & 0x7fffu, vmax >> 16 & 0x7fffu));
  if (lane == 0) sh.top[warp] = top;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t lo = __reduce_min_sync(0xffffffffu, i == r ? kmin : 0xffffffffu);
    const uint32_t hi = __reduce_max_sync(0xffffffffu, i == r ? kmax : 0);
    if (lane == 0) {
      rows[i].lo[warp] = lo;
      rows[i].hi[warp] = hi;
    }
  }
  __syncthreads();
  if (!kWide) {  // the two halves of the scores; a row has at most as many blocks as the CTA threads
    static_assert(32 * kWarpKeys <= kSelThreads, "one step");
    if (threadIdx.x < most) {
      const uint32_t low = key32[threadIdx.x];
      key32[threadIdx.x] =
          low == kBad ? 0u : order_key(__uint_as_float(low) + __uint_as_float(cand[threadIdx.x]));
    }
    __syncthreads();
  }
  top = __reduce_max_sync(0xffffffffu, sh.top[lane & 7]);
  if (!by_warp) {  // over the cluster
    if (threadIdx.x < cl.size) {  // thread c tells CTA c
      auto tell = [&](uint32_t* place, uint32_t x) {
        *(cl.size > 1 ? cg::this_cluster().map_shared_rank(place, threadIdx.x) : place) = x;
      };
      tell(&sh.tops[cl.rank], top);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int w = 0; w < kSelWarps; ++w) {
          lo = min(lo, rows[r].lo[w]);
          hi = max(hi, rows[r].hi[w]);
        }
        tell(&rows[r].los[cl.rank], lo);
        tell(&rows[r].his[cl.rank], hi);
      }
    }
    cl.sync();
    top = __reduce_max_sync(0xffffffffu, sh.tops[lane < cl.size ? lane : 0]);
  }
  auto bound = [&](const RowShared& x) {
    row.coef = x.coef;
    row.coef_low = x.coef_low;
    float size = 0.f;
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      size = add_ieee(size, x.size[w]);
      any |= x.any_q[w];
    }
    const float reach = mul_ieee(size, __uint_as_float(top << 16));  // bounds |score|, partial sums
    // A reach that is not finite bounds nothing.
    row.bounded = reach < 1e37f;
    row.exact = row.bounded && (any == 0 || top == 0);
    // Numbers that the products may take for zero are below 2^-126.
    row.eps = row.exact ? 0.f
                        : reach * (56.f * 0x1p-24f) + size * 0x1p-125f +
                              __uint_as_float(top << 16) * 0x1p-115f + 1e-35f;
  };
  auto count = [&](int r) { return kRows == 1 || r == 0 ? total[0] : total[kRows - 1]; };
  if constexpr (kWide) {
    if (!by_warp) {
      // One CTA selects where few blocks are at the border, another for the other row: a barrier of
      // the cluster with a read of another CTA's shared memory takes about a microsecond, and a
      // selection by all CTAs six.
#pragma unroll 1
      for (int r = 0; r < kRows; ++r) {
        if (count(r) == 0 || cl.rank != r % cl.size) continue;
        bound(rows[r]);
        const int c = lane < cl.size ? lane : 0;
        const uint32_t lo = __reduce_min_sync(0xffffffffu, rows[r].los[c]);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, rows[r].his[c]);
        Row whole = row;
        whole.table -= start;
        const Border found = select_few(whole, sh, hist, many ? gathered : key32 + r * chunk_cap, count(r),
                                        want, e0, lo, hi, out(r) + e0);
        if (many && threadIdx.x < cl.size)
          *cg::this_cluster().map_shared_rank(&rows[r].border, threadIdx.x) = found;
        else if (!many && threadIdx.x == 0)
          rows[r].border = found;
      }
      cl.sync();
#pragma unroll 1
      for (int r = 0; r < kRows; ++r) {
        if (count(r) == 0 || rows[r].border.settled) continue;
        bound(rows[r]);
        select_many(row, sh, hist, cl, key32 + r * chunk_cap, key64, cand, max(0, min(m, count(r) - start)),
                    e0 + start, rows[r].border, out(r) + e0);
      }
      return;
    }
  }
  // In a narrow kernel any one of the warps, so that those of an SM's CTAs are not all on one of
  // its four schedulers (by the hash 13.5 us for a decode step, always the first warp 13.6).
  const int turn = kWide ? warp : (warp + (int)(blockIdx.x * 2654435761u >> 29)) & (kSelWarps - 1);
  if (turn >= kRows || count(turn) == 0) return;
  bound(rows[turn]);
  select_by_warp(row, key32 + turn * chunk_cap, key64 + turn * 32 * kWarpKeys, cand + turn * 32 * kWarpKeys,
                 count(turn), want, e0, out(turn) + e0);
}

template <bool kWide, int kRows>
static cudaError_t launch_select_n(const SelectArgs& a, int C, int64_t segs, cudaStream_t stream) {
  // Rows of one warp each have 256 places in a CTA, whatever the cluster.
  const int alone = kRows == 1 && a.max_blocks < 32 * kWarpKeys ? a.max_blocks : kRows * 32 * kWarpKeys;
  int chunk_cap = ((a.max_blocks + C - 1) / C + 7) & ~7;
  if (chunk_cap < alone) chunk_cap = alone;
  // fp64 keys (or all fp32 keys of a cluster's row), fp32 keys, candidates
  const size_t shared = C > 1 && a.max_blocks > 2 * chunk_cap ? a.max_blocks : 2 * chunk_cap;
  const size_t smem = (shared + (kRows + 1) * chunk_cap) * 4;
  if (smem > 8 * 1024) {  // with the static part it may be more than a kernel gets unasked
    const cudaError_t e = cudaFuncSetAttribute(select_blocks_kernel<kWide, kRows>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * (kMaxKeys + (kRows + 1) * kMaxChunk));
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
  return cudaLaunchKernelEx(&cfg, select_blocks_kernel<kWide, kRows>, a, chunk_cap);
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream, int num_sms) {
  const bool wide = a.max_blocks > 32 * kWarpKeys;
  const int64_t single = (int64_t)a.B * a.q_len * a.Hkv;
  if (single == 0) return cudaSuccess;
  // Query rows of a sequence go by twos, which read the summaries once, where the rows alone are too
  // many for the widest clusters. Measured with 8 kv heads (us, by twos and one by one): 2 rows of
  // each of 8 sequences, 1,000 blocks 13.2 and 15.2, 4,000 26.6 and 35.4, 280 10.5 and 9.5; of 32
  // sequences, 280 blocks 17.0 and 21.3, 1,000 29.3 and 39.5; 4 rows of one sequence, 4,000 blocks
  // 14.4 and 14.8.
  const bool pairs = wide && a.q_len > 1 && single * kMaxCluster > 2 * (int64_t)num_sms;
  const int64_t segs = pairs ? (int64_t)a.B * ((a.q_len + 1) / 2) * a.Hkv : single;
  // Cluster width: as wide as a grid of one CTA per SM allows, or two where the rows are long, and
  // enough that a CTA's keys leave room for two CTAs per SM. Measured on GB300 (us for 1, 2, 4, 8
  // CTAs a row): 8 rows of 600 blocks 10.3, 9.7, 8.7, 7.9; 32 of 280 8.7, 8.8, 8.1, 8.5; 32 of 1,000
  // 12.9, 11.6, 10.0, 9.7; 32 of 8,000 -, -, 32, 30; 64 of 2,000 19.9, 15.0, 14.5, 21; 128 of 600
  // 12.7, 13.1, 20, 32; 128 of 2,000 28.8, 25.5, 32, 45; 128 of 8,000 -, -, 102, 118; 512 of 1,000
  // 53, 68, 83, 132.
  int C = 1;
  const int64_t most = (a.max_blocks >= 800 ? 2 : 1) * (int64_t)num_sms;
  while (C < kMaxCluster && (a.max_blocks > kMaxChunk * C || segs * 2 * C <= most)) C *= 2;
  if (pairs) return launch_select_n<true, 2>(a, C, segs, stream);
  if (wide) return launch_select_n<true, 1>(a, C, segs, stream);
  return launch_select_n<false, 1>(a, 1, segs, stream);
}

}  // namespace pkv
