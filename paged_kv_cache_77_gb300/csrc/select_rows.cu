// Eviction: the choice of the rows that stay.
//
// For each sequence and kv head the num_keep positions with the largest weights, ascending. The
// border, the weight of the last row taken, is found digit by digit (11, 11 and 10 bits of the
// weights' order-preserving integers): a histogram of the digit over the rows that share the
// digits before, and a scan from the top. Then each warp counts what it takes and, knowing what
// the warps before it take, writes its positions in order. The first num_sink and the last
// num_recent positions are taken without being ranked.
//
// A row (sequence, kv head) is the work of a cluster of 1 to 8 CTAs, each with its own run of
// blocks and, for the digits, its own histogram, which every CTA of the cluster sums up for
// itself through distributed shared memory. A warp's run of blocks is consecutive; it reads
// their weights once, keeps them as integers in shared memory, and reads those that do not fit
// there again, from L2, for each later pass.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32, BS = 128;
constexpr int HELD = 4;          // blocks of a warp in flight
constexpr int MAX_KEPT = 384;    // blocks of a CTA whose keys stay in shared memory
constexpr int MAX_CLUSTER = 8;
constexpr uint32_t ABSENT = 0, BAD = 1;  // keys of positions that are not ranked, and of bad blocks

// Whole numbers in the order of weights given by their bits: -0 equals 0, NaN is above all; the
// least, of -infinity, is 0x7fffff. (The weights are read as integers: as floats, the compiler may
// turn the tests below into comparisons that take subnormals for zero.)
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if ((u & 0x7fffffffu) == 0) return 0x80000000u;
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint4 weight_keys(uint4 w) {
  // Numbers from 0 to infinity, as sums of weights are, need one bit set.
  if (max(max(w.x, w.y), max(w.z, w.w)) <= 0x7f800000u)
    return make_uint4(w.x | 0x80000000u, w.y | 0x80000000u, w.z | 0x80000000u, w.w | 0x80000000u);
  return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
}

struct Shared {
  int hist[3][2048];
  int wsum[WARPS], wabove[WARPS], wequal[WARPS];
  int pick_bin, pick_left, pick_all;
  int above, equal;  // of this CTA
};

__global__ void __launch_bounds__(THREADS, 1) select_rows_kernel(const __grid_constant__ SelectRowsArgs a, int keep_blocks) {
  extern __shared__ uint4 kept_keys[];  // [WARPS][keep_blocks][32]
  __shared__ __align__(16) Shared sh;
  pdl_wait_then_launch();
  const int C = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int row = blockIdx.x / C, b = row / a.Hkv, g = row % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int raw = __ldg(a.seq_lens + b), n = clamp_len(raw, a.max_blocks * BS);
  if (n != raw && g == 0 && rank == 0 && tid == 0) flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  int32_t* out = a.out + (int64_t)row * a.num_keep;
  if (n <= a.num_keep) {
    for (int i = rank * THREADS + tid; i < a.num_keep; i += C * THREADS) out[i] = i < n ? i : -1;
    return;
  }
  const int lo = a.num_sink, hi = n - a.num_recent;  // ranked: [lo, hi)
  for (int i = rank * THREADS + tid; i < a.num_sink; i += C * THREADS) out[i] = i;
  for (int i = rank * THREADS + tid; i < a.num_recent; i += C * THREADS)
    out[a.num_keep - a.num_recent + i] = hi + i;
  int left = a.num_keep - a.num_sink - a.num_recent;  // rows still to take among those at the border
  if (left == 0) return;
  auto sync = [&] {
    if (C == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  };

  // This warp's blocks: `count` from `first` on.
  const int blocks = (hi + BS - 1) / BS, per = (blocks + C * WARPS - 1) / (C * WARPS);
  const int first = (rank * WARPS + warp) * per, count = max(0, min(per, blocks - first));
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks + first;
  uint4* mine = kept_keys + warp * keep_blocks * 32 + lane;
  // The warp's blocks in order, HELD at a time: f(block, its four keys of this lane).
  auto stream = [&](int q, auto&& f) {
    for (; q < count; q += HELD) {
      const int ids = lane < HELD && q + lane < count ? __ldg(table + q + lane) : 0;
      const bool wrong = ids < 0 || (int64_t)ids >= a.num_blocks;
      if (wrong) flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
      const unsigned bad = __ballot_sync(0xffffffffu, wrong);
      uint4 w[HELD];
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const int blk = __shfl_sync(0xffffffffu, ids, i);
        if (q + i < count && !(bad >> i & 1))
          w[i] = __ldg(reinterpret_cast<const uint4*>(a.weights + ((int64_t)blk * a.Hkv + g) * BS) + lane);
      }
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        if (q + i >= count) break;
        uint4 k = bad >> i & 1 ? make_uint4(BAD, BAD, BAD, BAD) : weight_keys(w[i]);
        const int pos = (first + q + i) * BS + 4 * lane;
        if (pos - 4 * lane < lo || pos - 4 * lane + BS > hi) {
          if (pos < lo || pos >= hi) k.x = ABSENT;
          if (pos + 1 < lo || pos + 1 >= hi) k.y = ABSENT;
          if (pos + 2 < lo || pos + 2 >= hi) k.z = ABSENT;
          if (pos + 3 < lo || pos + 3 >= hi) k.w = ABSENT;
        }
        f(q + i, k);
      }
    }
  };
  auto each = [&](auto&& f) {
    const int kept = min(count, keep_blocks);
#pragma unroll 2
    for (int q = 0; q < kept; ++q) f(q, mine[q * 32]);
    if (count > keep_blocks) stream(keep_blocks, f);
  };
  for (int i = tid; i < 3 * 2048 / 4; i += THREADS) reinterpret_cast<int4*>(sh.hist)[i] = make_int4(0, 0, 0, 0);
  __syncthreads();

  uint32_t border = 0;  // its digits so far
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    int* hist = sh.hist[pass];
    if (pass == 0) {
      stream(0, [&](int q, uint4 k) {
        if (q < keep_blocks) mine[q * 32] = k;
        // (Keys that are not ranked count in bin 0, which is put right below.)
        atomicAdd(hist + (k.x >> 21), 1);
        atomicAdd(hist + (k.y >> 21), 1);
        atomicAdd(hist + (k.z >> 21), 1);
        atomicAdd(hist + (k.w >> 21), 1);
      });
    } else {
      const uint32_t base = border << (shift + bits), span = 1u << (shift + bits);
      each([&](int, uint4 k) {
        auto add = [&](uint32_t x) {
          if (x - base < span && x != ABSENT) atomicAdd(hist + (x >> shift & ((1 << bits) - 1)), 1);
        };
        add(k.x);
        add(k.y);
        add(k.z);
        add(k.w);
      });
    }
    sync();
    // Thread t sums the bins 4 (511 - t) .. + 3 over the cluster; the scan runs from the top.
    int4 h = make_int4(0, 0, 0, 0);
    if (tid < 512 && (bits == 11 || tid >= 256)) {
      for (int r = 0; r < C; ++r) {
        const int* from = C == 1 ? hist : cg::this_cluster().map_shared_rank(hist, r);
        const int4 x = reinterpret_cast<const int4*>(from)[511 - tid];
        h = make_int4(h.x + x.x, h.y + x.y, h.z + x.z, h.w + x.w);
      }
    }
    const int sum = h.x + h.y + h.z + h.w;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.wsum[warp] = incl;
    __syncthreads();
    int before = lane < warp ? sh.wsum[lane & (WARPS - 1)] : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    incl += before;
    int rest = left - (incl - sum);  // to take from this thread's bins on
    if (rest > 0 && left <= incl) {
      int bin = 4 * (511 - tid) + 3, size = h.w;
      if (rest > size) {
        rest -= size;
        --bin;
        size = h.z;
        if (rest > size) {
          rest -= size;
          --bin;
          size = h.y;
          if (rest > size) {
            rest -= size;
            --bin;
            size = h.x;
          }
        }
      }
      sh.pick_bin = bin;
      sh.pick_left = rest;
      sh.pick_all = rest == size;
    }
    __syncthreads();
    border = border << bits | (uint32_t)sh.pick_bin;
    left = sh.pick_left;
    if (sh.pick_all && border > 0) {
      // Every row of the bin is taken: the border lies below its least weight.
      border = (border << shift) - 1;
      left = 0;
      break;
    }
    // (What a CTA writes next, the next digit's scan, comes behind that digit's barrier.)
  }

  // `left` rows of exactly the border's weight go, lowest position first.
  int above = 0, equal = 0;
  each([&](int, uint4 k) {
    above += (k.x > border) + (k.y > border) + (k.z > border) + (k.w > border);
    equal += (k.x == border) + (k.y == border) + (k.z == border) + (k.w == border);
  });
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sh.wabove[warp] = above;
    sh.wequal[warp] = equal;
  }
  __syncthreads();
  int at = lane < WARPS ? sh.wabove[lane] : 0, eq = lane < WARPS ? sh.wequal[lane] : 0;
  if (C > 1) {
    if (warp == 0) {
      const int x = __reduce_add_sync(0xffffffffu, at), y = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        sh.above = x;
        sh.equal = y;
      }
    }
    sync();
  }
  if (lane >= warp) at = eq = 0;
  if (C > 1 && lane < rank) {
    at += *cg::this_cluster().map_shared_rank(&sh.above, lane);
    eq += *cg::this_cluster().map_shared_rank(&sh.equal, lane);
  }
  at = __reduce_add_sync(0xffffffffu, at);  // rows above the border, and at it, before this warp's
  eq = __reduce_add_sync(0xffffffffu, eq);
  at += a.num_sink + min(eq, left);
  const unsigned lower = (1u << lane) - 1;
  each([&](int q, uint4 k) {
    unsigned take = (k.x > border) | (k.y > border) << 1 | (k.z > border) << 2 | (k.w > border) << 3;
    const unsigned same = (k.x == border) | (k.y == border) << 1 | (k.z == border) << 2 | (k.w == border) << 3;
    if (__any_sync(0xffffffffu, same)) {
      int rankq = eq;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned all = __ballot_sync(0xffffffffu, same >> j & 1);
        rankq += __popc(all & lower);
        eq += __popc(all);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (same >> j & 1 && rankq++ < left) take |= 1u << j;
    }
    int to = at;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned all = __ballot_sync(0xffffffffu, take >> j & 1);
      to += __popc(all & lower);
      at += __popc(all);
    }
    const int pos = (first + q) * BS + 4 * lane;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (take >> j & 1) out[to++] = pos + j;
  });
  if (C > 1) sync();  // no CTA goes while another may read its shared memory
}

}  // namespace

cudaError_t launch_select_rows(const SelectRowsArgs& a, cudaStream_t stream, int num_sms) {
  const int64_t rows = (int64_t)a.B * a.Hkv;
  // Cluster width: CTAs for every SM where the rows alone are too few, with two blocks or more a
  // warp; two CTAs per SM where the keys of a row do not fit one. Measured on GB300 (us for 1, 2, 4,
  // 8 CTAs a row): 8 rows of 256 blocks 16.0, 13.7, 11.5, 13.8; 16 of 8,192 578, 289, 147, 142; 128
  // of up to 1,024 72, 55, 68, 138; 512 of up to 256 42, 68, 138, 367.
  int C = 1;
  while (C < MAX_CLUSTER && a.max_blocks > 2 * WARPS * C &&
         rows * 2 * C <= (a.max_blocks > MAX_KEPT * C ? 2 : 1) * (int64_t)num_sms)
    C *= 2;
  // Blocks of a warp whose keys stay in shared memory.
  int keep = (a.max_blocks + C * WARPS - 1) / (C * WARPS);
  if (keep > MAX_KEPT / WARPS) keep = MAX_KEPT / WARPS;
  const size_t smem = (size_t)keep * WARPS * BS * 4;
  const cudaError_t e =
      cudaFuncSetAttribute(select_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_KEPT * BS * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(THREADS);
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
  return cudaLaunchKernelEx(&cfg, select_rows_kernel, a, keep);
}

}  // namespace pkv
