// Eviction: which rows of a sequence stay, and moving them to the front.
#include "device_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {
namespace {

// --------------------------------------------------------------------------------- select_rows
// For each sequence and kv head the num_keep positions with the largest weights, ascending: a
// radix search for the weight of the last one (digits of 11, 11 and 10 bits of the weights'
// order-preserving integers, histograms in shared memory), then one pass that counts and one
// that writes, each warp over its own run of positions. The first num_sink and the last
// num_recent positions are taken without being ranked.
constexpr int SEL_THREADS = 1024, SEL_WARPS = SEL_THREADS / 32, SEL_BINS = 2048;

// Whole numbers in the order of weights given by their bits: -0 equals 0, NaN is above all. 0 is
// left for rows of bad blocks. (The weights are read as integers: as floats, the compiler may
// turn the tests below into comparisons that take subnormals for zero.)
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if ((u & 0x7fffffffu) == 0) return 0x80000000u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(SEL_THREADS) select_rows_kernel(const __grid_constant__ SelectRowsArgs a) {
  __shared__ int hist[SEL_BINS];
  __shared__ int wsum[SEL_WARPS], wsum2[SEL_WARPS];
  __shared__ int pick_bin, pick_left;
  pdl_wait_then_launch();
  const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.max_blocks * a.block_size;
  const int raw = __ldg(a.seq_lens + b), n = clamp_len(raw, cap);
  if (n != raw && g == 0 && tid == 0) flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
  int32_t* out = a.out + (int64_t)blockIdx.x * a.num_keep;
  if (n <= a.num_keep) {
    for (int i = tid; i < a.num_keep; i += SEL_THREADS) out[i] = i < n ? i : -1;
    return;
  }
  const int lo = a.num_sink, hi = n - a.num_recent;  // ranked: [lo, hi)
  const int want = a.num_keep - a.num_sink - a.num_recent;
  for (int i = tid; i < a.num_sink; i += SEL_THREADS) out[i] = i;
  for (int i = tid; i < a.num_recent; i += SEL_THREADS) out[a.num_keep - a.num_recent + i] = hi + i;
  if (want == 0) return;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  auto key_at = [&](int pos) -> uint32_t {
    const int blk = __ldg(table + pos / a.block_size);
    if (blk < 0 || (int64_t)blk >= a.num_blocks) {
      flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
      return 0;
    }
    return weight_key(__ldg(reinterpret_cast<const uint32_t*>(a.weights) + ((int64_t)blk * a.Hkv + g) * a.block_size + pos % a.block_size));
  };
  uint32_t prefix = 0;
  int left = want;  // rows still to take among those that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < SEL_BINS; i += SEL_THREADS) hist[i] = 0;
    __syncthreads();
    for (int pos = lo + tid; pos < hi; pos += SEL_THREADS) {
      const uint32_t k = key_at(pos);
      if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    // Bins from the top: thread t holds bins 2046 - 2t and 2047 - 2t.
    const int x = hist[2047 - 2 * tid], y = hist[2046 - 2 * tid];
    int incl = x + y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < warp; ++i) before += wsum[i];
    incl += before;
    const int excl = incl - x - y;
    if (excl < left && left <= incl) {
      const bool upper = left <= excl + x;
      pick_bin = upper ? 2047 - 2 * tid : 2046 - 2 * tid;
      pick_left = left - (upper ? excl : excl + x);
    }
    __syncthreads();
    prefix = pass == 2 ? prefix << 10 | pick_bin : prefix << 11 | pick_bin;
    left = pick_left;
  }
  // prefix: the weight of the last row taken; `left` rows of exactly that weight go, lowest first.
  const int span = ((hi - lo + SEL_WARPS - 1) / SEL_WARPS + 31) & ~31;
  const int p0 = lo + warp * span, p1 = min(p0 + span, hi);
  int above = 0, equal = 0;
  for (int pos = p0 + lane; pos < p1; pos += 32) {
    const uint32_t k = key_at(pos);
    above += k > prefix;
    equal += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    wsum[warp] = above;
    wsum2[warp] = equal;
  }
  __syncthreads();
  int at = a.num_sink, eq = 0;  // rows written and rows of the border weight before this warp's
  for (int i = 0; i < warp; ++i) {
    at += wsum[i];
    eq += wsum2[i];
  }
  at += min(eq, left);
  for (int base = p0; base < p1; base += 32) {
    const int pos = base + lane;
    const uint32_t k = pos < p1 ? key_at(pos) : 0;
    const bool is_eq = pos < p1 && k == prefix;
    const unsigned eqs = __ballot_sync(0xffffffffu, is_eq);
    const bool take = pos < p1 && (k > prefix || (is_eq && eq + __popc(eqs & ((1u << lane) - 1)) < left));
    const unsigned takes = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(takes & ((1u << lane) - 1))] = pos;
    at += __popc(takes);
    eq += __popc(eqs);
  }
}

// -------------------------------------------------------------------------------- compact_rows
// Row i of every sequence and kv head becomes what row kept[i] was, in each of the given caches.
// One CTA moves one slice of the rows of one cache for one (sequence, kv head), from the first
// row to the last: kept ascends, so a row's place never lies behind the row, and a chunk may be
// written once it and all before it have been read (a barrier between), even in place.
constexpr int CMP_THREADS = 256, CMP_UNROLL = 8, CMP_ROWS = 1024;

template <typename V>
__global__ void __launch_bounds__(CMP_THREADS) compact_rows_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int64_t from[CMP_ROWS], to[CMP_ROWS];  // rows in units of (block, place), -1: skip
  pdl_wait_then_launch();
  const CompactCache& t = a.cache[blockIdx.y];
  if (t.vec != (int)sizeof(V) || (int)blockIdx.z >= t.slices) return;
  const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv, tid = threadIdx.x;
  const int32_t* kept = a.kept + (int64_t)blockIdx.x * a.num_keep;
  const int32_t* src_table = a.block_table + (int64_t)b * a.max_blocks;
  const int32_t* dst_table = a.new_table + (int64_t)b * a.new_max_blocks;
  uint8_t* base = t.data + g * t.head_stride + (int64_t)blockIdx.z * t.slice_bytes;
  const int pieces = t.slice_bytes / (int)sizeof(V);
  const int bs = a.block_size;
  for (int r0 = 0; r0 < a.num_keep; r0 += CMP_ROWS) {
    const int rows = min(CMP_ROWS, a.num_keep - r0);
    __syncthreads();
    for (int i = tid; i < rows; i += CMP_THREADS) {
      const int src = __ldg(kept + r0 + i), dst = r0 + i;
      int64_t f = -1, d = -1;
      if (src >= 0) {
        if (src / bs >= a.max_blocks || dst / bs >= a.new_max_blocks) {
          flag_status(a.dev_status, PKV_DEV_BAD_LENGTH);
        } else {
          const int sb = __ldg(src_table + src / bs), db = __ldg(dst_table + dst / bs);
          if (sb < 0 || (int64_t)sb >= a.num_blocks || db < 0 || (int64_t)db >= a.num_blocks) {
            flag_status(a.dev_status, PKV_DEV_BAD_BLOCK);
          } else {
            f = sb * t.block_stride + (src % bs) * t.row_stride;
            d = db * t.block_stride + (dst % bs) * t.row_stride;
            if (f == d) f = -1;
          }
        }
      }
      from[i] = f;
      to[i] = d;
    }
    __syncthreads();
    const int items = rows * pieces;
    for (int x0 = 0; x0 < items; x0 += CMP_THREADS * CMP_UNROLL) {
      V v[CMP_UNROLL];
#pragma unroll
      for (int u = 0; u < CMP_UNROLL; ++u) {
        const int x = x0 + u * CMP_THREADS + tid, i = x / pieces;
        if (x < items && from[i] >= 0)
          v[u] = __ldcg(reinterpret_cast<const V*>(base + from[i]) + (x - i * pieces));
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < CMP_UNROLL; ++u) {
        const int x = x0 + u * CMP_THREADS + tid, i = x / pieces;
        if (x < items && from[i] >= 0) reinterpret_cast<V*>(base + to[i])[x - i * pieces] = v[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_select_rows(const SelectRowsArgs& a, cudaStream_t stream) {
  return launch_dependent(select_rows_kernel, dim3(a.B * a.Hkv), dim3(SEL_THREADS), 0, stream, a);
}

cudaError_t launch_compact_rows(CompactArgs a, cudaStream_t stream) {
  int slices = 1;
  bool has[3] = {false, false, false};
  for (int i = 0; i < a.num_caches; ++i) {
    CompactCache& t = a.cache[i];
    t.vec = t.row_bytes % 16 == 0 ? 16 : t.row_bytes % 8 == 0 ? 8 : 4;
    t.slice_bytes = t.row_bytes % 64 == 0 ? 64 : t.row_bytes;
    t.slices = t.row_bytes / t.slice_bytes;
    slices = t.slices > slices ? t.slices : slices;
    has[t.vec == 16 ? 0 : t.vec == 8 ? 1 : 2] = true;
  }
  const dim3 grid(a.B * a.Hkv, a.num_caches, slices), block(CMP_THREADS);
  cudaError_t e = cudaSuccess;
  if (has[0]) e = launch_dependent(compact_rows_kernel<uint4>, grid, block, 0, stream, a);
  if (has[1] && e == cudaSuccess) e = launch_dependent(compact_rows_kernel<uint2>, grid, block, 0, stream, a);
  if (has[2] && e == cudaSuccess) e = launch_dependent(compact_rows_kernel<uint32_t>, grid, block, 0, stream, a);
  return e;
}

}  // namespace pkv
