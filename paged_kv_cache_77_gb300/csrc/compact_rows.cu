// Eviction: moving the rows that stay to the front of their sequences.
#include "device_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {
namespace {

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
