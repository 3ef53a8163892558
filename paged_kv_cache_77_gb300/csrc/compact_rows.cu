// Eviction: moving the rows that stay to the front of their sequences.
//
// Row i of every sequence and kv head becomes what row kept[i] was, in each of the given caches.
// In place, one CTA moves one slice (bytes of the row) of one cache for one (sequence, kv head),
// from the first row to the last: kept ascends, so a row's place never lies behind the row, and a
// chunk may be written once it and all before it have been read, a barrier between. Chunks are
// read into registers, 16 bytes a thread and load, eight loads in flight. Into blocks of their own
// the rows may move in any order: parts of the list go to CTAs of their own, without barriers and
// with four loads in flight in half as many registers again per SM (16 prompts cut to 2,000 4-bit
// rows 21.1 us with six CTAs per SM and four loads, 26.1 with four and eight; 64 x 2,048 bf16 rows
// in place 215 and 184 us).
// Roofline: HBM; every moved row read once and written once (+ 4 bytes of the list). Measured on GB300:
// 64 sequences x 8 heads x 2,048 bf16 rows in place 184 us, 86 % of the copy rate; the same 4-bit rows 81
// us (8-byte scales and 4-byte sums come and go in sectors of 32).
#include "device_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {
namespace {

constexpr int THREADS = 256, ROWS = 1024;  // rows whose places are looked up at a time

struct Places {
  int64_t from[ROWS], to[ROWS];  // byte offsets in the cache; from -1: the row does not move
};

// Moves rows r0 .. r0 + rows - 1 (their places in `at`), a slice of `pieces` V's each at `base`.
// Every thread has one piece of a row, and of every (THREADS / pieces)-th row.
template <typename V, bool kInPlace>
__device__ __forceinline__ void move_rows(const Places& at, uint8_t* base, int rows, int pieces) {
  constexpr int UNROLL = kInPlace ? 8 : 4;
  const int step = THREADS / pieces, first = (int)threadIdx.x / pieces, piece = (int)threadIdx.x % pieces;
  for (int i0 = 0; i0 < rows; i0 += step * UNROLL) {
    V v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * step + first;
      if (first < step && i < rows && at.from[i] >= 0) v[u] = __ldcg(reinterpret_cast<const V*>(base + at.from[i]) + piece);
    }
    if (kInPlace) __syncthreads();
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * step + first;
      if (first < step && i < rows && at.from[i] >= 0) reinterpret_cast<V*>(base + at.to[i])[piece] = v[u];
    }
  }
}

template <bool kInPlace>
__global__ void __launch_bounds__(THREADS, kInPlace ? 4 : 6) compact_rows_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ Places at;
  pdl_wait_then_launch();
  const CompactCache& t = a.cache[blockIdx.y];
  const int slice = (int)blockIdx.z % a.slices, part = (int)blockIdx.z / a.slices;
  if (slice >= t.slices) return;
  const int b = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv, bs = a.block_size;
  const int32_t* kept = a.kept + (int64_t)blockIdx.x * a.num_keep;
  const int32_t* src_table = a.block_table + (int64_t)b * a.max_blocks;
  const int32_t* dst_table = a.new_table + (int64_t)b * a.new_max_blocks;
  uint8_t* base = t.data + g * t.head_stride + (int64_t)slice * t.slice_bytes;
  const int pieces = min(t.slice_bytes, t.row_bytes - slice * t.slice_bytes) / t.vec;
  const int stop = (int)min((int64_t)(part + 1) * a.part_rows, (int64_t)a.num_keep);
  for (int r0 = part * a.part_rows; r0 < stop; r0 += ROWS) {
    const int rows = min(ROWS, stop - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += THREADS) {
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
      at.from[i] = f;
      at.to[i] = d;
    }
    __syncthreads();
    if (t.vec == 16)
      move_rows<uint4, kInPlace>(at, base, rows, pieces);
    else if (t.vec == 8)
      move_rows<uint2, kInPlace>(at, base, rows, pieces);
    else
      move_rows<uint32_t, kInPlace>(at, base, rows, pieces);
  }
}

}  // namespace

cudaError_t launch_compact_rows(CompactArgs a, cudaStream_t stream, int num_sms) {
  const bool in_place = a.new_table == a.block_table;
  const int64_t lists = (int64_t)a.B * a.Hkv;
  // Four CTAs per SM for the bulk of the bytes, if need be: slices of at least 64 bytes in place,
  // parts of at least 256 rows otherwise.
  int64_t heavy = 0;
  for (int i = 0; i < a.num_caches; ++i) heavy += a.cache[i].row_bytes >= 64;
  const int64_t ctas = lists * (heavy > 0 ? heavy : 1), want = 4 * (int64_t)num_sms;
  int cut = 1, parts = 1;
  if (in_place)
    while (cut < 4 && ctas * cut < want) cut *= 2;
  else
    while (parts < 64 && ctas * parts < want && a.num_keep > 256 * parts) parts *= 2;
  a.slices = 1;
  for (int i = 0; i < a.num_caches; ++i) {
    CompactCache& t = a.cache[i];
    t.vec = t.row_bytes % 16 == 0 ? 16 : t.row_bytes % 8 == 0 ? 8 : 4;
    int pieces = t.row_bytes / t.vec;
    int per = (pieces + cut - 1) / cut;  // pieces of a slice: 64 bytes at least, a thread each
    if (per * t.vec < 64) per = (64 + t.vec - 1) / t.vec;
    if (per > pieces) per = pieces;
    if (per > THREADS) per = THREADS;
    t.slice_bytes = per * t.vec;
    t.slices = (pieces + per - 1) / per;
    a.slices = t.slices > a.slices ? t.slices : a.slices;
  }
  a.part_rows = (a.num_keep + parts - 1) / parts;
  const dim3 grid((unsigned)lists, (unsigned)a.num_caches, (unsigned)(a.slices * parts));
  return launch_dependent(in_place ? compact_rows_kernel<true> : compact_rows_kernel<false>, grid, dim3(THREADS), 0,
                          stream, a);
}

}  // namespace pkv
