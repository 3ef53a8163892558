// Device helpers shared by the kernels: bf16 bit handling, cp.async, streaming loads,
// and the balanced tile partition used by every split-KV decode kernel.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_kv.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_nc_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Pairs of fp32 values in one 64-bit register, for the paired fp32 instructions
// (one fma.f32x2 / add.f32x2 does the work of two scalar ones).
__device__ __forceinline__ uint64_t f2pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2unpack(uint64_t v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
  return make_float2(lo, hi);
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Arithmetic that keeps subnormals whatever the build's flags: each result is the IEEE one.
__device__ __forceinline__ float mul_ieee(float a, float b) {
  float r;
  asm("mul.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float add_ieee(float a, float b) {
  float r;
  asm("add.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fma_ieee(float a, float b, float c) {
  float r;
  asm("fma.rn.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float div_ieee(float a, float b) {
  float r;
  asm("div.rn.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Maximum and minimum; a NaN gives way to the other operand.
__device__ __forceinline__ float max_ieee(float a, float b) {
  float r;
  asm("max.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_ieee(float a, float b) {
  float r;
  asm("min.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ double widen_ieee(float a) {
  double r;
  asm("cvt.f64.f32 %0, %1;\n" : "=d"(r) : "f"(a));
  return r;
}

// Maximum of v over the 32 lanes of a full warp (one redux instruction; NaN inputs
// are ignored like fmaxf does).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(v));
  return r;
}

// Programmatic dependent launch. An attention kernel lets the merge kernel that
// follows it on the stream be launched at once; the merge runs its prologue (which
// reads only the call's inputs), then waits for the attention kernel to complete and
// its writes to be visible before it reads the workspace or writes any output.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void pdl_wait_primary() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Launch of a kernel that may start while the previous kernel on the stream is still
// running (it must call pdl_wait_primary() before depending on that kernel).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void flag_status(int* dev_status, int bits) {
  if (dev_status) atomicOr(dev_status, bits);
}

// --------------------------------------------------------------------------
// Balanced split of the decode work.
//
// The work of a decode call is the list of (sequence b, kv head g, live block j)
// tiles, ordered by b, then g, then j. A sequence of length len has live blocks
// [jlo, jhi) with jhi = ceil(len / bs) and, for a window W > 0,
// jlo = floor(max(0, len - W) / bs) (blocks wholly before the window are never
// read). The tiles of one (b, g) form a segment. CTA i of G processes tiles
// [floor(i*T/G), floor((i+1)*T/G)), so every CTA streams the same number of
// blocks (+-1). A maximal run of one CTA's tiles inside one segment is a piece;
// a piece that starts at its segment's first tile stores its partial result in
// slot b*H_kv + g, any other piece in slot B*H_kv + i. A segment whose tiles all
// fall in one CTA is finished by that CTA directly.
// --------------------------------------------------------------------------
struct SeqRange {
  int jlo, n;  // first live block, number of live blocks
};

// Lengths are clamped to [0, max_blocks * bs] so that no table row is indexed past
// its end; the attention kernels flag PKV_DEV_BAD_LENGTH when a clamp happens.
__device__ __forceinline__ int clamp_len(int len, int cap) { return len < 0 ? 0 : (len > cap ? cap : len); }

__device__ __forceinline__ SeqRange live_blocks(int len, int bs, int window) {
  SeqRange r;
  if (len <= 0) {
    r.jlo = 0;
    r.n = 0;
    return r;
  }
  int jhi = (len + bs - 1) / bs;
  int lo = (window > 0 && len > window) ? len - window : 0;
  r.jlo = lo / bs;
  r.n = jhi - r.jlo;
  return r;
}

__device__ __forceinline__ int64_t cta_tile_start(int64_t i, int64_t T, int64_t G) {
  return (i * T) / G;
}

// Cursor over one CTA's tiles. All threads of a CTA walk identical cursors.
struct TileCursor {
  int b, g, j;          // current tile (j relative to jlo)
  int jlo, n;           // live range of sequence b
  int len;              // length of sequence b
  int64_t seg_base;     // global index of tile (b, g, 0)
  int64_t t, t_end;     // current global tile index, end of this CTA's range
};

// The rows whose tiles a decode call walks. Dense attention: one per sequence, reading its
// live blocks in order. Sparse attention: one per query row, reading at most `keep` blocks
// of the row's own list; row r is query r % q_len of sequence r / q_len and sees the first
// len - q_len + 1 + r % q_len positions of it.
struct DenseRows {
  const int* seq_lens;
  int bs, window, cap;
  __device__ __forceinline__ int raw(int b) const { return __ldg(seq_lens + b); }
  __device__ __forceinline__ int len(int b) const { return clamp_len(raw(b), cap); }
  __device__ __forceinline__ SeqRange blocks(int len) const { return live_blocks(len, bs, window); }
};
struct SparseRows {
  const int* seq_lens;
  int bs, q_len, keep, cap;
  __device__ __forceinline__ int raw(int r) const { return __ldg(seq_lens + r / q_len); }
  __device__ __forceinline__ int len(int r) const {
    const int n = clamp_len(raw(r), cap) - q_len + 1 + r % q_len;
    return n > 0 ? n : 0;
  }
  __device__ __forceinline__ SeqRange blocks(int len) const {
    SeqRange s;
    s.jlo = 0;
    s.n = (len + bs - 1) / bs;
    if (s.n > keep) s.n = keep;
    return s;
  }
};

// Sum of live blocks over all rows (one warp, result in every lane).
template <typename Rows>
__device__ __forceinline__ int64_t total_live_blocks(const Rows& rows, int B, int* dev_status) {
  int64_t s = 0;
  for (int b = threadIdx.x & 31; b < B; b += 32) {
    const int raw = rows.raw(b);
    if (clamp_len(raw, rows.cap) != raw && blockIdx.x == 0) flag_status(dev_status, PKV_DEV_BAD_LENGTH);
    s += rows.blocks(rows.len(b)).n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The same over dense rows (the kernels that have no sparse form).
__device__ __forceinline__ int64_t total_live_blocks(const int* seq_lens, int B, int bs, int window,
                                                     int cap, int* dev_status) {
  return total_live_blocks(DenseRows{seq_lens, bs, window, cap}, B, dev_status);
}

// Position the cursor at global tile t (a single thread's scan; B is small).
template <typename Rows>
__device__ inline void cursor_seek(TileCursor& c, const Rows& rows, int B, int Hkv, int64_t t,
                                   int64_t t_end) {
  c.t = t;
  c.t_end = t_end;
  int64_t base = 0;
  c.b = B;
  c.g = 0;
  c.j = 0;
  c.jlo = 0;
  c.n = 0;
  c.len = 0;
  c.seg_base = 0;
  if (t >= t_end) return;
  for (int b = 0; b < B; ++b) {
    int len = rows.len(b);
    SeqRange r = rows.blocks(len);
    int64_t seg = (int64_t)r.n * Hkv;
    if (t < base + seg) {
      int64_t off = t - base;
      c.b = b;
      c.g = (int)(off / r.n);
      c.j = (int)(off % r.n);
      c.jlo = r.jlo;
      c.n = r.n;
      c.len = len;
      c.seg_base = base + (int64_t)c.g * r.n;
      return;
    }
    base += seg;
  }
}

__device__ inline void cursor_seek(TileCursor& c, const int* seq_lens, int B, int Hkv, int bs,
                                   int window, int cap, int64_t t, int64_t t_end) {
  cursor_seek(c, DenseRows{seq_lens, bs, window, cap}, B, Hkv, t, t_end);
}

// Advance to the next tile; returns false when the CTA's range is exhausted.
template <typename Rows>
__device__ inline bool cursor_next(TileCursor& c, const Rows& rows, int B, int Hkv) {
  ++c.t;
  if (c.t >= c.t_end) return false;
  if (++c.j < c.n) return true;
  c.j = 0;
  c.seg_base += c.n;
  if (++c.g < Hkv) return true;
  c.g = 0;
  for (;;) {
    if (++c.b >= B) return false;
    c.len = rows.len(c.b);
    SeqRange r = rows.blocks(c.len);
    c.jlo = r.jlo;
    c.n = r.n;
    if (r.n > 0) return true;
  }
}
__device__ inline bool cursor_next(TileCursor& c, const int* seq_lens, int B, int Hkv, int bs,
                                   int window, int cap) {
  return cursor_next(c, DenseRows{seq_lens, bs, window, cap}, B, Hkv);
}

// First CTA whose range starts at or before tile `t`.
__device__ __forceinline__ int64_t cta_of_tile(int64_t t, int64_t T, int64_t G) {
  return ((t + 1) * G + T - 1) / T - 1;
}

}  // namespace pkv
