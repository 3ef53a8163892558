// The 4-bit cache's quantising write and widening read (fp4.cuh has the format). The caches
// are head-major, [num_blocks, H_kv, block_size, 64] codes and [.., 8] scales, so that the
// 128 rows that one tile of the decode reads are one contiguous piece of each array.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "fast_divide.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {

// Where the rows of a call lie: item w (row order token, side, head; eight lanes each) and its place.
struct Fp4Row {
  int64_t t, row;  // token; row of the caches
  int h;
  bool is_v, bad;
  int32_t slot;
  __device__ __forceinline__ Fp4Row(const KvFp4Args& a, uint32_t w) {
    const uint32_t ts = a.heads.divide(w);
    h = (int)(w - ts * a.hkv);
    t = ts >> 1;
    is_v = ts & 1;
    slot = __ldg(a.slots + t);
    bad = (int64_t)slot >= a.num_blocks * a.block_size;
    const uint32_t blk = a.block.divide((uint32_t)slot);  // (of no use for a slot that is bad or negative)
    row = ((int64_t)blk * a.hkv + h) * a.block_size + ((uint32_t)slot - blk * a.block_size);
  }
};

// kv_cache_write_fp4: eight lanes per row of 128 values, 16 values and so one scale per lane:
// the largest magnitude, the scale and the codes need no other lane. A row is 256 bytes read
// (two 16-byte loads a lane), 64 + 8 written.
// Roofline: HBM; 328 bytes per row (+ 4 of slot per token). Measured on GB300: 131,071 tokens of 8 heads
// in slot order 116 us, 87 % of the copy rate, 16,001 tokens 16.7 us (22.4 with divisions by the head
// count and the block size and IEEE quotients).
__global__ void __launch_bounds__(256) kv_write_fp4_kernel(const __grid_constant__ KvFp4Args a,
                                                           const uint16_t* __restrict__ k,
                                                           const uint16_t* __restrict__ v, int64_t k_stride,
                                                           int64_t v_stride) {
  pdl_wait_then_launch();
  const int c = threadIdx.x & 7;
  for (uint32_t w = blockIdx.x * 32 + (threadIdx.x >> 3); w < a.items; w += gridDim.x * 32) {
    const Fp4Row r(a, w);
    if (r.slot < 0) continue;
    if (r.bad) {
      if (c == 0 && !r.is_v && r.h == 0) flag_status(a.dev_status, PKV_DEV_BAD_SLOT);
      continue;
    }
    const uint16_t* src = (r.is_v ? v + r.t * v_stride : k + r.t * k_stride) + r.h * 128 + c * 16;
    const uint4 r0 = ld_nc_v4(src), r1 = ld_nc_v4(src + 8);
    const uint32_t x[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
    uint32_t top = 0;  // magnitudes in bf16's order, as pairs of 16-bit integers
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxs2(top, x[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    uint32_t scale = fp4::kNanScale;
    uint2 code = make_uint2(0, 0);
    if (top < 0x7f80) {  // neither an infinity nor a NaN among them
      scale = fp4::scale_byte(__uint_as_float(top << 16));
      code = fp4::quantise(x, scale);
    }
    reinterpret_cast<uint2*>((r.is_v ? a.v_cache : a.k_cache) + r.row * fp4::kCodeBytes)[c] = code;
    ((r.is_v ? a.v_scale : a.k_scale) + r.row * fp4::kScaleBytes)[c] = (uint8_t)scale;
  }
}

// kv_cache_read_fp4: the rows back in bf16 (code times scale, exact in fp16 as in bf16), through a
// slot mapping; eight lanes per row, one 8-byte load of codes and two 16-byte stores a lane. A
// negative slot reads as zeros.
// Roofline: HBM; 72 bytes read and 256 written per row (+ 4 of slot per token). Measured on GB300:
// 131,071 tokens of 8 heads 117 us in slot order, 87 % of the copy rate, and 133 us in random order, 75 %:
// the memory's accesses are 64 bytes, of which a scattered row's scales fill 8 (820 MB in all, 90 %).
__global__ void __launch_bounds__(256) kv_read_fp4_kernel(const __grid_constant__ KvFp4Args a,
                                                          uint8_t* __restrict__ k, uint8_t* __restrict__ v) {
  pdl_wait_then_launch();
  const int c = threadIdx.x & 7;
  for (uint32_t w = blockIdx.x * 32 + (threadIdx.x >> 3); w < a.items; w += gridDim.x * 32) {
    const Fp4Row r(a, w);
    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r.bad) {
      if (c == 0 && !r.is_v && r.h == 0) flag_status(a.dev_status, PKV_DEV_BAD_SLOT);
    } else if (r.slot >= 0) {
      const uint2 code =
          __ldg(reinterpret_cast<const uint2*>((r.is_v ? a.v_cache : a.k_cache) + r.row * fp4::kCodeBytes) + c);
      const uint32_t u = __ldg((r.is_v ? a.v_scale : a.k_scale) + r.row * fp4::kScaleBytes + c);
      const uint32_t scale = fp4::scale_dup0(u);
      uint32_t lo[4], hi[4];
      fp4::widen(code.x, lo);
      fp4::widen(code.y, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t y = fp4::mul2(i < 4 ? lo[i & 3] : hi[i & 3], scale);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y));
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
        x[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((r.is_v ? v : k) + (r.t * a.hkv + r.h) * 256 + c * 32);
    dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
    dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

static dim3 prepare(KvFp4Args& a, int num_sms) {
  a.items = (uint32_t)(a.num_tokens * a.hkv * 2);
  a.heads = FastDivide(a.hkv);
  a.block = FastDivide(a.block_size);
  const int64_t blocks = ((int64_t)a.items + 31) / 32, cap = (int64_t)num_sms * 64;
  return dim3((unsigned)(blocks < cap ? blocks : cap));
}

cudaError_t launch_kv_write_fp4(KvFp4Args a, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, cudaStream_t stream, int num_sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  const dim3 grid = prepare(a, num_sms);
  return launch_dependent(kv_write_fp4_kernel, grid, dim3(256), 0, stream, a, (const uint16_t*)k,
                          (const uint16_t*)v, k_stride, v_stride);
}

cudaError_t launch_kv_read_fp4(KvFp4Args a, void* k, void* v, cudaStream_t stream, int num_sms) {
  if (a.num_tokens == 0) return cudaSuccess;
  const dim3 grid = prepare(a, num_sms);
  return launch_dependent(kv_read_fp4_kernel, grid, dim3(256), 0, stream, a, (uint8_t*)k, (uint8_t*)v);
}

}  // namespace pkv
