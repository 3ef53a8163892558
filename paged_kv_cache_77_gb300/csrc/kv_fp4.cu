// The 4-bit cache's quantising write and widening read (fp4.cuh has the format). The caches
// are head-major, [num_blocks, H_kv, block_size, 64] codes and [.., 8] scales, so that the
// 128 rows that one tile of the decode reads are one contiguous piece of each array.
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "fp4.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {

// kv_cache_write_fp4: eight lanes per row of 128 values, 16 values and so one scale per lane:
// the largest magnitude, the scale and the codes need no other lane. A row is 256 bytes read
// (two 16-byte loads a lane), 64 + 8 written.
// Roofline: HBM; 328 bytes per row (+ 4 of slot per token).
__global__ void __launch_bounds__(256) kv_write_fp4_kernel(
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, uint8_t* __restrict__ k_scale,
    uint8_t* __restrict__ v_scale, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
    int64_t k_stride, int64_t v_stride, const int32_t* __restrict__ slots, int64_t num_tokens,
    int64_t num_slots, int hkv, int block_size, int* dev_status) {
  pdl_wait_then_launch();
  const int c = threadIdx.x & 7;
  const int64_t rows = num_tokens * hkv * 2;
  for (int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3; w < rows;
       w += (int64_t)gridDim.x * 32) {
    // Row order (token, side, head).
    const int64_t ts = w / hkv;
    const int h = (int)(w - ts * hkv);
    const int64_t t = ts >> 1;
    const bool is_v = ts & 1;
    const int32_t slot = __ldg(slots + t);
    if (slot < 0) continue;
    if ((int64_t)slot >= num_slots) {
      if (c == 0 && !is_v && h == 0) flag_status(dev_status, PKV_DEV_BAD_SLOT);
      continue;
    }
    const uint16_t* src = (is_v ? v + t * v_stride : k + t * k_stride) + h * 128 + c * 16;
    const uint4 r0 = ld_nc_v4(src), r1 = ld_nc_v4(src + 8);
    const uint32_t u[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
    float x[16], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf16lo(u[i]);
      x[2 * i + 1] = bf16hi(u[i]);
      amax = max_nan(amax, max_nan(abs_ieee(x[2 * i]), abs_ieee(x[2 * i + 1])));
    }
    uint32_t scale = fp4::kNanScale;
    uint2 code = make_uint2(0, 0);
    if (amax < INFINITY) {  // false for NaN too
      scale = fp4::scale_byte(amax);
      code = fp4::quantise(x, scale);
    }
    const int64_t blk = slot / block_size, off = slot - blk * block_size;
    const int64_t row = (blk * hkv + h) * block_size + off;
    reinterpret_cast<uint2*>((is_v ? v_cache : k_cache) + row * fp4::kCodeBytes)[c] = code;
    ((is_v ? v_scale : k_scale) + row * fp4::kScaleBytes)[c] = (uint8_t)scale;
  }
}

// kv_cache_read_fp4: the rows back in bf16 (code times scale, exact), through a slot mapping;
// eight lanes per row, one 8-byte load of codes and two 16-byte stores a lane. A negative
// slot reads as zeros.
// Roofline: HBM; 72 bytes read and 256 written per row (+ 4 of slot per token).
__global__ void __launch_bounds__(256) kv_read_fp4_kernel(
    uint8_t* __restrict__ k, uint8_t* __restrict__ v, const uint8_t* __restrict__ k_cache,
    const uint8_t* __restrict__ v_cache, const uint8_t* __restrict__ k_scale,
    const uint8_t* __restrict__ v_scale, const int32_t* __restrict__ slots, int64_t num_tokens,
    int64_t num_slots, int hkv, int block_size, int* dev_status) {
  pdl_wait_then_launch();
  const int c = threadIdx.x & 7;
  const int64_t rows = num_tokens * hkv * 2;
  for (int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3; w < rows;
       w += (int64_t)gridDim.x * 32) {
    const int64_t ts = w / hkv;
    const int h = (int)(w - ts * hkv);
    const int64_t t = ts >> 1;
    const bool is_v = ts & 1;
    const int32_t slot = __ldg(slots + t);
    uint32_t r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if ((int64_t)slot >= num_slots) {
      if (c == 0 && !is_v && h == 0) flag_status(dev_status, PKV_DEV_BAD_SLOT);
    } else if (slot >= 0) {
      const int64_t blk = slot / block_size, off = slot - blk * block_size;
      const int64_t row = (blk * hkv + h) * block_size + off;
      const uint2 code =
          __ldg(reinterpret_cast<const uint2*>((is_v ? v_cache : k_cache) + row * fp4::kCodeBytes) + c);
      const uint32_t u = __ldg((is_v ? v_scale : k_scale) + row * fp4::kScaleBytes + c);
      const float s = fp4::scale_value(u);
      uint32_t f[8];
      fp4::widen(code.x, *reinterpret_cast<uint32_t(*)[4]>(f));
      fp4::widen(code.y, *reinterpret_cast<uint32_t(*)[4]>(f + 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(mul_ieee(x.x, s), mul_ieee(x.y, s));
        r[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * hkv + h) * 256 + c * 32);
    dst[0] = make_uint4(r[0], r[1], r[2], r[3]);
    dst[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

static int64_t grid_of(int64_t rows, int num_sms) {
  const int64_t blocks = (rows + 31) / 32, cap = (int64_t)num_sms * 64;
  return blocks < cap ? blocks : cap;
}

cudaError_t launch_kv_write_fp4(const KvFp4Args& a, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, cudaStream_t stream, int num_sms) {
  const int64_t rows = a.num_tokens * a.hkv * 2;
  if (rows == 0) return cudaSuccess;
  return launch_dependent(kv_write_fp4_kernel, dim3((unsigned)grid_of(rows, num_sms)), dim3(256), 0, stream,
                          a.k_cache, a.v_cache, a.k_scale, a.v_scale, (const uint16_t*)k,
                          (const uint16_t*)v, k_stride, v_stride, a.slots, a.num_tokens,
                          a.num_blocks * a.block_size, a.hkv, a.block_size, a.dev_status);
}

cudaError_t launch_kv_read_fp4(const KvFp4Args& a, void* k, void* v, cudaStream_t stream, int num_sms) {
  const int64_t rows = a.num_tokens * a.hkv * 2;
  if (rows == 0) return cudaSuccess;
  return launch_dependent(kv_read_fp4_kernel, dim3((unsigned)grid_of(rows, num_sms)), dim3(256), 0, stream,
                          (uint8_t*)k, (uint8_t*)v, (const uint8_t*)a.k_cache, (const uint8_t*)a.v_cache,
                          (const uint8_t*)a.k_scale, (const uint8_t*)a.v_scale, a.slots, a.num_tokens,
                          a.num_blocks * a.block_size, a.hkv, a.block_size, a.dev_status);
}

}  // namespace pkv
