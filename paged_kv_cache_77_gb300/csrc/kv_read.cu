// kv_cache_read_fp8: rows of the FP8 cache widened back to bf16, value = code * scale (one
// fp32 product, rounded to nearest even), gathered through a slot mapping: the way a
// quantised prefix reaches the prefill attention, which reads bf16. Eight lanes per row of
// 128 codes; a lane widens 16 codes (one 16-byte load, two 16-byte stores that fill one
// 32-byte sector). A negative slot reads as zeros.
// Roofline: HBM; per row 128 B codes + 4 B scale read + 256 B written (+ 4 B slot per token).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "ieee_math.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace pkv {

__global__ void __launch_bounds__(256) kv_read_fp8_kernel(
    uint8_t* __restrict__ k, uint8_t* __restrict__ v, const uint8_t* __restrict__ k_cache,
    const uint8_t* __restrict__ v_cache, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, const int32_t* __restrict__ slots, int64_t num_tokens,
    int64_t num_slots, int hkv, int block_size, int* dev_status) {
  pdl_wait_then_launch();
  const int c = threadIdx.x & 7;
  const int64_t rows = num_tokens * hkv * 2;
  for (int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3; w < rows;
       w += (int64_t)gridDim.x * 32) {
    // Row order (token, side, head): both sides of a token write whole lines.
    const int64_t ts = w / hkv;
    const int h = (int)(w - ts * hkv);
    const int64_t t = ts >> 1;
    const bool is_v = ts & 1;
    const int32_t slot = __ldg(slots + t);
    uint4 o0 = make_uint4(0, 0, 0, 0), o1 = o0;
    if ((int64_t)slot >= num_slots) {
      if (c == 0 && !is_v && h == 0) flag_status(dev_status, PKV_DEV_BAD_SLOT);
    } else if (slot >= 0) {
      const int64_t blk = slot / block_size, off = slot - blk * block_size;
      const uint4 code = ld_nc_v4((is_v ? v_cache : k_cache) + ((int64_t)slot * hkv + h) * 128 + c * 16);
      const float scale = __ldg((is_v ? v_scale : k_scale) + (blk * hkv + h) * block_size + off);
      const uint32_t u[4] = {code.x, code.y, code.z, code.w};
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
        const __nv_bfloat162 b = __floats2bfloat162_rn(mul_ieee(f.x, scale), mul_ieee(f.y, scale));
        r[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      o0 = make_uint4(r[0], r[1], r[2], r[3]);
      o1 = make_uint4(r[4], r[5], r[6], r[7]);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * hkv + h) * 256 + c * 32);
    dst[0] = o0;
    dst[1] = o1;
  }
}

cudaError_t launch_kv_read_fp8(void* k, void* v, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* slots,
                               int64_t num_tokens, int64_t num_blocks, int block_size, int hkv,
                               int* dev_status, cudaStream_t stream, int num_sms) {
  const int64_t rows = num_tokens * hkv * 2;
  if (rows == 0) return cudaSuccess;
  int64_t blocks = (rows + 31) / 32;
  // Many small CTAs, so that an SM's loads and stores overlap across them: 131,071 tokens of 8
  // heads in random order take 129.4 us on GB300 with up to 64 CTAs per SM of grid (93 % of
  // the copy rate, 98 % with the 32-byte sectors that the scattered 4-byte scales come in),
  // 153 us with 8. Two or four rows per lane at a time measured 135 to 180 us.
  const int64_t cap = (int64_t)num_sms * 64;
  if (blocks > cap) blocks = cap;
  return launch_dependent(kv_read_fp8_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, (uint8_t*)k,
                          (uint8_t*)v, (const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale,
                          slots, num_tokens, num_blocks * block_size, hkv, block_size, dev_status);
}

}  // namespace pkv
