// Self-tests.
//
// The kernels' failure path: every wait on an mbarrier inside the
// attention kernels is bounded, and a wait that gives up sets PKV_DEV_TIMEOUT in the
// caller's status word and lets the kernel wind down instead of hanging the GPU. This
// kernel waits, with the same wait routines, on an mbarrier that nothing completes,
// so that a test can watch that path run out and check the status and that the CUDA
// context is still usable afterwards. Nothing here faults or spins without a limit.
//
// The bf16 matrix products whose error the block selection bounds: the same products, handed
// out for a test to compare with 64 bits.
#include "device_common.cuh"
#include "launch.h"
#include "mma_bf16.cuh"
#include "tc_ptx.cuh"

namespace pkv {

__global__ void __launch_bounds__(64) bounded_wait_kernel(int* dev_status) {
  using namespace tc;
  __shared__ __align__(8) uint64_t bar;  // initialised with one expected arrival that never comes
  const uint32_t b = smem_u32(&bar);
  if (threadIdx.x == 0) {
    mbar_init(b, 1);
    fence_mbar_init();
  }
  __syncthreads();
  bool ok = true;
  // Phase 0 never completes: the spinning wait (issuing threads) and the sleeping wait
  // (producer threads) each give up after their cycle limit.
  if (threadIdx.x == 0) ok = mbar_wait(b, 0);
  if (threadIdx.x == 32) ok = mbar_wait_sleepy(b, 0);
  if (!ok) flag_status(dev_status, PKV_DEV_TIMEOUT);
}

cudaError_t launch_bounded_wait(int* dev_status, cudaStream_t stream) {
  bounded_wait_kernel<<<1, 64, 0, stream>>>(dev_status);
  return cudaGetLastError();
}

// d[i] = a[i] b[i]: a [n, 16, 16] by rows, b [n, 16, 8] by columns, d [n, 16, 8] by rows; a warp each.
__global__ void __launch_bounds__(32) bf16_products_kernel(float* __restrict__ d, const uint32_t* __restrict__ a,
                                                           const uint32_t* __restrict__ b) {
  const int i = threadIdx.x >> 2, c = threadIdx.x & 3;
  a += (int64_t)blockIdx.x * 128;  // (pairs of elements)
  b += (int64_t)blockIdx.x * 64;
  d += (int64_t)blockIdx.x * 128;
  float x[4];
  mma16816(x, a[8 * i + c], a[8 * (i + 8) + c], a[8 * i + c + 4], a[8 * (i + 8) + c + 4], b[8 * i + c],
           b[8 * i + c + 4]);
  for (int k = 0; k < 4; ++k) d[8 * (i + 8 * (k >> 1)) + 2 * c + (k & 1)] = x[k];
}

cudaError_t launch_bf16_products(float* d, const void* a, const void* b, int n, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  bf16_products_kernel<<<n, 32, 0, stream>>>(d, (const uint32_t*)a, (const uint32_t*)b);
  return cudaGetLastError();
}

}  // namespace pkv
