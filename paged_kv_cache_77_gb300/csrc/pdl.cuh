// Programmatic dependent launch of kernels that read nothing before their wait.
#pragma once

#include "device_common.cuh"

namespace pkv {

// At the top of a kernel launched with launch_dependent: wait for the kernel before on the
// stream, then let the one behind launch. In this order a kernel behind that reads inputs
// before its own wait (the attention merges read the lengths) finds everything that precedes
// this kernel done and visible; the other order would let it overtake the kernel before this.
__device__ __forceinline__ void pdl_wait_then_launch() {
  pdl_wait_primary();
  pdl_launch_dependents();
}

}  // namespace pkv
