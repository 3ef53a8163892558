// Decode over selected blocks on the tcgen05 decode kernel (decode_tc.cuh): every query row
// and kv head brings a list of blocks of its sequence and attends to the visible tokens in
// them. Rows are independent, so q_len rows of a sequence are q_len rows of the kernel.
// Kept apart from decode_tc.cu so that the translation units compile in parallel.
#include "decode_tc.cuh"

namespace pkv {

cudaError_t launch_decode_sparse(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.n_rep) {
    case 1: return launch_tc_n<1, 1, true>(a, stream);
    case 2: return launch_tc_n<2, 1, true>(a, stream);
    case 4: return launch_tc_n<4, 1, true>(a, stream);
    case 8: return launch_tc_n<8, 1, true>(a, stream);
    case 16: return launch_tc_n<16, 1, true>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
