// Forward kernels of differential attention for block 128, head dim 128.
#include "bsa_diff_fwd_kernel.cuh"

namespace bsa {

cudaError_t launch_diff_fwd_b128_d128(bool split, const DiffFwdParams& p, const CUtensorMap& q,
                                   const CUtensorMap& k, const CUtensorMap& v, int grid,
                                   cudaStream_t stream) {
  return split ? launch_diff_fwd<128, 128, true>(p, q, k, v, grid, stream)
               : launch_diff_fwd<128, 128, false>(p, q, k, v, grid, stream);
}

}  // namespace bsa
