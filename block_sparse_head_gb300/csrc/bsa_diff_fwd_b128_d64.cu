// Forward kernels of differential attention for block 128, head dim 64.
#include "bsa_diff_fwd_kernel.cuh"

namespace bsa {

cudaError_t launch_diff_fwd_b128_d64(bool split, const DiffFwdParams& p, const CUtensorMap& q,
                                   const CUtensorMap& k, const CUtensorMap& v, int grid,
                                   cudaStream_t stream) {
  if (split) return cudaErrorInvalidValue;  // 32 numbers a map: no such tile
  return launch_diff_fwd<128, 64, false>(p, q, k, v, grid, stream);
}

}  // namespace bsa
