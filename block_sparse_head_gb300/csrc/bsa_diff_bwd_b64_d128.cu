// Backward kernels of differential attention for block 64, head dim 128.
#include "bsa_diff_bwd_kernel.cuh"

namespace bsa {

cudaError_t launch_diff_bwd_b64_d128(bool split, bool kv, const DiffBwdParams& p,
                                   const CUtensorMap& a, const CUtensorMap& b,
                                   const CUtensorMap& x, const CUtensorMap& y, int grid,
                                   cudaStream_t stream) {
  if (split)
    return kv ? launch_diff_bwd<64, 128, true, true>(p, a, b, x, y, grid, stream)
              : launch_diff_bwd<64, 128, true, false>(p, a, b, x, y, grid, stream);
  return kv ? launch_diff_bwd<64, 128, false, true>(p, a, b, x, y, grid, stream)
            : launch_diff_bwd<64, 128, false, false>(p, a, b, x, y, grid, stream);
}

}  // namespace bsa
