// Tile kernels over an e4m3 cache, head dim 128.
#include "bsa_cache_tile.cuh"

namespace bsa {

cudaError_t launch_cache_tile_e4m3_d128(bool fp16, const CacheFwdParams& p, void* workspace,
                                       int sms, cudaStream_t stream) {
  return fp16 ? launch_tile<__half, E4M3, 128, false>(p, workspace, sms, stream)
              : launch_tile<__nv_bfloat16, E4M3, 128, false>(p, workspace, sms, stream);
}

}  // namespace bsa
