// Tile kernels over an int8 cache, head dim 64.
#include "bsa_cache_tile.cuh"

namespace bsa {

cudaError_t launch_cache_tile_int8_d64(bool fp16, const CacheFwdParams& p, void* workspace,
                                       int sms, cudaStream_t stream) {
  return fp16 ? launch_tile<__half, Int8, 64, false>(p, workspace, sms, stream)
              : launch_tile<__nv_bfloat16, Int8, 64, false>(p, workspace, sms, stream);
}

}  // namespace bsa
