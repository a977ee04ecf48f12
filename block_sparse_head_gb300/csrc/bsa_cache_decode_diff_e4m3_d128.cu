// Decode kernels of differential attention over an e4m3 cache, head dim 128.
#include "bsa_cache_decode.cuh"

namespace bsa {

cudaError_t launch_cache_decode_diff_e4m3_d128(bool fp16, int rows, const CUtensorMap& k,
                                         const CUtensorMap& v, const CacheFwdParams& p,
                                         void* workspace, int sms, cudaStream_t stream) {
  return launch_decode<E4M3, 128, true>(fp16, rows, k, v, p, workspace, sms, stream);
}

}  // namespace bsa
