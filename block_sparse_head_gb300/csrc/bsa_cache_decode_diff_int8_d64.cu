// Decode kernels of differential attention over an int8 cache, head dim 64.
#include "bsa_cache_decode.cuh"

namespace bsa {

cudaError_t launch_cache_decode_diff_int8_d64(bool fp16, int rows, const CUtensorMap& k,
                                         const CUtensorMap& v, const CacheFwdParams& p,
                                         void* workspace, int sms, cudaStream_t stream) {
  return launch_decode<Int8, 64, true>(fp16, rows, k, v, p, workspace, sms, stream);
}

}  // namespace bsa
