// bsa_cache_append.cu -- writes new keys and values into the 8-bit cache.
//
// The new tokens of one page are a run of consecutive tokens of the call.  Per run, head
// and side (K or V): s = max(scale kept, scale_for(max |x|)), the kept scale counting only
// when the page keeps tokens before the run; kept numbers become rn(y * s_old / s), new
// ones rn(x / s).  Both rounds are to 8 bits, once; scale_for explains the power of two.
//
// One CTA per (token, head); the CTA of a run's first token does the run, the others leave.
#include "bsa_cache.cuh"
#include "bsa_internal.h"

namespace bsa {

namespace {

constexpr int kThreads = 128;

template <class A, class C, int D>
__global__ void __launch_bounds__(kThreads) bsa_cache_append_kernel(const CacheAppendParams p) {
  const int t = blockIdx.x, h = blockIdx.y;
  const int slot = p.slots[t], pid = slot >> p.page_shift;
  if (pid < 0 || pid >= p.n_pages) return;
  if (t > 0 && (p.slots[t - 1] >> p.page_shift) == pid) return;  // not the run's first
  int t1 = t + 1;
  while (t1 < p.T && (p.slots[t1] >> p.page_shift) == pid) ++t1;
  const int page = 1 << p.page_shift, start = slot & (page - 1);
  __shared__ float s_max[kThreads / 32];
  constexpr int HD = D / 2;  // pairs of a token
  for (int side = 0; side < 2; ++side) {
    const A* x = static_cast<const A*>(p.x[side]) + h * p.head_stride[side];
    const int64_t tile = static_cast<int64_t>(pid) * p.heads + h;
    uint16_t* cache = static_cast<uint16_t*>(p.cache[side]) + tile * page * HD;
    float amax = 0.f;
    for (int i = threadIdx.x; i < (t1 - t) * HD; i += kThreads) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          x + (t + i / HD) * p.token_stride[side] + 2 * (i % HD));
      const float2 f = act_to_float2<A>(w);
      if (isfinite(f.x)) amax = fmaxf(amax, fabsf(f.x));
      if (isfinite(f.y)) amax = fmaxf(amax, fabsf(f.y));
    }
    for (int n = 16; n >= 1; n /= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, n));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float was = start > 0 ? p.scale[side][tile] : 0.f;
    const float now = fmaxf(was, scale_for<C>(amax));
    __syncthreads();
    if (threadIdx.x == 0) p.scale[side][tile] = now;
    if (start > 0 && now != was) {
      const float ratio = was / now;
      for (int i = threadIdx.x; i < start * HD; i += kThreads) {
        const float2 y = stored_to_float2<C>(cache[i]);
        cache[i] = static_cast<uint16_t>(float2_to_stored<C>(y.x * ratio, y.y * ratio));
      }
    }
    const float inv = 1.f / now;  // exact: a power of two
    for (int i = threadIdx.x; i < (t1 - t) * HD; i += kThreads) {
      const int u = t + i / HD;
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(x + u * p.token_stride[side] + 2 * (i % HD));
      const float2 f = act_to_float2<A>(w);
      cache[(p.slots[u] & (page - 1)) * HD + i % HD] =
          static_cast<uint16_t>(float2_to_stored<C>(f.x * inv, f.y * inv));
    }
  }
}

template <class A, class C>
cudaError_t launch(int d, const CacheAppendParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(p.heads));
  if (d == 128) bsa_cache_append_kernel<A, C, 128><<<grid, kThreads, 0, stream>>>(p);
  else bsa_cache_append_kernel<A, C, 64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(int d, int dtype, int cache_dtype, const CacheAppendParams& p,
                                cudaStream_t stream) {
  if (dtype == BSA_BF16)
    return cache_dtype == BSA_E4M3 ? launch<__nv_bfloat16, E4M3>(d, p, stream)
                                   : launch<__nv_bfloat16, Int8>(d, p, stream);
  return cache_dtype == BSA_E4M3 ? launch<__half, E4M3>(d, p, stream)
                                 : launch<__half, Int8>(d, p, stream);
}

}  // namespace bsa
