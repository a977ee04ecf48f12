// bsa_cache_append.cu -- writes new keys and values into the 8-bit cache.
//
// The new tokens of one page are a run of consecutive tokens of the call.  Per run, head
// and side (K or V): s = max(scale kept, scale_for(max |x|)), the kept scale counting only
// when the page keeps tokens before the run; kept numbers become rn(y * s_old / s), new
// ones rn(x / s).  Both rounds are to 8 bits, once; scale_for explains the power of two.
//
// Bound: memory (a number is read as 16 bits and written as 8).  A CTA takes CT tokens of one
// head and side and does the runs that begin there, however far they go: a run of up to two
// tokens (a decode step) is a warp's, any other the CTA's, which holds its share of the page in
// registers (at most sixteen 16-byte pieces a thread) between the maximum and the rounding, so
// that the numbers are read once.  CT is 1 for up to kSmallRows rows, where the call is as long
// as one CTA's way (256 tokens of 8 heads one by one: 9.4 us, 7.8 with 16 a CTA; 128: 5.6
// against 7.6), then 16 for up to kMediumRows and for pages of up to 32 tokens (512 one by one:
// 8.0 us, 21 with 64 a CTA), and 64 for long prompts (6,400 tokens in pages of 64: 13 us, 19
// with 16 a CTA), which leaves few CTAs that only see that no run begins in their tokens.
//
// Measured: 16,384 tokens of 8 heads, d = 128, one prompt: 20.1 us, 5.0 TB/s (0.74 of a copy;
// 23.3 before the prefetch, the maxima two numbers at once and CTAs of 128 threads instead of
// 256); 1,000 tokens of 16 heads of 64 in five chunks, pages of 16: 8.0 us (10.6 with 256
// threads); 64 requests a token each: 3.4 us.  The launch and three trips to memory one after
// the other (slots, old scales, numbers) are about 3 us of each.
#include "bsa_cache.cuh"
#include "bsa_internal.h"

#include <type_traits>

namespace bsa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kShortRun = 2;      // tokens of a run that a warp takes
// Token rows (tokens x heads x 2) up to which a CTA takes one token, and 16.
constexpr int kSmallRows = 2048, kMediumRows = 32768;

// Bits of the smallest magnitude that is not finite.
template <class A>
constexpr uint32_t kInfBits = std::is_same<A, __half>::value ? 0x7C00u : 0x7F80u;

// Largest magnitudes of the halves of w and m; NaN where there is one.
template <class A>
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t w) {
  uint32_t r;
  if constexpr (std::is_same<A, __half>::value)
    asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %2;\n\tmax.NaN.f16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  else
    asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  return r;
}
// The same over the finite ones (as bits, which order like the numbers).
template <class A>
__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint32_t w) {
  w &= 0x7FFF7FFFu;
  if ((w & 0xFFFFu) >= kInfBits<A>) w &= 0xFFFF0000u;
  if ((w >> 16) >= kInfBits<A>) w &= 0xFFFFu;
  return __vmaxu2(m, w);
}
template <class A>
__device__ __forceinline__ bool has_nonfinite(uint32_t m) {
  return (m & 0xFFFFu) >= kInfBits<A> || (m >> 16) >= kInfBits<A>;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t m) {
#pragma unroll
  for (int s = 1; s < 32; s *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, s));
  return m;
}
// The larger half of m as a number.
template <class A>
__device__ __forceinline__ float larger(uint32_t m) {
  const float2 f = act_to_float2<A>(m);
  return fmaxf(f.x, f.y);
}

template <class A, class C>
__device__ __forceinline__ uint32_t quantise4(uint32_t a, uint32_t b, float inv) {
  const float2 f = act_to_float2<A>(a), h = act_to_float2<A>(b);
  return float2_to_stored<C>(f.x * inv, f.y * inv) | float2_to_stored<C>(h.x * inv, h.y * inv) << 16;
}

// Rounds `words` words of kept numbers to a grown scale; every `step`-th from `first` on.
template <class C>
__device__ __forceinline__ void rescale(uint32_t* cache, int words, float ratio, int first, int step) {
  for (int i = first; i < words; i += step) {
    const uint32_t w = cache[i];
    const float2 lo = stored_to_float2<C>(w & 0xFFFFu), hi = stored_to_float2<C>(w >> 16);
    cache[i] = float2_to_stored<C>(lo.x * ratio, lo.y * ratio) |
               float2_to_stored<C>(hi.x * ratio, hi.y * ratio) << 16;
  }
}

template <class A, class C, int D, int CT>
__global__ void __launch_bounds__(kThreads) bsa_cache_append_kernel(const CacheAppendParams p) {
  constexpr int NS = (CT + 31) / 32;   // a warp looks at 32 tokens at a time
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
  const bool v = blockIdx.z;
  const int t0 = blockIdx.x * CT, page = 1 << p.page_shift;
  const int64_t stride = v ? p.token_stride[1] : p.token_stride[0];
  const A* const in = static_cast<const A*>(v ? p.x[1] : p.x[0]) + h * (v ? p.head_stride[1] : p.head_stride[0]);
  uint8_t* const out = static_cast<uint8_t*>(v ? p.cache[1] : p.cache[0]);
  float* const scales = v ? p.scale[1] : p.scale[0];
  auto page_of = [&](int t) {  // -1: no such token or page
    if (t < 0 || t >= p.T) return -1;
    const int id = p.slots[t] >> p.page_shift;
    return id < p.n_pages ? id : -1;
  };
  if constexpr (CT > 1) {
    // The chunk's numbers on their way to L2 while the slots are looked at.
    constexpr int LINES = D / 64;  // 128 bytes each, of a token
    for (int i = tid; i < CT * LINES; i += kThreads)
      if (t0 + i / LINES < p.T)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + (t0 + i / LINES) * stride + i % LINES * 64));
  }
  // Every warp looks at the chunk's tokens: which begin a run.
  int pid[NS], before[NS];
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    const int i = 32 * u + lane;
    pid[u] = i < CT ? page_of(t0 + i) : -1;
    before[u] = i < CT ? page_of(t0 + i - 1) : -1;
  }
  const int after = page_of(t0 + CT + lane);
  uint32_t goes_on[NS];
#pragma unroll
  for (int u = 0; u < NS; ++u) goes_on[u] = __ballot_sync(0xffffffffu, pid[u] >= 0 && pid[u] == before[u]);
  __shared__ uint32_t s_max[kWarps];
  int k = 0;  // runs of the chunk so far
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    for (uint32_t heads = __ballot_sync(0xffffffffu, pid[u] >= 0 && pid[u] != before[u]); heads != 0;
         heads &= heads - 1, ++k) {
      const int i = __ffs(heads) - 1, t = t0 + 32 * u + i;
      const int id = __shfl_sync(0xffffffffu, pid[u], i), start = p.slots[t] & (page - 1);
      const int64_t tile = static_cast<int64_t>(id) * p.heads + h;
      const float was = start > 0 ? scales[tile] : 0.f;
      // Tokens of the run; they fill the page from `start` on.
      int n = 1;
      bool open = true;  // the run may go on
#pragma unroll
      for (int w = u; w < NS; ++w) {
        const int from = w == u ? i + 1 : 0, width = min(32, CT - 32 * w) - from;
        if (open && width > 0) {
          const uint32_t rest = ~(goes_on[w] >> from);
          const int more = rest == 0 ? 32 : __ffs(rest) - 1;
          n += min(more, width);
          open = more >= width;
        }
      }
      for (int at = t0 + CT + lane; open && n < page; at += 32) {
        const uint32_t same =
            __ballot_sync(0xffffffffu, (at == t0 + CT + lane ? after : page_of(at)) == id);
        n += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        open = same == 0xffffffffu;
      }
      n = min(n, page - start);
      uint8_t* const cache = out + tile * page * D;
      if (n <= kShortRun) {
        // ---- a warp
        if (k % kWarps != warp) continue;
        constexpr int E = D / 64;  // words of a token per lane
        uint32_t x[kShortRun][E], m = 0;
#pragma unroll
        for (int w = 0; w < kShortRun; ++w)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[w][e] = 0;
            if (w < n)
              x[w][e] = *reinterpret_cast<const uint32_t*>(in + (t + w) * stride + 2 * (lane * E + e));
            m = max_finite<A>(m, x[w][e]);
          }
        const float now = fmaxf(was, scale_for<C>(larger<A>(warp_max(m))));
        if (start > 0 && now != was)
          rescale<C>(reinterpret_cast<uint32_t*>(cache), start * (D / 4), was / now, lane, 32);
        const float inv = 1.f / now;  // exact: a power of two
#pragma unroll
        for (int w = 0; w < kShortRun; ++w) {
          if (w >= n) break;
          uint8_t* dst = cache + (start + w) * D + lane * 2 * E;
          if constexpr (E == 2) {
            *reinterpret_cast<uint32_t*>(dst) = quantise4<A, C>(x[w][0], x[w][1], inv);
          } else {
            const float2 f = act_to_float2<A>(x[w][0]);
            *reinterpret_cast<uint16_t*>(dst) =
                static_cast<uint16_t>(float2_to_stored<C>(f.x * inv, f.y * inv));
          }
        }
        if (lane == 0) scales[tile] = now;
        continue;
      }
      // ---- the CTA: 16-byte pieces, kThreads at a time
      constexpr int PPT = D / 8;                  // pieces of a token
      constexpr int RMAX = 128 * PPT / kThreads;  // of the longest run, per thread
      const int pieces = n * PPT;
      const A* const src = in + (t + tid / PPT) * stride + 8 * (tid % PPT);
      uint4 x[RMAX];
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < RMAX; ++r) {
        x[r] = make_uint4(0, 0, 0, 0);
        if (r * kThreads + tid < pieces)
          x[r] = *reinterpret_cast<const uint4*>(src + r * (kThreads / PPT) * stride);
      }
#pragma unroll
      for (int r = 0; r < RMAX; ++r)
        if (r * kThreads < pieces)
          m = max_abs<A>(max_abs<A>(max_abs<A>(max_abs<A>(m, x[r].x), x[r].y), x[r].z), x[r].w);
      if (has_nonfinite<A>(m)) {
        m = 0;
#pragma unroll
        for (int r = 0; r < RMAX; ++r)
          m = max_finite<A>(max_finite<A>(max_finite<A>(max_finite<A>(m, x[r].x), x[r].y), x[r].z), x[r].w);
      }
      m = warp_max(m);
      __syncthreads();  // s_max of the run before has been read
      if (lane == 0) s_max[warp] = m;
      __syncthreads();  // and every thread has the old scale
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = __vmaxu2(m, s_max[w]);
      const float now = fmaxf(was, scale_for<C>(larger<A>(m)));
      if (start > 0 && now != was)
        rescale<C>(reinterpret_cast<uint32_t*>(cache), start * (D / 4), was / now, tid, kThreads);
      const float inv = 1.f / now;
      uint8_t* const dst = cache + (start + tid / PPT) * D + 8 * (tid % PPT);
#pragma unroll
      for (int r = 0; r < RMAX; ++r) {
        if (r * kThreads >= pieces) break;
        if (r * kThreads + tid < pieces)
          *reinterpret_cast<uint2*>(dst + r * (kThreads / PPT) * D) =
              make_uint2(quantise4<A, C>(x[r].x, x[r].y, inv), quantise4<A, C>(x[r].z, x[r].w, inv));
      }
      if (tid == 0) scales[tile] = now;
    }
  }
}

template <class A, class C, int D>
cudaError_t launch(const CacheAppendParams& p, cudaStream_t stream) {
  auto grid = [&](int ct) { return dim3((p.T + ct - 1) / ct, p.heads, 2); };
  const int64_t rows = static_cast<int64_t>(p.T) * p.heads * 2;
  if (rows <= kSmallRows)
    bsa_cache_append_kernel<A, C, D, 1><<<grid(1), kThreads, 0, stream>>>(p);
  else if (rows <= kMediumRows || p.page_shift <= 5)
    bsa_cache_append_kernel<A, C, D, 16><<<grid(16), kThreads, 0, stream>>>(p);
  else
    bsa_cache_append_kernel<A, C, D, 64><<<grid(64), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class A, class C>
cudaError_t launch(int d, const CacheAppendParams& p, cudaStream_t stream) {
  return d == 128 ? launch<A, C, 128>(p, stream) : launch<A, C, 64>(p, stream);
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
