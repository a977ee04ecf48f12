// bsa_cache_fwd.cu -- attention of each request's newest tokens over its paged 8-bit cache.
//
// Query i of the n queries of request b stands at position pos = kv_len[b] - n + i and sees
// the keys c <= pos that the window and the layout's row (kv head, pos / block) leave:
//     s_c = scale * k_scale[page(c)] * <q, k8_c>   (soft-capped if set)
//     out = sum_c exp(s_c - lse) * v_scale[page(c)] * v8_c
// in one pass over the keys with a running maximum and sum (base 2).
//
// One CTA per (token, query head); its warps take the keys in turn, each lane D / 32 of a
// key's numbers, and are joined at the end.
#include "bsa_cache.cuh"
#include "bsa_internal.h"
#include "bsa_ptx.cuh"

namespace bsa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <class A, class C, int D>
__global__ void __launch_bounds__(kThreads) bsa_cache_fwd_kernel(const CacheFwdParams p) {
  constexpr int E = D / 32;  // numbers of a key per lane
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / p.group;
  if (t == 0 && hq == 0 && threadIdx.x == 0) *p.status = 0;
  if (t < p.cu_q[0] || t >= p.cu_q[p.B]) return;
  int b = 0, hi = p.B;  // cu_q[b] <= t < cu_q[hi]
  while (hi - b > 1) {
    const int mid = (b + hi) >> 1;
    if (p.cu_q[mid] <= t) b = mid;
    else hi = mid;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = max(0, min(p.kv_len[b], p.max_pages << p.page_shift));
  const int pos = len - (p.cu_q[b + 1] - t);
  const int first = p.window >= 0 ? max(0, pos - p.window) : 0;

  float q[E];
  const A* qp = static_cast<const A*>(p.q) + t * p.q_token_stride + hq * p.q_head_stride;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 f = act_to_float2<A>(*reinterpret_cast<const uint32_t*>(qp + lane * E + e));
    q[e] = f.x;
    q[e + 1] = f.y;
  }
  float m = -INFINITY, l = 0.f, o[E] = {};
  auto keys = [&](int c0, int c1) {
    for (int c = c0 + warp; c < c1; c += kWarps) {
      const int id = p.table[static_cast<int64_t>(b) * p.max_pages + (c >> p.page_shift)];
      if (id < 0 || id >= p.n_pages) continue;
      const int64_t tile = static_cast<int64_t>(id) * p.Hkv + h;
      const int64_t at = ((tile << p.page_shift) + (c & ((1 << p.page_shift) - 1))) * D + lane * E;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 k =
            stored_to_float2<C>(*reinterpret_cast<const uint16_t*>(p.k_cache + at + e));
        s = fmaf(q[e], k.x, fmaf(q[e + 1], k.y, s));
      }
#pragma unroll
      for (int n = 16; n >= 1; n /= 2) s += __shfl_xor_sync(0xffffffffu, s, n);
      s *= p.k_scale[tile];
      s = p.softcap_log2 > 0.f ? p.softcap_log2 * tanhf(s * p.softcap_inv) : s * p.scale_log2;
      const float mn = fmaxf(m, s);
      const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = s == -INFINITY ? 0.f : exp2f(s - mn);
      const float vs = w * p.v_scale[tile];
      m = mn;
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v =
            stored_to_float2<C>(*reinterpret_cast<const uint16_t*>(p.v_cache + at + e));
        o[e] = o[e] * a + vs * v.x;
        o[e + 1] = o[e + 1] * a + vs * v.y;
      }
    }
  };
  if (pos >= 0) {
    if (p.row_ptr == nullptr) {
      keys(first, pos + 1);
    } else {
      const int row = h * p.nb + (pos >> p.block_shift);
      for (int e = p.row_ptr[row]; e < p.row_ptr[row + 1]; ++e) {
        const int c0 = p.col_idx[e] << p.block_shift;
        keys(max(first, c0), min(pos + 1, c0 + (1 << p.block_shift)));
      }
    }
  }
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  const float sink = p.sinks ? p.sinks[hq] * 1.4426950408889634f : -INFINITY;
  float top = sink;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  const int64_t row = static_cast<int64_t>(t) * p.Hq + hq;
  float z = sink == -INFINITY ? 0.f : exp2f(sink - top), f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - top);
    z += s_l[w] * f[w];
  }
  if (threadIdx.x < D / 2) {
    float2 r = make_float2(0.f, 0.f);
    for (int w = 0; w < kWarps; ++w) {
      r.x += s_o[w][2 * threadIdx.x] * f[w];
      r.y += s_o[w][2 * threadIdx.x + 1] * f[w];
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
    reinterpret_cast<uint32_t*>(static_cast<A*>(p.out) + row * D)[threadIdx.x] =
        float2_to_act<A>(r.x * inv, r.y * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = z == 0.f ? -INFINITY : (top + log2f(z)) * 0.6931471805599453f;
}

template <class A, class C>
cudaError_t launch(int d, const CacheFwdParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(p.Hq));
  if (d == 128) bsa_cache_fwd_kernel<A, C, 128><<<grid, kThreads, 0, stream>>>(p);
  else bsa_cache_fwd_kernel<A, C, 64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_fwd(int d, int dtype, int cache_dtype, const CacheFwdParams& p,
                             cudaStream_t stream) {
  if (dtype == BSA_BF16)
    return cache_dtype == BSA_E4M3 ? launch<__nv_bfloat16, E4M3>(d, p, stream)
                                   : launch<__nv_bfloat16, Int8>(d, p, stream);
  return cache_dtype == BSA_E4M3 ? launch<__half, E4M3>(d, p, stream)
                                 : launch<__half, Int8>(d, p, stream);
}

}  // namespace bsa
