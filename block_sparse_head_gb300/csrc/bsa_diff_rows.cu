// bsa_diff_rows.cu -- what comes before the walks of differential attention's backward: the row
// terms, and the zeros that they count on.
#include <cuda_bf16.h>

#include "bsa_internal.h"

namespace bsa {
namespace {

// Per query: D_1 = sum dO O_1, D_0 = sum dO out + lam D_1 (out = O_0 - lam O_1), the two lse in
// log2 units and lam, laid out as the kernels read them.  Bound: memory, 6 d bytes a query.
// D / 8 lanes a row, 16-byte loads.  Measured: 16 heads of 128, 8,192 tokens 20 us, 5.0 TB/s; 2 x
// 8 heads of 64, 2,999 tokens 5 us; 2 x 2 heads, 333 tokens 2.5 us, the launch.
// Blocks behind the rows' write zeros: the counts, and the gradients of columns without an active
// block, 256 columns a block.
template <int D>
__global__ void __launch_bounds__(256) bsa_diff_rows_kernel(const DiffRowsParams p, const DiffBwdParams w,
                                                            int row_blocks, int counts) {
  constexpr int R = D / 8;
  constexpr float kLog2e = 1.4426950408889634f;
  wait_before();
  if (static_cast<int>(blockIdx.x) >= row_blocks) {
    __shared__ int empty[256], n;
    if (threadIdx.x == 0) n = 0;
    __syncthreads();
    const long long first = static_cast<long long>(blockIdx.x - row_blocks) * 256;
    const long long mine = first + threadIdx.x;
    const int col = static_cast<int>(mine % w.cols);
    if (mine < static_cast<long long>(w.B) * w.cols && w.col_ptr[col] == w.col_ptr[col + 1])
      empty[atomicAdd(&n, 1)] = threadIdx.x;
    if (first == 0)
      for (int i = threadIdx.x; i < counts; i += 256) w.count[i] = 0;
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      const int b = static_cast<int>((first + empty[i]) / w.cols);
      const int c = static_cast<int>(first + empty[i] - static_cast<long long>(b) * w.cols);
      const int kv = c / w.nb, key = (c - kv * w.nb) * w.block;
      const int64_t at = (static_cast<int64_t>(b * (w.cols / w.nb) + kv) * w.L + key) * D;
      for (int x = threadIdx.x; x < min(w.block, w.L - key) * R; x += 256) {
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w.dk) + at)[x] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w.dv) + at)[x] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const int tiles = diff_vec_tiles((p.L + 63) / 64);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / R) + threadIdx.x / R;
  const int64_t pair = r / (64 * tiles);
  const int q = static_cast<int>(r - pair * (64 * tiles));
  const bool in = pair < p.pairs, live = in && q < p.L;
  float a0 = 0.f, a1 = 0.f;
  if (live) {
    const int64_t at = (pair * p.L + q) * D + (lane % R) * 8;
    const uint4 o = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.out) + at);
    const uint4 o2 = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.out2) + at);
    const uint4 g = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dout) + at);
    const __nv_bfloat162* vo = reinterpret_cast<const __nv_bfloat162*>(&o);
    const __nv_bfloat162* vo2 = reinterpret_cast<const __nv_bfloat162*>(&o2);
    const __nv_bfloat162* vg = reinterpret_cast<const __nv_bfloat162*>(&g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(vo[i]), y = __bfloat1622float2(vo2[i]);
      const float2 z = __bfloat1622float2(vg[i]);
      a0 = fmaf(z.x, x.x, fmaf(z.y, x.y, a0));
      a1 = fmaf(z.x, y.x, fmaf(z.y, y.y, a1));
    }
  }
#pragma unroll
  for (int w = R / 2; w >= 1; w /= 2) {
    a0 += __shfl_xor_sync(0xffffffffu, a0, w);
    a1 += __shfl_xor_sync(0xffffffffu, a1, w);
  }
  if (!in || lane % R >= 5) return;
  // Lane i of a row writes term i, negated.  Rows past the end, and rows without an active key,
  // get -lse = -inf: their P is 0.
  const int i = lane % R;
  const float lam = live ? (p.lam_rows ? p.lam[pair * p.L + q] : p.lam[pair % p.H]) : 0.f;
  float x;
  if (i < 2) {
    x = live ? p.lse[(2 * pair + i) * p.L + q] * -kLog2e : -INFINITY;
    if (x == INFINITY) x = -INFINITY;
  } else {
    x = -(i == 2 ? fmaf(lam, a1, a0) : i == 3 ? a1 : lam);
  }
  p.vec[(pair * tiles + (q >> 6)) * kDiffVecFloats + ((q >> 5) & 1) * (kDiffVecFloats / 2) + 32 * i +
        (q & 31)] = x;
}

}  // namespace

cudaError_t launch_diff_rows(const DiffRowsParams& p, const DiffBwdParams& b, int counts, cudaStream_t stream) {
  const int64_t rows = p.pairs * 64 * diff_vec_tiles((p.L + 63) / 64);
  const int per = 256 / (p.d / 8);
  const int64_t blocks = (rows + per - 1) / per, more = (static_cast<int64_t>(b.B) * b.cols + 255) / 256;
  if (blocks + more > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto* kernel = p.d == 128 ? bsa_diff_rows_kernel<128> : bsa_diff_rows_kernel<64>;
  return launch_after(kernel, dim3(static_cast<unsigned>(blocks + more)), 256, 0, stream, p, b,
                      static_cast<int>(blocks), counts);
}

}  // namespace bsa
