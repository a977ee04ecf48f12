// bsa_diff_rows.cu -- the small kernels of differential attention's backward: the row terms
// before its walks, the joining of cut columns and the sum of the weight's gradient after them.
#include <cuda_bf16.h>

#include "bsa_internal.h"

namespace bsa {
namespace {

// Per query: D_1 = sum dO O_1, D_0 = sum dO out + lam D_1 (out = O_0 - lam O_1), the two lse in
// log2 units and lam, laid out as the kernels read them.  Bound: memory, 6 d bytes a query.
// D / 8 lanes a row, 16-byte loads.
template <int D>
__global__ void __launch_bounds__(256) bsa_diff_rows_kernel(const DiffRowsParams p) {
  constexpr int R = D / 8;
  constexpr float kLog2e = 1.4426950408889634f;
  wait_before();
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

// dlam[h] = sum over b and rows of rows[b, h, :], by one CTA in fp64 and a fixed order.
__device__ void sum_lam(const float* rows, float* dlam, int B, int H, int h, int L) {
  __shared__ double part[8];
  double s = 0.0;
  for (int b = 0; b < B; ++b) {
    const float* r = rows + (static_cast<int64_t>(b) * H + h) * L;
    float x[8];
    for (int i = threadIdx.x; i < L; i += 8 * 256) {
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i + 256 * u < L ? r[i + 256 * u] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += static_cast<double>(x[u]);
    }
  }
#pragma unroll
  for (int w = 16; w >= 1; w /= 2) s += __shfl_xor_sync(0xffffffffu, s, w);
  __syncthreads();  // the head before has read its parts
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) s += part[w];
    dlam[h] = static_cast<float>(s);
  }
}

// Block x < grid of the dK/dV walk: the column cut at the start of CTA x's share, if CTA x - 1 has
// its first piece, is the sum of its pieces in the CTAs' order.  Blocks behind: the zeros of
// columns without an active block.  y: a share of the column's rows; and, behind the last share,
// the weight's gradient of heads x, x + gridDim.x, .. (where it is one number a head).
__global__ void __launch_bounds__(256) bsa_diff_join_kernel(const DiffBwdParams p, int grid, int shares,
                                                            float* dlam, int H) {
  wait_before();
  if (static_cast<int>(blockIdx.y) == shares) {
    for (int h = blockIdx.x; h < H; h += gridDim.x) sum_lam(p.dlam, dlam, p.B, H, h, p.L);
    return;
  }
  const int d = p.d, lanes = d / 2;  // threads of a row, four numbers of dV | dK each
  const int r0 = threadIdx.x / lanes, at = threadIdx.x % lanes * 4;
  const int rows = p.block / shares, step = 256 / lanes;
  auto store = [&](int b, int col, int row, float4 x) {
    const int kv = col / p.nb, key = (col - kv * p.nb) * p.block + row;
    if (key >= p.L) return;
    const int64_t to = (static_cast<int64_t>(b * (p.cols / p.nb) + kv) * p.L + key) * d;
    const float f = at < d ? 1.f : p.scale;
    __nv_bfloat162 y[2] = {__floats2bfloat162_rn(x.x * f, x.y * f), __floats2bfloat162_rn(x.z * f, x.w * f)};
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(at < d ? p.dv : p.dk) + to + (at < d ? at : at - d);
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
  };
  const int row0 = blockIdx.y * rows;
  if (static_cast<int>(blockIdx.x) >= grid) {
    // 256 columns a block, a thread each.
    __shared__ int empty[256], n;
    if (threadIdx.x == 0) n = 0;
    __syncthreads();
    const long long mine = (blockIdx.x - grid) * 256ll + threadIdx.x;
    const int col = static_cast<int>(mine % p.cols);
    if (mine < static_cast<long long>(p.B) * p.cols && p.col_ptr[col] == p.col_ptr[col + 1])
      empty[atomicAdd(&n, 1)] = threadIdx.x;
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      const long long it = (blockIdx.x - grid) * 256ll + empty[i];
      const int b = static_cast<int>(it / p.cols);
      for (int r = r0; r < rows; r += step)
        store(b, static_cast<int>(it - static_cast<long long>(b) * p.cols), row0 + r, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    return;
  }
  const long long start = blockIdx.x * p.share;
  if (blockIdx.x == 0 || start >= p.steps) return;
  const int per = p.pairs * p.halves;
  const long long entry = diff_div(start, per);
  const int b = static_cast<int>(diff_div(entry, p.nnz));
  const long long base = static_cast<long long>(b) * p.nnz;
  const int x = static_cast<int>(entry - base);
  const int lo = diff_column(p, x);
  const long long first = (base + p.col_ptr[lo]) * per, end = (base + p.col_ptr[lo + 1]) * per;
  const int root = static_cast<int>(diff_div(first, p.share)), last = static_cast<int>(diff_div(end - 1, p.share));
  if (first == start || root != static_cast<int>(blockIdx.x) - 1) return;
  const int64_t slot = static_cast<int64_t>(p.block) * 2 * d;
  // Two rows a thread, four pieces at once: their loads wait together.
  const float* src = p.parts + (row0 + r0) * (2 * d) + at;
  float4 sum[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    sum[u] = *reinterpret_cast<const float4*>(src + u * step * 2 * d + (2 * static_cast<int64_t>(root) + 1) * slot);
  for (int i = root + 1; i <= last; i += 4) {
    float4 y[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        y[j][u] = i + j <= last ? *reinterpret_cast<const float4*>(src + u * step * 2 * d + 2 * static_cast<int64_t>(i + j) * slot)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sum[u].x += y[j][u].x;
        sum[u].y += y[j][u].y;
        sum[u].z += y[j][u].z;
        sum[u].w += y[j][u].w;
      }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) store(b, lo, row0 + r0 + u * step, sum[u]);
}

}  // namespace

cudaError_t launch_diff_join(const DiffBwdParams& p, int grid, float* dlam, int H, cudaStream_t stream) {
  const int more = static_cast<int>((static_cast<long long>(p.B) * p.cols + 255) / 256);
  const int shares = p.block * p.d / 1024;  // a thread has two rows
  return launch_after(bsa_diff_join_kernel, dim3(grid + more, shares + (dlam != nullptr)), 256, 0, stream, p, grid,
                      shares, dlam, H);
}

cudaError_t launch_diff_rows(const DiffRowsParams& p, cudaStream_t stream) {
  const int64_t rows = p.pairs * 64 * diff_vec_tiles((p.L + 63) / 64);
  const int per = 256 / (p.d / 8);
  const int64_t grid = (rows + per - 1) / per;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto* kernel = p.d == 128 ? bsa_diff_rows_kernel<128> : bsa_diff_rows_kernel<64>;
  return launch_after(kernel, dim3(static_cast<unsigned>(grid)), 256, 0, stream, p);
}

}  // namespace bsa
