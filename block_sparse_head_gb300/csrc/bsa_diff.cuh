// bsa_diff.cuh -- what the kernels of differential attention share: their work list and the
// weight of the second map.
//
// A tile holds 64 queries of both maps of one head as 128 rows, so that one pass over the key
// blocks serves both softmaxes: K and V are loaded once, every product has 128 rows, and the
// pipelines are those of the plain kernels.  Queries of d / 2 numbers (a key half for each map)
// are laid out over d columns, zero in the half that the other map's keys take, so that one
// product over d columns gives each row its own map's scores.
#pragma once

#include "bsa_fwd_kernel.cuh"

namespace bsa {

// u / by for u below 2^31, with mul = ceil(2^(31 + shift) / by) and 2^shift >= by: mul * by passes
// 2^(31 + shift) by less than 2^shift, so that the product is off by less than 1 / by.  The roles
// that walk the list divide two to four times an item or step; divisions proper were 11 KB of code in
// the forward, where code is short of cache (bsa_diff_fwd_kernel.cuh).
__device__ __forceinline__ unsigned diff_over(unsigned u, uint32_t mul, int shift) {
  return __umulhi(2 * u, mul) >> shift;
}

// CTA c's u-th sub-item of the work list (descending cost): c, 2G - 1 - c, 2G + c, ... of the
// list of items times pairs times halves, forwards and backwards in turn.
__device__ __forceinline__ int2 stream_range(const DiffList& p) {
  const int grid = gridDim.x, c = blockIdx.x;
  const int full = p.n / grid, rest = p.n - full * grid;
  return make_int2(0, full + (((full & 1) ? grid - 1 - c : c) < rest ? 1 : 0));
}

__device__ __forceinline__ unsigned diff_place(int u) {
  const int grid = gridDim.x, c = blockIdx.x;
  return u * grid + ((u & 1) ? grid - 1 - c : c);
}
__device__ __forceinline__ int4 stream_item(const DiffList& p, int u) {
  return p.list[diff_over(diff_place(u), p.each_mul, p.each_shift)];
}
// Sub-item u of this CTA as a record {b * H + h, first query / 64, first col_idx entry, nnz |
// (dpos + 1) << 16}, from its item's.
__device__ __forceinline__ int4 stream_place(const DiffList& p, int u, const int4& r) {
  if (r.w < 0) return r;  // the end
  const unsigned at = diff_place(u), item = diff_over(at, p.each_mul, p.each_shift);
  int pair = at - item * (p.pairs * p.halves);
  const int half = pair >= p.pairs ? 1 : 0;
  pair -= half * p.pairs;
  return make_int4(r.x * p.pairs + pair, r.y * p.halves + half, r.z, r.w);
}
__device__ __forceinline__ int2 stream_range(const DiffFwdParams& p) {
  return stream_range(static_cast<const DiffList&>(p));
}
__device__ __forceinline__ int4 stream_item(const DiffFwdParams& p, int u) {
  return stream_item(static_cast<const DiffList&>(p), u);
}
__device__ __forceinline__ int4 stream_place(const DiffFwdParams& p, int u, const int4& r) {
  return stream_place(static_cast<const DiffList&>(p), u, r);
}

}  // namespace bsa
