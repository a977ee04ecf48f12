// bsa_cache_resize.cu -- block tables and slots of new tokens from request lengths.
//
// Request b goes from kv_len[b] to new_len[b] tokens, so from had_b = ceil(kv_len[b] / page)
// to has_b = ceil(new_len[b] / page) pages.  Three prefix sums over the requests (new
// tokens, pages taken, pages given back) place everything: page g of those taken is entry
// count + freed - 1 - g of the stack (free pages, then freed pages), and token t of the
// packed new tokens belongs to the last request whose offset is <= t.
//
// One CTA: it scans the requests (kThreads at a time in consecutive pieces), writes the
// freed pages behind the stack, and after a barrier the new table entries, the slots and
// the lengths.  Nothing is written that a later read of this call needs, except the freed
// pages, so kv_len_out and free_count_out may alias their inputs.
#include "bsa_internal.h"

#include <climits>

namespace bsa {

namespace {

constexpr int kThreads = 1024;

struct Sums {
  long long fresh, grow, shrink;
};

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
  return {a.fresh + b.fresh, a.grow + b.grow, a.shrink + b.shrink};
}

__device__ __forceinline__ Sums shfl_up(const Sums& a, int n) {
  return {__shfl_up_sync(0xffffffffu, a.fresh, n), __shfl_up_sync(0xffffffffu, a.grow, n),
          __shfl_up_sync(0xffffffffu, a.shrink, n)};
}

__global__ void __launch_bounds__(kThreads) bsa_cache_resize_kernel(const CacheResizeParams p) {
  extern __shared__ int smem[];
  const int B = p.B, page = 1 << p.page_shift;
  int* s_cu = smem;               // [B + 1] offsets of the new tokens
  int* s_grow = s_cu + B + 1;     // [B + 1] pages taken before request b
  int* s_freed = s_grow + B + 1;  // [B + 1] pages given back before request b
  int* s_old = s_freed + B + 1;   // [B]
  __shared__ Sums s_warp[kThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = B;
  __syncthreads();

  const long long most = static_cast<long long>(p.max_pages) * page;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto pages_of = [&](int n) {
    return static_cast<int>((static_cast<long long>(n) + page - 1) >> p.page_shift);
  };
  auto sums_of = [&](int b, int old, int now) {
    if (old < 0 || now < 0 || old > most || now > most) {
      atomicMin(&s_bad, b);
      return Sums{0, 0, 0};
    }
    const int d = pages_of(now) - pages_of(old);
    return Sums{max(0, now - old), max(0, d), max(0, -d)};
  };
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) mine = add(mine, sums_of(b, p.kv_len[b], p.new_len[b]));
  Sums inc = mine;
  for (int n = 1; n < 32; n *= 2) {
    const Sums up = shfl_up(inc, n);
    if (lane >= n) inc = add(inc, up);
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Sums before{0, 0, 0}, total{0, 0, 0};
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before = add(before, s_warp[w]);
    total = add(total, s_warp[w]);
  }
  before = add(before, {inc.fresh - mine.fresh, inc.grow - mine.grow, inc.shrink - mine.shrink});
  const int count = *p.free_count;
  int status = 0;
  if (s_bad < B) status = -1 - s_bad;
  else if (total.fresh > p.tokens) status = INT_MIN;
  else if (count < 0 || count + total.shrink > p.n_pages) status = INT_MIN + 1;
  else if (total.grow > count + total.shrink)
    status = static_cast<int>(min(total.grow - count - total.shrink, static_cast<long long>(INT_MAX)));
  const bool ok = status == 0;
  for (int b = b0; b < b1; ++b) {
    const int old = p.kv_len[b];
    s_old[b] = old;
    s_cu[b] = ok ? static_cast<int>(before.fresh) : 0;
    s_grow[b] = static_cast<int>(before.grow);
    s_freed[b] = static_cast<int>(before.shrink);
    before = add(before, sums_of(b, old, p.new_len[b]));
  }
  if (tid == 0) {
    s_cu[B] = ok ? static_cast<int>(total.fresh) : 0;
    s_grow[B] = static_cast<int>(total.grow);
    s_freed[B] = static_cast<int>(total.shrink);
  }
  __syncthreads();

  // Freed pages behind the stack, in the order of requests and pages.
  if (ok && total.shrink > 0) {
    for (int b = warp; b < B; b += kThreads / 32) {
      const int n = s_freed[b + 1] - s_freed[b];
      if (n == 0) continue;
      const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages + pages_of(p.new_len[b]);
      for (int j = lane; j < n; j += 32) p.free_pages[count + s_freed[b] + j] = row[j];
    }
  }
  __syncthreads();

  const int top = ok ? count + static_cast<int>(total.shrink) - 1 : 0;
  if (ok && total.grow > 0) {
    for (int b = warp; b < B; b += kThreads / 32) {
      const int n = s_grow[b + 1] - s_grow[b];
      if (n == 0) continue;
      int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages + pages_of(s_old[b]);
      for (int j = lane; j < n; j += 32) row[j] = p.free_pages[top - s_grow[b] - j];
    }
  }
  const int live = s_cu[B];
  for (int t = tid; t < p.tokens; t += kThreads) {
    int slot = -1;
    if (t < live) {
      int lo = 0, hi = B;  // s_cu[lo] <= t < s_cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int pos = s_old[lo] + t - s_cu[lo];
      const int j = pos >> p.page_shift, had = pages_of(s_old[lo]);
      const int id = j < had ? p.table[static_cast<int64_t>(lo) * p.max_pages + j]
                             : p.free_pages[top - s_grow[lo] - (j - had)];
      if (id >= 0 && id < p.n_pages) slot = (id << p.page_shift) + (pos & (page - 1));
    }
    p.slots[t] = slot;
  }
  for (int b = tid; b <= B; b += kThreads) {
    p.cu_new[b] = s_cu[b];
    if (b < B) p.kv_len_out[b] = ok ? p.new_len[b] : s_old[b];
  }
  if (tid == 0) {
    *p.free_count_out = ok ? top + 1 - static_cast<int>(total.grow) : count;
    *p.status = status;
  }
}

}  // namespace

cudaError_t launch_cache_resize(const CacheResizeParams& p, cudaStream_t stream) {
  const int smem = (4 * p.B + 3) * 4;
  static int done[64];
  const cudaError_t e =
      set_smem_once(bsa_cache_resize_kernel, (4 * kMaxResizeBatch + 3) * 4, done);
  if (e != cudaSuccess) return e;
  bsa_cache_resize_kernel<<<1, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace bsa
