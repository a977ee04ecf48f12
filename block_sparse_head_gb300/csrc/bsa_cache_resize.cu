// bsa_cache_resize.cu -- block tables and slots of new tokens from request lengths.
//
// Request b goes from kv_len[b] to new_len[b] tokens, so from had_b = ceil(kv_len[b] / page)
// to has_b = ceil(new_len[b] / page) pages.  Three prefix sums over the requests (new
// tokens, pages taken, pages given back) place everything: page g of those taken is entry
// count + freed - 1 - g of the stack (free pages, then freed pages), and token t of the
// packed new tokens belongs to the last request whose offset is <= t.
//
// Bound: latency.  One launch of one CTA, or of a cluster of eight where there is more to
// write than one CTA does in the time of a cluster barrier.  Every CTA scans all requests
// (kThreads at a time in consecutive pieces, so no sum has to be passed on), then they share
// the work: freed pages behind the stack; after the one barrier the new table entries, the
// slots (four neighbours a thread) and the lengths.  All inputs are read before the barrier
// and no output is written before it, so kv_len_out and free_count_out may alias their
// inputs; free pages read after it may have been written in this call.
#include "bsa_internal.h"

#include <climits>

namespace bsa {

namespace {

constexpr int kThreads = 1024;

// Three sums at a time; 32-bit where the host knows that no sum passes it.
template <class I>
struct Sums {
  I fresh, grow, shrink;
};

template <class I>
__device__ __forceinline__ Sums<I> add(const Sums<I>& a, const Sums<I>& b) {
  return {a.fresh + b.fresh, a.grow + b.grow, a.shrink + b.shrink};
}

// Inclusive scan over a warp.
template <class I>
__device__ __forceinline__ Sums<I> warp_scan(Sums<I> x, int lane) {
#pragma unroll
  for (int n = 1; n < 32; n *= 2) {
    const Sums<I> up{__shfl_up_sync(0xffffffffu, x.fresh, n), __shfl_up_sync(0xffffffffu, x.grow, n),
                     __shfl_up_sync(0xffffffffu, x.shrink, n)};
    if (lane >= n) x = add(x, up);
  }
  return x;
}

template <int CL>
__device__ __forceinline__ void barrier_all() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
  }
}

// CL: CTAs of the cluster, which is the grid.
template <int CL, class I>
__global__ void __launch_bounds__(kThreads) bsa_cache_resize_kernel(const CacheResizeParams p) {
  extern __shared__ int smem[];
  const int B = p.B, page = 1 << p.page_shift;
  int* s_cu = smem;               // [B + 1] offsets of the new tokens
  int* s_grow = s_cu + B + 1;     // [B + 1] pages taken before request b
  int* s_freed = s_grow + B + 1;  // [B + 1] pages given back before request b
  int* s_old = s_freed + B + 1;   // [B]
  __shared__ Sums<I> s_warp[kThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL == 1 ? 0 : static_cast<int>(blockIdx.x);
  const int all_warps = CL * kThreads / 32, my_warp = rank * (kThreads / 32) + warp;
  if (tid == 0) s_bad = B;
  __syncthreads();

  const long long most = static_cast<long long>(p.max_pages) * page;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const int count = *p.free_count;
  auto pages_of = [&](int n) {
    return static_cast<int>((static_cast<uint32_t>(n) + page - 1) >> p.page_shift);
  };
  auto sums_of = [&](int old, int now) {
    if (old < 0 || now < 0 || old > most || now > most) return Sums<I>{0, 0, 0};
    const int d = pages_of(now) - pages_of(old);
    return Sums<I>{max(0, now - old), max(0, d), max(0, -d)};
  };
  Sums<I> mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int old = p.kv_len[b], now = p.new_len[b];
    s_old[b] = old;
    if (old < 0 || now < 0 || old > most || now > most) atomicMin(&s_bad, b);
    mine = add(mine, sums_of(old, now));
  }
  const Sums<I> inc = warp_scan(mine, lane);
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  static_assert(kThreads / 32 == 32, "one warp's sum a lane");
  const Sums<I> upto = warp_scan(s_warp[lane], lane);
  auto at = [&](I x, int from) { return __shfl_sync(0xffffffffu, x, from); };
  const Sums<I> total{at(upto.fresh, 31), at(upto.grow, 31), at(upto.shrink, 31)};
  const int w1 = max(0, warp - 1);
  Sums<I> before{at(upto.fresh, w1), at(upto.grow, w1), at(upto.shrink, w1)};
  if (warp == 0) before = {0, 0, 0};
  before = add(before, Sums<I>{inc.fresh - mine.fresh, inc.grow - mine.grow, inc.shrink - mine.shrink});
  const long long freed = total.shrink, needed = total.grow;
  int status = 0;
  if (s_bad < B) status = -1 - s_bad;
  else if (total.fresh > p.tokens) status = INT_MIN;
  else if (count < 0 || count + freed > p.n_pages) status = INT_MIN + 1;
  else if (needed > count + freed)
    status = static_cast<int>(min(needed - count - freed, static_cast<long long>(INT_MAX)));
  const bool ok = status == 0;
  for (int b = b0; b < b1; ++b) {
    s_cu[b] = ok ? static_cast<int>(before.fresh) : 0;
    s_grow[b] = static_cast<int>(before.grow);
    s_freed[b] = static_cast<int>(before.shrink);
    if (per > 1) before = add(before, sums_of(s_old[b], p.new_len[b]));
  }
  if (tid == 0) {
    s_cu[B] = ok ? static_cast<int>(total.fresh) : 0;
    s_grow[B] = static_cast<int>(total.grow);
    s_freed[B] = static_cast<int>(total.shrink);
  }
  __syncthreads();

  // Freed pages behind the stack, in the order of requests and pages.
  if (ok && total.shrink > 0) {
    for (int b = my_warp; b < B; b += all_warps) {
      const int n = s_freed[b + 1] - s_freed[b];
      if (n == 0) continue;
      const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages + pages_of(p.new_len[b]);
      for (int j = lane; j < n; j += 32) p.free_pages[count + s_freed[b] + j] = row[j];
    }
  }
  barrier_all<CL>();

  const int top = ok ? count + static_cast<int>(total.shrink) - 1 : 0;
  if (ok && total.grow > 0) {
    for (int b = my_warp; b < B; b += all_warps) {
      const int n = s_grow[b + 1] - s_grow[b];
      if (n == 0) continue;
      int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages + pages_of(s_old[b]);
      for (int j = lane; j < n; j += 32) row[j] = __ldcg(p.free_pages + top - s_grow[b] - j);
    }
  }
  const int live = s_cu[B];
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (int t = 4 * (rank * kThreads + tid); t < p.tokens; t += 4 * CL * kThreads) {
    int slot[4] = {-1, -1, -1, -1};
    if (t < live) {
      int lo = 0, hi = B;  // s_cu[lo] <= t < s_cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      int id = -1, seen = -1;  // page of the last token, and its place in the table
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t + i >= live) break;
        while (s_cu[lo + 1] <= t + i) {
          ++lo;
          seen = -1;
        }
        const int pos = s_old[lo] + t + i - s_cu[lo], j = pos >> p.page_shift;
        if (j != seen) {
          const int had = pages_of(s_old[lo]);
          id = j < had ? p.table[static_cast<int64_t>(lo) * p.max_pages + j]
                       : __ldcg(p.free_pages + top - s_grow[lo] - (j - had));
          seen = j;
        }
        if (id >= 0 && id < p.n_pages) slot[i] = (id << p.page_shift) + (pos & (page - 1));
      }
    }
    if (wide && t + 4 <= p.tokens) {
      *reinterpret_cast<int4*>(p.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t + i < p.tokens) p.slots[t + i] = slot[i];
    }
  }
  for (int b = rank * kThreads + tid; b <= B; b += CL * kThreads) {
    p.cu_new[b] = s_cu[b];
    if (b < B) p.kv_len_out[b] = ok ? p.new_len[b] : s_old[b];
  }
  if (rank == 0 && tid == 0) {
    *p.free_count_out = ok ? top + 1 - static_cast<int>(total.grow) : count;
    *p.status = status;
  }
}

template <int CL, class I>
cudaError_t launch(const CacheResizeParams& p, cudaStream_t stream) {
  static int done[64];
  const cudaError_t e =
      set_smem_once(bsa_cache_resize_kernel<CL, I>, (4 * kMaxResizeBatch + 3) * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CL);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (4 * p.B + 3) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CL;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, bsa_cache_resize_kernel<CL, I>, p);
}

}  // namespace

cudaError_t launch_cache_resize(const CacheResizeParams& p, cudaStream_t stream) {
  const bool narrow = static_cast<int64_t>(p.B) * p.max_pages << p.page_shift <= INT_MAX;
  if (!narrow) return launch<8, long long>(p, stream);
  // One CTA writes a few thousand slots in the time that a cluster takes to start and meet.
  return p.tokens <= 4 * kThreads ? launch<1, int>(p, stream) : launch<8, int>(p, stream);
}

}  // namespace bsa
