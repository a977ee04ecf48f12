// bsa_cache_resize.cu -- block tables and slots of new tokens from request lengths.
//
// Request b goes from kv_len[b] to new_len[b] tokens, so from had_b = ceil(kv_len[b] / page)
// to has_b = ceil(new_len[b] / page) pages.  Three prefix sums over the requests (new
// tokens, pages taken, pages given back) place everything: page g of those taken is entry
// count + freed - 1 - g of the stack (free pages, then freed pages), and token t of the
// packed new tokens belongs to the last request whose offset is <= t.
//
// Bound: latency, a chain of a few trips to memory and of searches in shared memory, so one
// launch and one round of work for each thread.  Every CTA scans all requests (kThreads at a
// time in consecutive pieces; no sum has to be passed on), then the CTAs share the freed pages,
// the new table entries, the slots (four neighbours a thread) and the lengths.  Where the new
// lengths go to buffers of their own, nothing that a CTA reads is written in the call (new
// pages that were freed in it are taken from the table that they were freed from), and any
// number of CTAs works side by side.  Where they replace the old ones (kv_len_out is kv_len),
// all have to be read before one is written: one CTA, or a cluster of eight and its barrier,
// where there is more to write than one CTA does in that time.  1000 requests with 60 prompts,
// 113,000 new tokens: 10.5 us apart, 12.8 in place (one CTA: 57); 32 requests a token each: 4.2.
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
  } else if constexpr (CL > 1) {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
  }
}

// CL: CTAs of the cluster, which is the grid; 0: outputs apart from the inputs, any grid.
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
  const int ctas = CL == 0 ? static_cast<int>(gridDim.x) : CL;
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

  // Last b with sums[b] <= x, so that x lies in request b's part (x < sums[B]).
  auto find = [&](const int* sums, int x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  const int all = ctas * kThreads, me = rank * kThreads + tid;

  // Page g of those given back, by request b.
  auto freed_page = [&](int g, int b) -> const int32_t* {
    return p.table + static_cast<int64_t>(b) * p.max_pages + pages_of(p.new_len[b]) + g - s_freed[b];
  };
  // Page g of those taken: from the top of the stack, where the freed ones are.
  auto taken_page = [&](int g) -> const int32_t* {
    const int at = count + static_cast<int>(total.shrink) - 1 - g;
    if (CL == 0 && at >= count) return freed_page(at - count, find(s_freed, at - count));
    return p.free_pages + at;
  };

  // Freed pages behind the stack, in the order of requests and pages.
  if (ok)
    for (int g = me; g < static_cast<int>(total.shrink); g += all) {
      const int b = find(s_freed, g);
      p.free_pages[count + g] = *freed_page(g, b);
    }
  barrier_all<CL>();

  if (ok)
    for (int g = me; g < static_cast<int>(total.grow); g += all) {
      const int id = __ldcg(taken_page(g)), b = find(s_grow, g);
      p.table[static_cast<int64_t>(b) * p.max_pages + pages_of(s_old[b]) + g - s_grow[b]] = id;
    }
  const int live = s_cu[B];
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  for (int t = 4 * me; t < p.tokens; t += 4 * all) {
    int slot[4] = {-1, -1, -1, -1};
    if (t < live) {
      int lo = find(s_cu, t);
      // Where token t + i of the call stands: its entry of the table or of the stack.
      auto entry = [&](int pos) -> const int32_t* {
        const int j = pos >> p.page_shift, fresh = j - pages_of(s_old[lo]);
        return fresh < 0 ? p.table + static_cast<int64_t>(lo) * p.max_pages + j
                         : taken_page(s_grow[lo] + fresh);
      };
      const int pos = s_old[lo] + t - s_cu[lo];
      if (t + 4 <= s_cu[lo + 1]) {  // of one request: two pages at most
        const int id0 = __ldcg(entry(pos)), id1 = __ldcg(entry(pos + 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int off = (pos + i) & (page - 1), id = off >= (pos & (page - 1)) ? id0 : id1;
          if (id >= 0 && id < p.n_pages) slot[i] = (id << p.page_shift) + off;
        }
      } else {
        // Where the four pages stand, then the pages: the loads do not wait for one another.
        int id[4], off[4];
        const int32_t* from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          from[i] = p.free_pages;  // not used
          off[i] = 0;
          if (t + i < live) {
            while (s_cu[lo + 1] <= t + i) ++lo;
            const int at = s_old[lo] + t + i - s_cu[lo];
            off[i] = at & (page - 1);
            from[i] = entry(at);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = __ldcg(from[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i < live && id[i] >= 0 && id[i] < p.n_pages)
            slot[i] = (id[i] << p.page_shift) + off[i];
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
  for (int b = me; b <= B; b += all) {
    p.cu_new[b] = s_cu[b];
    if (b < B) p.kv_len_out[b] = ok ? p.new_len[b] : s_old[b];
  }
  if (me == 0) {
    *p.free_count_out = ok ? count + static_cast<int>(freed - needed) : count;
    *p.status = status;
  }
}

template <int CL, class I>
cudaError_t launch(const CacheResizeParams& p, int ctas, cudaStream_t stream) {
  static int done[64];
  const cudaError_t e =
      set_smem_once(bsa_cache_resize_kernel<CL, I>, (4 * kMaxResizeBatch + 3) * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
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

template <class I>
cudaError_t launch(const CacheResizeParams& p, cudaStream_t stream) {
  auto apart = [&](const int32_t* out, int n) {
    auto clear = [&](const int32_t* in, int m) { return out + n <= in || in + m <= out; };
    return clear(p.kv_len, p.B) && clear(p.new_len, p.B) && clear(p.free_count, 1);
  };
  const int rounds = (p.tokens + 4 * kThreads - 1) / (4 * kThreads);
  if (apart(p.kv_len_out, p.B) && apart(p.free_count_out, 1))
    return launch<0, I>(p, rounds < 1 ? 1 : rounds > 64 ? 64 : rounds, stream);
  return rounds <= 1 ? launch<1, I>(p, 1, stream) : launch<8, I>(p, 8, stream);
}

}  // namespace

cudaError_t launch_cache_resize(const CacheResizeParams& p, cudaStream_t stream) {
  const bool narrow = static_cast<int64_t>(p.B) * p.max_pages << p.page_shift <= INT_MAX;
  return narrow ? launch<int>(p, stream) : launch<long long>(p, stream);
}

}  // namespace bsa
