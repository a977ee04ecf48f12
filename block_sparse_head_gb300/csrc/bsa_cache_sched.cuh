// bsa_cache_sched.cuh -- how the attention kernels over a cache share their work out.
//
// A unit is (request b, kv head h, query tile t): TQ consecutive queries of b, the rows of
// all G query heads of h packed together, against the keys those queries can see.  (TQ is a power
// of two, and with a layout tiles begin at multiples of it: 5 queries of 3 heads are two decode
// tiles of 4 queries, 12 of 16 rows, and read the cache twice.)  Its keys
// are taken in slices of 2^SL keys (of the dense range, or of the layout row's blocks).
// Every length sits on the device, so the split is made there: all units are laid end to
// end on one axis, a unit taking a few places for its fixed work and one a slice, and CTA c
// takes the c-th piece of equal length.  A CTA thus runs whole units and at most two cut ones;
// cut units leave partial results (reference, sum, accumulator) in the workspace, and the
// CTA that leaves the last one joins them.  Any mix of lengths splits evenly, one long request
// over all CTAs as well as a thousand short ones, and the result does not depend on which CTA
// is first.
#pragma once

#include "bsa_internal.h"

namespace bsa {

// One CTA's share of one unit.
struct CacheSeg {
  int b, h;
  int q0, nq;       // first packed token and number of queries (0: no more segments)
  int pos0;         // position of the first query
  int lo_key;       // no query of the tile sees a key before it (window)
  int s0, s1;       // pieces [s0, s1): of the key axis (dense) or of the row's block list
  int rp;           // layout row: first col_idx entry
  int starts, ends; // whether the unit's first / last piece is in this segment
  int before, more; // CTAs before and after this one that have a piece of the unit
};

struct CacheUnits {
  const CacheFwdParams& p;
  int tq_shift;  // log2 queries of a tile
  int sl;        // log2 keys of a piece, at most those of a layout block (decode: and of a page)
  int overhead;  // places for a unit's fixed work
  int least;     // places of a CTA's share at least (a power of two)

  struct Request {
    int q0, n, len, p0, o, tiles;
  };
  __device__ __forceinline__ Request request(int b) const {
    Request r;
    const int c0 = max(0, min(p.cu_q[b], p.T)), c1 = max(c0, min(p.cu_q[b + 1], p.T));
    r.q0 = c0;
    r.n = c1 - c0;
    r.len = max(0, min(p.kv_len[b], p.max_pages << p.page_shift));
    r.p0 = r.len - r.n;
    // With a layout, tiles begin at multiples of their size (negative positions included), so that
    // the queries of a tile share one layout row.
    const int tq = 1 << tq_shift;
    r.o = p.row_ptr != nullptr ? (r.p0 & ~(tq - 1)) : r.p0;
    r.tiles = r.n > 0 ? (r.len - r.o + tq - 1) >> tq_shift : 0;
    return r;
  }
  // Pieces of tile t; fills the tile's part of s.
  __device__ __forceinline__ int unit(const Request& r, int h, int t, CacheSeg& s) const {
    const int a = max(r.p0, r.o + (t << tq_shift));
    const int e = min(r.len, r.o + ((t + 1) << tq_shift)), last = e - 1;
    s.h = h;
    s.nq = e - a;
    s.q0 = r.q0 + (a - r.p0);
    s.pos0 = a;
    s.lo_key = p.window >= 0 ? max(0, a - p.window) : 0;
    s.rp = 0;
    s.s0 = 0;
    if (last < 0) return 0;
    if (p.row_ptr != nullptr) {
      const int32_t* row = p.row_ptr + h * p.nb + (last >> p.block_shift);
      s.rp = row[0];
      return (row[1] - row[0]) << (p.block_shift - sl);
    }
    s.s0 = s.lo_key >> sl;
    return (last >> sl) + 1 - s.s0;
  }
  // Places of a unit before its pieces: those of the fixed work, and as many as make the unit a
  // multiple of the least share, so that in the smallest calls no CTA has parts of two units.
  __device__ __forceinline__ int fixed(int pieces) const { return overhead + (-pieces & (least - 1)); }
  __device__ __forceinline__ int places(const Request& r, int h, int t, CacheSeg& s) const {
    const int pieces = unit(r, h, t, s);
    return fixed(pieces) + pieces;
  }
  __device__ __forceinline__ long long head_places(const Request& r, int h) const {
    long long n = 0;
    CacheSeg s;
    for (int t = 0; t < r.tiles; ++t) n += places(r, h, t, s);
    return n;
  }
};

// ceil(a / b) for a >= 0, b > 0: 32-bit division where the numbers allow it (a 64-bit one is
// several times as long, and these stand in the way of the first load).
__device__ __forceinline__ long long div_up(long long a, long long b) {
  if (a + b < (1ll << 31))
    return (static_cast<uint32_t>(a) + static_cast<uint32_t>(b) - 1) / static_cast<uint32_t>(b);
  return (a + b - 1) / b;
}

// Walks a CTA's segments.
struct CacheWalk {
  int b, h, t;
  long long off;   // places of unit (b, h, t) that lie before this CTA
  long long left;  // places of this CTA still to hand out
  long long chunk;
  CacheUnits::Request r;  // of request b

  // Next segment into s (s.nq = 0 at the end).
  __device__ void next(const CacheUnits& u, CacheSeg& s) {
    s.nq = 0;
    if (left <= 0) return;
    for (; b < u.p.B; h = 0, ++b < u.p.B ? (void)(r = u.request(b)) : (void)0) {
      if (r.tiles == 0) continue;
      for (; h < u.p.Hkv; ++h, t = 0) {
        if (t >= r.tiles) continue;
        s.b = b;
        const int pieces = u.unit(r, h, t, s);
        const int fixed = u.fixed(pieces);
        const long long size = fixed + pieces;
        const long long take = min(left, size - off), end = off + take;
        // the unit's fixed places come first
        s.s1 = s.s0 + static_cast<int>(max(0ll, end - fixed));
        s.s0 += static_cast<int>(max(0ll, off - fixed));
        s.starts = off == 0;
        s.ends = end == size;
        s.before = off > 0 ? static_cast<int>(div_up(off, chunk)) : 0;
        s.more = size > end ? static_cast<int>(div_up(size - end, chunk)) : 0;
        left -= take;
        off = 0;
        ++t;
        return;
      }
    }
  }
};

// Splits the axis: every thread of the CTA calls it, thread 0 of the caller gets the walk
// through `out` (shared memory).  scratch: kThreads / 32 + 1 long longs.
template <int kThreads>
__device__ __forceinline__ void cache_split(const CacheUnits& u, long long* scratch,
                                            CacheWalk* out) {
  const CacheFwdParams& p = u.p;
  // Without a layout the heads of a request have the same places, so the requests are
  // scanned; with one, the (request, head) pairs are.
  const bool lay = p.row_ptr != nullptr;
  const int n = lay ? p.B * p.Hkv : p.B, mult = lay ? 1 : p.Hkv;
  const int per = (n + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  auto places = [&](int i, CacheUnits::Request& r) {
    const int b = lay ? i / p.Hkv : i;
    r = u.request(b);
    return u.head_places(r, lay ? i - b * p.Hkv : 0);
  };
  CacheUnits::Request r{};
  long long mine = 0, one = 0;
  for (int i = i0; i < i1; ++i) {
    one = places(i, r);
    mine += one * mult;
  }
  long long inc = mine;
#pragma unroll
  for (int k = 1; k < 32; k *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, k);
    if (lane >= k) inc += up;
  }
  if (lane == 31) scratch[warp] = inc;
  if (tid == 0) {
    out->b = p.B;
    out->left = 0;
  }
  __syncthreads();
  long long before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const long long chunk = max(static_cast<long long>(u.least), div_up(total, gridDim.x));
  const long long start = blockIdx.x * chunk;
  if (start >= before && start < before + mine) {
    // The thread whose items hold the start finds the item, the head and the tile.
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      if (per > 1) one = places(i, r);  // else still at hand
      if (start >= at + one * mult) {
        at += one * mult;
        continue;
      }
      CacheWalk w;
      w.b = lay ? i / p.Hkv : i;
      w.h = lay ? i - w.b * p.Hkv
                : (start - at < (1ll << 31) && one < (1ll << 31)
                       ? static_cast<uint32_t>(start - at) / static_cast<uint32_t>(one)
                       : static_cast<int>((start - at) / one));
      w.off = start - at - (lay ? 0 : w.h * one);
      w.chunk = chunk;
      w.left = min(chunk, total - start);
      w.r = r;
      CacheSeg s;
      for (w.t = 0; w.t < r.tiles - 1; ++w.t) {
        const long long size = u.places(r, w.h, w.t, s);
        if (w.off < size) break;
        w.off -= size;
      }
      *out = w;
      break;
    }
  }
  __syncthreads();
}

// Partial results of a cut unit: slot 2c holds the piece at the start of CTA c's share (a
// unit begun earlier), slot 2c + 1 the piece at its end.  Slot s: R rows of D fp32 at
// o + s * R * D, and R (reference, sum) pairs at ml + s * R.
// count[c]: pieces so far of the unit that was cut at the end of CTA c's share; zero before
// and after every call.
struct CacheParts {
  int* status;
  int* count;
  float* o;
  float2* ml;
};

__device__ __forceinline__ CacheParts cache_parts(void* ws, int grid, int rows, int d) {
  CacheParts c;
  c.status = static_cast<int*>(ws);
  c.count = c.status + 4;
  c.o = reinterpret_cast<float*>(c.count + (grid + 3) / 4 * 4);
  c.ml = reinterpret_cast<float2*>(c.o + static_cast<int64_t>(grid) * 2 * rows * d);
  return c;
}

}  // namespace bsa
