// bsa_cache_tile.cuh -- attention over the paged 8-bit cache for many query rows: tiles of
// 128 rows (queries of a tile times query heads of a kv head), prompts and their chunks.
//
// Bound: the tensor pipe (4 D flops a row and key), with the conversion of the cache beside
// it.  Products are tcgen05.mma kind::f16 on fp16 operands, in which every stored number is
// exact; e4m3 operands (kind::f8f6f4) would need the queries and the weights rounded to 8
// bits, and int8 has no such kind.  A step is 128 keys, two pieces of 64 from anywhere in the
// cache; work is split on the device (bsa_cache_sched.cuh), one persistent CTA per SM:
//   warp 0      S issuer (one thread): S(t) = Q K(t)^T into one of three TMEM buffers, which
//               lets it run ahead of the softmax.
//   warp 1      PV issuer: O += P(t) V(t), P read from the S buffer it was written over.
//   warp 2      looks pages and scales up, a batch of four steps at a time, up to eight steps
//               ahead, while the numbers of the steps before are on their way.
//   warp 3      idle: the roles after it have to begin at a warpgroup.
//   softmax     warps 4-11, 64 scores a thread: lanes t and t + 16 hold the two halves of each
//               piece of a row.  The K scale of a page belongs to 16 keys at least, so it is
//               folded into the exponent's multiplier per group of 16, and log2 of the V scale
//               into its addend, as in the decode kernel: w = exp2(s + log2 vs - m), the sum
//               takes w / vs, weights are rounded to fp16 (2^-11) relative to a reference m that
//               makes the largest 2^7 to 2^15, as there.  An item's O is read out at the next
//               item's first step.
//   converters  warps 12-15 for K, 16-19 for V: stored numbers, loaded into registers a step
//               ahead, to fp16 tiles in the 128-byte-swizzled layout that the products read.  A
//               lane's pieces are chosen so that its writes meet no other's banks.  At an item's
//               first step all eight turn its queries into an fp16 tile, bf16 ones scaled per
//               row by a power of two into fp16's range.
// Shared memory holds two tiles each of Q, K and V in fp16 (192 KB): a step writes 64 KB of
// fp16 into it and the products read 96 KB of it, which bounds a step at about 1,280 cycles
// against the 1,024 of its products.
//
// Measured, 2,048 queries on 16,384 tokens, 32 query and 8 kv heads, d = 128, e4m3: 526 us,
// 980 TFLOP/s, 0.51 of a cuBLAS bf16 product.  A step takes about 2,450 cycles: the softmax
// warps' chain of waits, TMEM loads, maxima, exponentials and conversions is the limit (without
// the conversion of the cache the time is 12 % less, without the exponentials 5 %, with an
// eighth of the products 3 %).  What counted on the way there, at these sizes: the raw bytes by
// TMA into shared memory and the conversion from there (664 us) against loads into registers;
// two S buffers instead of three (606); scores read from TMEM twice with 32 at a time in
// registers, where all threads have 96 registers (592), against once with the register split
// below (577); causal and window masks decided by the look-ups, once a step, instead of by
// votes (554); requesting the next step's numbers before the fence that publishes this one's
// (531).  A few registers spilled in these loops cost a quarter of the speed, and unrolling more
// of them costs as much in instruction fetches: the roles' loops together just fit that cache.
//
// Three chunks of up to 1,000 queries under a block layout that leaves them five blocks of 64
// each (16 heads, 64 of a tile's 128 rows in use): 58 us.  Of the 6 us that an item takes there
// about 2 are its change: the queries (2 us; 5 with one thread a row of them) and the read-out
// of O before it (1.6 us), partly beside the last steps.
//
// Every wait is bounded, by a count of tries: one that runs out records a timeout, and all roles
// leave their loops, let the products in flight finish, free TMEM and return.
#pragma once

#include "bsa_cache_decode.cuh"

namespace bsa {

template <int D>
struct TileCfg {
  static constexpr int kThreads = 640;
  static constexpr int kRows = 128;
  // Registers a thread: of the launch, then of warps 0-3, the softmax and the converter warps.
  static constexpr int kRegs = 96, kRegCtl = 64, kRegSoft = 120, kRegConv = 88;
  static_assert(128 * kRegCtl + 256 * (kRegSoft + kRegConv) <= kThreads * kRegs, "register split");
  static constexpr int kTileB = 128 * D * 2;   // one fp16 tile of Q, K or V
  static constexpr int kHalfB = 128 * 128;     // its 64-column halves, [128][64] swizzled
  static constexpr int kInfo = 8;              // steps looked up ahead
  static constexpr int kItems = 8;             // items whose row factors are kept
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTileB;
  static constexpr int kOffV = kOffK + 2 * kTileB;
  static constexpr int kOffFactor = kOffV + 2 * kTileB;          // [kItems][128] fp32
  static constexpr int kOffSegs = kOffFactor + kItems * 128 * 4; // the producer's segments
  static constexpr int kOffInfo = kOffSegs + 4 * 64;
  static constexpr int kInfoB = 256;
  static constexpr int kOffBar = kOffInfo + kInfo * kInfoB;
  // barriers
  static constexpr int kSF = 0;                 // [3] S(t) computed
  static constexpr int kPVD = 3;                // [3] PV(t) complete
  static constexpr int kPF = 6;                 // [3] P(t) written (softmax warps)
  static constexpr int kKF = 9;                 // [2] K(t) converted (4 warps)
  static constexpr int kVF = 11;                // [2] V(t) converted (4 warps)
  static constexpr int kQF = 13;                // [kItems] Q of an item converted
  static constexpr int kIF = kQF + kItems;      // [kInfo] step looked up
  static constexpr int kIE = kIF + kInfo;       // [kInfo] step no longer needed
  static constexpr int kQE = kIE + kInfo;       // [2] Q tile read by its item's last product
  static constexpr int kDrain = kQE + 2;        // [2] S, PV issuers' last products
  static constexpr int kJoin = kDrain + 2;      // softmax warps
  static constexpr int kNumBars = kJoin + 1;
  static constexpr int kOffScan = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffWalk = kOffScan + 32 * 8;
  static constexpr int kOffCtl = kOffWalk + 96;  // TMEM address, status, abort flag, join
  static constexpr int kSmemB = kOffCtl + 16 + 1024;
  static_assert(kSmemB <= 232448, "shared memory");
  // Two CTAs never share an SM: each takes all 512 TMEM columns.
  static constexpr int kLaunchSmem = kSmemB > 120 * 1024 ? kSmemB : 120 * 1024;
  static constexpr int kOCol = 384;  // TMEM columns: three S buffers (P over them), O
  static constexpr uint32_t kIdesc = (1u << 4);  // fp16 inputs, fp32 sums
  static constexpr uint32_t kIdescS = kIdesc | (128u / 8) << 17 | (128u / 16) << 24;
  static constexpr uint32_t kIdescPV = kIdesc | 1u << 16 | (D / 8u) << 17 | (128u / 16) << 24;
};

constexpr int kStepMask = 8;  // beside DecodeFlags: some query of the tile does not see all keys

// What the roles need to know of a step.
struct alignas(16) TileStep {
  int flags;        // DecodeFlags, kStepMask
  int cut;          // bits 0-7: groups of 16 keys that are there; bit 8: of those, some keys unseen
  int key0[2];      // first key of each piece (kNoKeys: none)
  uint32_t off[8];  // per group: where it starts in the cache (in 16 rows; 0 where it is not there)
  struct {
    float ks[2];    // scales of the scores (1 where the keys are not there)
    float lv[2];    // log2 of the value scales (-inf where the keys are not there)
  } f[4];           // of two groups each
  float rv[8];      // reciprocals of the value scales (0 where the keys are not there)
  CacheSeg seg;     // of every step (13 words)
};
static_assert(sizeof(TileStep) <= 256, "step slots");

// A barrier of a ring of N: its address and the parity of the phase to wait for (or to fill)
// next.
template <int N>
struct RingBar {
  uint32_t bar, first, parity;
  __device__ __forceinline__ explicit RingBar(uint32_t b) : bar(b), first(b), parity(0) {}
  __device__ __forceinline__ void advance() {
    bar += 8;
    if (bar == first + 8 * N) {
      bar = first;
      parity ^= 1;
    }
  }
  __device__ __forceinline__ int index() const { return static_cast<int>(bar - first) >> 3; }
  __device__ __forceinline__ bool wait(volatile int* ctl, int site) const {
    return mbar_wait_tries(bar, parity, ctl, site);
  }
};

// ---------------------------------------------------------------------- look-ups

template <int D>
__device__ __forceinline__ void tile_lookup(const CacheFwdParams& p, uint8_t* smem,
                                            const CacheUnits& units, volatile int* ctl) {
  using Cfg = TileCfg<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  CacheWalk walk = *reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk);
  // Up to four steps of one segment at a time: lane 8 i + j looks up group j (16 keys) of step
  // i.  A batch is looked up while the ring still holds the steps of the one before.
  struct Batch {
    int seg, s, steps;  // place of its segment, first step, steps of the segment (0: the end)
    int key, pid, tile;
    float ks, vs;
  };
  auto seg_at = [&](int i) -> CacheSeg& {
    return *reinterpret_cast<CacheSeg*>(smem + Cfg::kOffSegs + 64 * (i & 3));
  };
  auto place = [&](const Batch& before, Batch& x) {
    if (before.s + 4 < before.steps) {
      x.seg = before.seg;
      x.s = before.s + 4;
      x.steps = before.steps;
    } else {
      CacheSeg seg;
      walk.next(units, seg);  // every lane walks the same way
      x.seg = before.seg + 1;
      x.s = 0;
      x.steps = seg.nq == 0 ? 0 : max(1, (seg.s1 - seg.s0 + 1) / 2);
      if (lane == 0) seg_at(x.seg) = seg;
      __syncwarp();
    }
    const CacheSeg& seg = seg_at(x.seg);
    const int piece = seg.s0 + 2 * x.s + (lane >> 2);
    x.key = kNoKeys;
    if (x.steps > 0 && piece < seg.s1)
      x.key = p.row_ptr != nullptr ? p.col_idx[seg.rp + (piece >> (p.block_shift - 6))] : piece << 6;
  };
  auto find_page = [&](Batch& x) {
    x.pid = -1;
    if (x.key == kNoKeys) return;
    const CacheSeg& seg = seg_at(x.seg);
    if (p.row_ptr != nullptr) {
      const int piece = seg.s0 + 2 * x.s + (lane >> 2), sub = p.block_shift - 6;
      x.key = (x.key << p.block_shift) + ((piece & ((1 << sub) - 1)) << 6);
    }
    const int k = x.key + 16 * (lane & 3);
    if (k < seg.pos0 + seg.nq && k + 16 > seg.lo_key)
      x.pid = p.table[static_cast<int64_t>(seg.b) * p.max_pages + (k >> p.page_shift)];
  };
  auto find_scales = [&](Batch& x) {
    x.tile = -1;
    if (x.pid < 0 || x.pid >= p.n_pages) return;
    x.tile = x.pid * p.Hkv + seg_at(x.seg).h;
    x.ks = p.k_scale[x.tile];
    x.vs = p.v_scale[x.tile];
  };
  Batch cur{}, next{};
  next.seg = -1;
  const int i = lane >> 3, j = lane & 7;
  bool any = false;  // cur holds a batch
  for (int t = 0;;) {
    place(any ? cur : next, next);
    if (any) {
      // Publishes cur, whose look-ups have been made.
      const bool end = cur.steps == 0;
      const int n = end ? 1 : min(4, cur.steps - cur.s);
      bool ok = true;
#pragma unroll 1
      for (int u = t; u < t + n; ++u)
        ok = ok && (u < Cfg::kInfo || mbar_wait_tries(bar(Cfg::kIE + u % Cfg::kInfo),
                                                      (u / Cfg::kInfo - 1) & 1, ctl, kSiteProdKEmpty));
      if (!__all_sync(0xffffffffu, ok)) break;
      const int slot = (t + i) % Cfg::kInfo;
      TileStep& st = *reinterpret_cast<TileStep*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
      const bool on = cur.tile >= 0 && !end;
      const uint32_t there = __ballot_sync(0xffffffffu, on);
      if (i < n) {
        const float lv = log2_scale(cur.vs);
        const int row = (cur.key + 16 * (j & 3)) & ((1 << p.page_shift) - 1);
        st.off[j] = on ? (static_cast<uint32_t>(cur.tile) << (p.page_shift - 4)) + (row >> 4) : 0;
        st.f[j >> 1].ks[j & 1] = on ? cur.ks : 1.f;
        st.f[j >> 1].lv[j & 1] = on ? lv : -INFINITY;
        st.rv[j] = on ? ex2_approx(-lv) : 0.f;
        if ((j & 3) == 0) st.key0[j >> 2] = cur.key;
        const CacheSeg& seg = seg_at(cur.seg);
        // Lanes 0 and 4 have the two pieces' first keys.  Of some keys: the tile's last query
        // (or its window's first key) cuts; of some query: the first one (the last's window).
        const int lo = cur.key - seg.lo_key, hi = seg.pos0 + seg.nq - 64 - cur.key;
        const uint32_t mine = 255u << (8 * i), active = 0xffffffffu >> (32 - 8 * n);
        const uint32_t part = __ballot_sync(active, (j & 3) == 0 && (lo < 0 || hi < 0));
        const bool inner = (p.window >= 0 && cur.key < seg.pos0 + seg.nq - 1 - p.window) ||
                           cur.key > seg.pos0 - 63 || !on;
        const uint32_t mask = __ballot_sync(active, inner);
        if (j == 0) {
          st.cut = (there & mine) >> (8 * i) | (part & mine ? 256 : 0);
          st.flags = end ? kStageEnd
                         : (cur.s + i == 0 ? kStageFirst : 0) |
                               (cur.s + i + 1 == cur.steps ? kStageLast : 0) | (mask & mine ? kStepMask : 0);
        }
        const int* from = reinterpret_cast<const int*>(&seg);
        for (int w = j; w < static_cast<int>(sizeof(CacheSeg) / 4); w += 8)
          reinterpret_cast<int*>(&st.seg)[w] = from[w];
      }
      __syncwarp();
      if (i < n && j == 0) mbar_arrive(bar(Cfg::kIF + slot));
      if (end) break;
      t += n;
    }
    find_page(next);
    find_scales(next);
    cur = next;
    any = true;
  }
}

// ------------------------------------------------------------------- MMA issuers

template <int D>
struct TileDescs {
  using Cfg = TileCfg<D>;
  uint32_t hi, q0, k0, v0;
  __device__ __forceinline__ explicit TileDescs(uint32_t sbase) {
    const uint64_t k = sdesc_sw128(sbase + Cfg::kOffK, 16, 1024);
    hi = static_cast<uint32_t>(k >> 32);
    k0 = static_cast<uint32_t>(k);
    q0 = static_cast<uint32_t>(sdesc_sw128(sbase + Cfg::kOffQ, 16, 1024));
    v0 = static_cast<uint32_t>(sdesc_sw128(sbase + Cfg::kOffV, Cfg::kHalfB, 1024));
  }
};

template <int D>
__device__ __forceinline__ void tile_mma_s(uint8_t* smem, uint32_t tmem, volatile int* ctl) {
  using Cfg = TileCfg<D>;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const TileDescs<D> md(sbase);
  RingBar<Cfg::kInfo> info(bar(Cfg::kIF));
  RingBar<Cfg::kItems> queries(bar(Cfg::kQF));
  RingBar<2> keys(bar(Cfg::kKF));
  RingBar<3> done(bar(Cfg::kPVD));
  uint32_t s = 0, k = 0, q = Cfg::kTileB >> 4;  // S buffer's columns, offsets of the K, Q tile
  for (int t = 0;; ++t) {
    if (!info.wait(ctl, kSiteCacheInfo)) break;
    const int flags =
        reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + info.index() * Cfg::kInfoB)->flags;
    mbar_arrive(info.bar + 8 * Cfg::kInfo);  // its kIE
    info.advance();
    if (flags & kStageEnd) break;
    if (flags & kStageFirst) {
      if (!queries.wait(ctl, kSiteMmaStage)) break;
      queries.advance();
      q ^= Cfg::kTileB >> 4;
    }
    if (!keys.wait(ctl, kSiteMmaStage)) break;
    keys.advance();
    if (t >= 3) {  // S[t % 3] was last read by PV(t - 3)
      if (!done.wait(ctl, kSiteMmaPvDone)) break;
      done.advance();
    }
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * Cfg::kHalfB + (kk & 3) * 32) >> 4;
      tc_mma_ss_lh(tmem + s, md.q0 + q + off, md.hi, md.k0 + k + off, md.hi, Cfg::kIdescS, kk > 0 ? 1u : 0u);
    }
    tc_commit(bar(Cfg::kSF) + s / 16);
    if (flags & kStageLast) tc_commit(bar(Cfg::kQE) + (q ? 8 : 0));
    s = s == 256 ? 0 : s + 128;
    k ^= Cfg::kTileB >> 4;
  }
  tc_commit(bar(Cfg::kDrain));
  mbar_drain_wait(bar(Cfg::kDrain), 0);
}

template <int D>
__device__ __forceinline__ void tile_mma_pv(uint8_t* smem, uint32_t tmem, volatile int* ctl) {
  using Cfg = TileCfg<D>;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const TileDescs<D> md(sbase);
  RingBar<Cfg::kInfo> info(bar(Cfg::kIF));
  RingBar<3> weights(bar(Cfg::kPF));
  RingBar<2> values(bar(Cfg::kVF));
  uint32_t ps = 0, v = 0;  // columns of the S buffer, offset of the V tile
  for (;;) {
    if (!info.wait(ctl, kSiteCacheInfo)) break;
    const int flags =
        reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + info.index() * Cfg::kInfoB)->flags;
    mbar_arrive(info.bar + 8 * Cfg::kInfo);
    info.advance();
    if (flags & kStageEnd) break;
    // V(t) converted, P(t) written (at an item's first step: the previous item's O read out
    // before that).
    if (!values.wait(ctl, kSiteMmaStage) || !weights.wait(ctl, kSiteMmaPFull)) break;
    values.advance();
    weights.advance();
    tc_fence_after();
    const bool first = flags & kStageFirst;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)  // 16 keys each
      tc_mma_ts_lh(tmem + Cfg::kOCol, tmem + ps + kk * 8, md.v0 + v + ((kk * 16 * 128) >> 4), md.hi,
                   Cfg::kIdescPV, kk == 0 && first ? 0u : 1u);
    tc_commit(bar(Cfg::kPVD) + ps / 16);
    ps = ps == 256 ? 0 : ps + 128;
    v ^= Cfg::kTileB >> 4;
  }
  tc_commit(bar(Cfg::kDrain + 1));
  mbar_drain_wait(bar(Cfg::kDrain + 1), 0);
}

// -------------------------------------------------------------------- converters

// A load that stays where it is written: ahead of the waits that follow it.
__device__ __forceinline__ uint4 load16(const void* ptr) {
  uint4 x;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(ptr));
  return x;
}

// Queries of a tile into fp16, a share of the rows for each of eight warps: 16 bytes a lane, as
// many rows at once as a warp holds, a few loads in flight.
template <class A, int D, bool DIFF>
__device__ __forceinline__ void tile_queries(const CacheFwdParams& p, const CacheSeg& s, uint8_t* tile,
                                             float* factor, int warp, int lane) {
  constexpr int L = D / 8, RPI = 32 / L;  // lanes of a row, rows at once
  constexpr int N = 4;
  const int c = lane % L, rows = s.nq * p.group;
  const A* const q = static_cast<const A*>(p.q) + static_cast<int64_t>(s.q0) * p.q_token_stride +
                     static_cast<int64_t>(s.h) * p.group * p.q_head_stride + 8 * c;
  tile += (c >> 3) * TileCfg<D>::kHalfB;
#pragma unroll 1
  for (int i = 0; i < 16; i += N * RPI) {
    const int first = warp * 16 + i + lane / L;
    uint4 x[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int r = first + u * RPI, qi = static_cast<int>((r * p.group_inv) >> 16);
      x[u] = make_uint4(0, 0, 0, 0);
      // Split queries: the columns of the other map's key half are zero.
      const bool split = DIFF && p.split;
      if (r < rows && !(split && c / (L / 2) != (r & 1)))
        x[u] = *reinterpret_cast<const uint4*>(q + qi * p.q_token_stride + (r - qi * p.group) * p.q_head_stride -
                                               (split ? (r & 1) * (D / 2) : 0));
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int r = first + u * RPI;
      float back = 1.f;
      if constexpr (!std::is_same<A, __half>::value) {
        // The row's largest number to [2^14, 2^15), as far as the factors' exponents go.
        uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
        for (int k = 1; k < L; k *= 2) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, k));
        const int e = static_cast<int>(max(top & 0xFFFFu, top >> 16) >> 7) - 127;
        const int k = max(-113, min(120, 14 - e));
        const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
        back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float2 f = act_to_float2<A>(w[v]);
          w[v] = float2_to_act<__half>(f.x * up, f.y * up);
        }
        x[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (c == 0) factor[r] = back;
      *reinterpret_cast<uint4*>(tile + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x[u];
    }
  }
}

// One side (V: values, else keys) and half the queries; 128 threads.  One piece of code for both.
template <class A, class C, int D, bool DIFF>
__device__ __forceinline__ void tile_convert(const CacheFwdParams& p, uint8_t* smem, const bool V,
                                             volatile int* ctl) {
  using Cfg = TileCfg<D>;
  constexpr int RPP = 128 * 16 / D;   // rows of a pass of the 128 threads, 16 numbers each
  constexpr int NP = 128 / RPP;       // passes of a tile
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  // Row of a pass and 16-number piece of it.  d = 128: eight neighbouring lanes read the left
  // half of one row and the right half of the next, and write four 16-byte pieces of an even
  // and four of an odd row, which the swizzle puts on different banks.
  const int piece = D == 128 ? lane & 7 : lane & 3;
  const int r0 = warp * (RPP / 4) +
                 (D == 128 ? (((lane >> 2) ^ (lane >> 3)) & 1) | ((lane >> 3) & 2) : lane >> 2);
  const uint8_t* const cache = (V ? p.v_cache : p.k_cache) + (r0 & 15) * D + piece * 16;
  const int row0 = (piece >> 2) * Cfg::kHalfB + r0 * 128;
  const int dst0 = row0 + (((2 * (piece & 3)) ^ (r0 & 7)) << 4);
  const int dst1 = row0 + (((2 * (piece & 3) + 1) ^ (r0 & 7)) << 4);
  uint4 x[NP];
  // A step's stored numbers into registers; what no query of the tile sees is zero (the cache
  // may hold anything there).
  auto load = [&](const TileStep& st) {
    uint32_t off[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) off[i] = st.off[RPP == 16 ? i : (i * RPP + r0) >> 4];
#pragma unroll
    for (int i = 0; i < NP; ++i) x[i] = load16(cache + static_cast<int64_t>(off[i]) * (16 * D));
    const int cut = st.cut;
    if (cut != 255) {
      const int lo = st.seg.lo_key, last = st.seg.pos0 + st.seg.nq - 1;
      const int k0 = st.key0[0] + r0, k1 = st.key0[1] + r0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int key = (i < NP / 2 ? k0 : k1) + (i * RPP & 63);
        if (!(cut >> ((i * RPP + r0) >> 4) & 1) || key < lo || key > last) x[i] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  // Rings: look-ups, and what last read the tile that a step overwrites: S(t - 2) for K,
  // PV(t - 2) for V.
  RingBar<Cfg::kInfo> info(bar(Cfg::kIF));
  RingBar<3> free2(bar(V ? Cfg::kPVD : Cfg::kSF));
  int tile = V ? Cfg::kOffV : Cfg::kOffK;
  RingBar<2> free_q(bar(Cfg::kQE));
  int item = 0, flags = 0;
  bool ok = true;
  auto step = [&]() -> const TileStep& {
    return *reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + info.index() * Cfg::kInfoB);
  };
  // Iteration t stores step t and then requests step t + 1 (t = -1: requests the first).
  for (int t = -1;; ++t) {
    if (t >= 0) {
      if (flags & kStageFirst) {
        if (item >= 2) {  // the products of the item before the last
          if (!__all_sync(0xffffffffu, free_q.wait(ctl, kSiteProdKEmpty))) break;
          free_q.advance();
        }
        tile_queries<A, D, DIFF>(p, step().seg, smem + Cfg::kOffQ + (item & 1) * Cfg::kTileB,
                           reinterpret_cast<float*>(smem + Cfg::kOffFactor) + (item % Cfg::kItems) * 128,
                           warp + (V ? 4 : 0), lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Cfg::kQF + item % Cfg::kItems));
        ++item;
      }
      if (t >= 2) {
        if (!__all_sync(0xffffffffu, free2.wait(ctl, V ? kSiteProdVEmpty : kSiteProdKEmpty))) break;
        free2.advance();
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t h[8];
        stored4_to_half2<C>(x[i].x, h[0], h[1]);
        stored4_to_half2<C>(x[i].y, h[2], h[3]);
        stored4_to_half2<C>(x[i].z, h[4], h[5]);
        stored4_to_half2<C>(x[i].w, h[6], h[7]);
        const int at = tile + i * RPP * 128;
        *reinterpret_cast<uint4*>(smem + dst0 + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(smem + dst1 + at) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      const uint32_t release = info.bar + 8 * Cfg::kInfo;
      info.advance();
      ok = __all_sync(0xffffffffu, info.wait(ctl, kSiteCacheInfo));
      flags = step().flags;
      if (ok && !(flags & kStageEnd)) load(step());
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(V ? Cfg::kVF : Cfg::kKF) + 8 * (t & 1));
        mbar_arrive(release);
      }
      tile += t & 1 ? -Cfg::kTileB : Cfg::kTileB;
    } else {
      ok = __all_sync(0xffffffffu, info.wait(ctl, kSiteCacheInfo));
      flags = step().flags;
      if (ok && !(flags & kStageEnd)) load(step());
    }
    if (!ok || (flags & kStageEnd)) break;
  }
}

// ----------------------------------------------------------------------- softmax

// FOLD: positive scale and no soft-cap, so that the scores' factor goes into the exponent's
// multiplier; else they are transformed first.
template <class A, int D, bool FOLD, bool DIFF>
__device__ __forceinline__ void tile_softmax(const CacheFwdParams& p, uint8_t* smem, uint32_t tmem,
                                             const CacheParts& parts, int* join_flag, volatile int* ctl) {
  using Cfg = TileCfg<D>;
  constexpr int R = Cfg::kRows, kJoinRows = 4;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const int w8 = (threadIdx.x >> 5) - 4, wg = w8 >> 2, wq = w8 & 3;
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const int row = wq * 32 + wg * 16 + (lane & 15);
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32 + wg * 16) << 16);
  const uint32_t to = tl + Cfg::kOCol;
  const int qi = static_cast<int>((row * p.group_inv) >> 16);
  auto wait_ring = [&](const auto& ring, int site) -> bool {
    const bool w = __all_sync(0xffffffffu, ring.wait(ctl, site));
    if (w) tc_fence_after();
    return w;
  };
  uint32_t join_phase = 0;
  auto meet = [&]() -> bool {  // of the softmax warps
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Cfg::kJoin));
    const bool ok = mbar_wait_tries(bar(Cfg::kJoin), join_phase, ctl, kSiteCacheJoin);
    join_phase ^= 1;
    return __all_sync(0xffffffffu, ok);
  };

  CacheSeg seg{};          // of the item whose O is pending
  float m = -INFINITY, l = 0.f, rf = 1.f;
  int qpos = -1;
  bool live = false;

  // The finished item's rows: its O (this thread's columns 64 c + 32 half + ..) scaled and
  // stored, or left as a piece of a cut unit.
  auto finish = [&]() -> bool {
    const bool whole = seg.starts && seg.ends;
    const int head = seg.h * p.group + row - qi * p.group;
    const int64_t orow = static_cast<int64_t>(seg.q0 + qi) * p.Hq + head;
    float f = 1.f, z = l, top = m;
    if (whole) {
      if (p.sinks != nullptr && live) {
        const float sink = p.sinks[head] * kLog2e;
        const float mx = fmaxf(m, sink);
        f = m == -INFINITY ? 0.f : ex2_approx(m - mx);
        z = z * f + (sink == -INFINITY ? 0.f : ex2_approx(sink - mx));
        top = mx;
      }
      f = z == 0.f ? 0.f : f / z;
    }
    const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (seg.starts ? 1 : 0)) * R + row;
#pragma unroll 1
    for (int c = 0; c < D / 64; ++c) {
      uint32_t r[32];
      tmem_ld_16x32bx2_x32<32>(to + c * 64, r);
      tmem_ld_wait(r);
      if constexpr (DIFF) {
        if (whole) {
          // The row pair's two lanes exchange halves of these columns, and each stores one.
          const bool odd = lane & 1;
          const float lam = live ? diff_lam(p, orow >> 1, head >> 1) : 0.f;
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float y[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float a = __uint_as_float(r[2 * i + u]) * f, b = __uint_as_float(r[16 + 2 * i + u]) * f;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              y[u] = odd ? fmaf(-lam, b, got) : fmaf(-lam, got, a);
            }
            w[i] = float2_to_act<A>(y[0], y[1]);
          }
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<A*>(p.out) + (orow >> 1) * D + c * 64 + half * 32 +
                                                  (odd ? 16 : 0));
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
          continue;
        }
      }
      if (!live) continue;
      if (whole) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<A*>(p.out) + orow * D + c * 64 + half * 32);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = float2_to_act<A>(__uint_as_float(r[8 * q + 2 * i]) * f,
                                    __uint_as_float(r[8 * q + 2 * i + 1]) * f);
          dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        uint4* dst = reinterpret_cast<uint4*>(parts.o + slot * D + c * 64 + half * 32);
#pragma unroll
        for (int q = 0; q < 8; ++q) dst[q] = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
      }
    }
    if (live && half == 0) {
      if (whole) p.lse[orow] = z == 0.f ? -INFINITY : (top + log2f(z)) * kLn2;
      else parts.ml[slot] = make_float2(m, l);
    }
    return true;
  };
  // After a cut unit's piece is stored: the CTA that left the last one joins them.
  auto join = [&]() -> bool {
    if (seg.starts && seg.ends) return true;
    // Once for the count, then for what it said, then for the word's next use.
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {
      if (!meet()) return false;
      if (i == 0 && w8 == 0 && lane == 0) {
        __threadfence();
        int* count = parts.count + (blockIdx.x - seg.before);
        const bool now = add_acq_rel(count, 1) == seg.before + seg.more;
        if (now) *count = 0;
        *join_flag = now;
      }
      if (i == 1 && *reinterpret_cast<volatile int*>(join_flag)) {
#pragma unroll 1
        for (int r = DIFF ? 2 * w8 : w8; r < seg.nq * p.group; r += 8 * kJoinRows)
          join_rows<A, D, R, kJoinRows, DIFF>(p, parts, seg, blockIdx.x - seg.before, seg.before + seg.more, r,
                                              DIFF ? 16 : 8, lane);
      }
    }
    return true;
  };

  // A group's factor of the scores (one, where they have been changed already); a zero one would
  // turn a masked score into a NaN.
  auto factor = [&](float ks) { return FOLD ? fmaxf(rf * ks, 1.17549435e-38f) : 1.f; };
  bool pending = false;
  RingBar<Cfg::kInfo> info(bar(Cfg::kIF));
  RingBar<Cfg::kItems> queries(bar(Cfg::kQF));
  RingBar<3> scores(bar(Cfg::kSF)), before(bar(Cfg::kPVD));  // S(t), PV(t - 1)
  uint32_t ts = tl;  // the step's S buffer
  if (!wait_ring(info, kSiteCacheInfo)) return;
  for (int t = 0;; ++t) {
    const TileStep& st =
        *reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + info.index() * Cfg::kInfoB);
    const int4 head = *reinterpret_cast<const int4*>(&st);
    const int flags = head.x;
    const bool first = flags & kStageFirst;
    if (flags & (kStageFirst | kStageEnd)) {
      // The previous item's O goes out before this step's P is handed over (the product that
      // reads it overwrites O).
      if (pending && !(wait_ring(before, kSiteSoftItemDone) && finish() && join())) break;
      if (flags & kStageEnd) break;
      pending = true;
      if (!wait_ring(queries, kSiteSoftSFull)) break;
      seg = st.seg;
      live = qi < seg.nq;
      qpos = live ? seg.pos0 + qi : -1;
      rf = reinterpret_cast<const float*>(smem + Cfg::kOffFactor)[queries.index() * 128 + row] *
           (FOLD || p.softcap_log2 == 0.f ? p.scale_log2 : p.softcap_inv);
      queries.advance();
      m = -INFINITY;
      l = 0.f;
    }
    if (!wait_ring(scores, kSiteSoftSFull)) break;
    scores.advance();
    if constexpr (!FOLD) {
      // Scores changed in place, in a loop: unrolled it would not fit the instruction cache (with
      // a soft-cap 1.17 ms for the case of the file's head, 1.04 so).
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t x[32];
        tmem_ld_16x32bx2_x32<32>(ts + 64 * h, x);
        const float2 ks = *reinterpret_cast<const float2*>(st.f[2 * h + half].ks);
        const float c0 = rf * ks.x, c1 = rf * ks.y;
        tmem_ld_wait(x);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float y0 = __uint_as_float(x[i]) * (i < 16 ? c0 : c1);
          float y1 = __uint_as_float(x[i + 1]) * (i < 16 ? c0 : c1);
          if (p.softcap_log2 > 0.f) softcap2(y0, y1, p.softcap_log2);
          x[i] = __float_as_uint(y0);
          x[i + 1] = __float_as_uint(y1);
        }
        tmem_st_16x32bx2_x32<32>(ts + 64 * h, x);
      }
      tmem_st_wait();
    }
    // 32 keys of each piece a thread (lane t the first of a piece, t + 16 the others).
    uint32_t x[2][32];
    tmem_ld_16x32bx2_x32<32>(ts, x[0]);
    tmem_ld_16x32bx2_x32<32>(ts + 64, x[1]);
    float cf[4], la[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 f = *reinterpret_cast<const float4*>(&st.f[2 * h + half]);
      cf[2 * h] = factor(f.x);
      cf[2 * h + 1] = factor(f.y);
      la[2 * h] = f.z;
      la[2 * h + 1] = f.w;
    }
    tmem_ld_wait(x[0]);
    tmem_ld_wait(x[1]);
    float mx = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (flags & kStepMask) {
        // Bit i: score i is seen.
        const int k = (h ? head.w : head.z) + 32 * half;
        int lo = 0, hi = min(31, qpos - k);
        if (p.window >= 0) lo = max(lo, qpos - p.window - k);
        const uint32_t seen = hi < lo ? 0u : (0xffffffffu >> (31 - (hi - lo))) << lo;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!((seen >> i) & 1)) x[h][i] = __float_as_uint(-INFINITY);
      }
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        t0 = fmax3(t0, __uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1]));
        t1 = fmax3(t1, __uint_as_float(x[h][16 + i]), __uint_as_float(x[h][17 + i]));
      }
      mx = fmax3(mx, fmaf(t0, cf[2 * h], la[2 * h]), fmaf(t1, cf[2 * h + 1], la[2 * h + 1]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    float alpha = 1.f;
    if (first) {
      m = mx - kLift;
    } else if (mx > m + (kLift + kSlack)) {
      alpha = ex2_approx(m - (mx - kLift));
      m = mx - kLift;
    }
    const float neg_m = m == -INFINITY ? 0.f : -m;
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t pk[16];
      const float c0 = cf[2 * h], c1 = cf[2 * h + 1];
      const float a0 = la[2 * h] + neg_m, a1 = la[2 * h + 1] + neg_m;
      uint64_t s0 = 0ull, s1 = 0ull;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t y0 = f2_fma(f2_pack(__uint_as_float(x[h][2 * i]), __uint_as_float(x[h][2 * i + 1])),
                                   f2_pack(c0, c0), f2_pack(a0, a0));
        const uint64_t y1 =
            f2_fma(f2_pack(__uint_as_float(x[h][16 + 2 * i]), __uint_as_float(x[h][17 + 2 * i])),
                   f2_pack(c1, c1), f2_pack(a1, a1));
        const uint64_t e0 = f2_pack(ex2_approx(f2_lo(y0)), ex2_approx(f2_hi(y0)));
        const uint64_t e1 = f2_pack(ex2_approx(f2_lo(y1)), ex2_approx(f2_hi(y1)));
        s0 = f2_add(s0, e0);
        s1 = f2_add(s1, e1);
        pk[i] = float2_to_act<__half>(f2_lo(e0), f2_hi(e0));
        pk[8 + i] = float2_to_act<__half>(f2_lo(e1), f2_hi(e1));
      }
      // w / vs
      const float2 rv = *reinterpret_cast<const float2*>(st.rv + 4 * h + 2 * half);
      sum = fmaf(f2_lo(s0) + f2_hi(s0), rv.x, fmaf(f2_lo(s1) + f2_hi(s1), rv.y, sum));
      // over scores that both lanes of the row have read
      tmem_st_16x32bx2_x16<16>(ts + 32 * h, pk);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    l = l * alpha + sum;
    if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
      // PV(t - 1) must be complete before O is rescaled.
      if (!wait_ring(before, kSiteSoftPvDone)) break;
#pragma unroll 1
      for (int g = 0; g < D / 64; ++g) {
        uint32_t r[32];
        tmem_ld_16x32bx2_x32<32>(to + g * 64, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
        tmem_st_16x32bx2_x32<32>(to + g * 64, r);
      }
    }
    // The next step's look-ups, long there, while the weights' stores are under way.
    const uint32_t release = info.bar + 8 * Cfg::kInfo;
    info.advance();
    if (!wait_ring(info, kSiteCacheInfo)) break;
    tmem_st_wait();
    // P(t) handed over, the step's look-ups no longer needed.
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar(Cfg::kPF) + ((ts - tl) >> 4));
      mbar_arrive(release);
    }
    if (t > 0) before.advance();
    ts = ts == tl + 256 ? tl : ts + 128;
  }
  tmem_st_wait();  // TMEM is freed after this: no store of a loop that was left early is under way
}

// ------------------------------------------------------------------------ kernel

// DIFF: differential attention.  Rows 2i and 2i + 1 of a tile are the two maps of an output row.
// Measured, 2,048 queries on 16,384 tokens, 16 heads of two maps, 8 kv heads, d = 128, e4m3: 518
// us, as plain attention of 32 heads.
template <class A, class C, int D, bool FOLD, bool DIFF>
__global__ void __launch_bounds__(640, 1) bsa_cache_tile_kernel(const CacheFwdParams p, void* workspace) {
  using Cfg = TileCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffCtl);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);  // abort word, join flag
  volatile int* const ctl = err;
  const CacheParts parts = cache_parts(workspace, gridDim.x, Cfg::kRows, D);
  // Queries of a tile: as many as fill its rows, and of one layout row.
  int tq_shift = 31 - __clz(static_cast<int>((128u * p.group_inv) >> 16));
  if (p.row_ptr != nullptr) tq_shift = min(tq_shift, p.block_shift);
  // A unit's fixed work (its queries, O, sums) takes about as long as 256 keys.
  const CacheUnits units{p, tq_shift, 6, 4, 4};
  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(Cfg::kSF + i), 1);
      mbar_init(bar(Cfg::kPVD + i), 1);
      mbar_init(bar(Cfg::kPF + i), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Cfg::kKF + i), 4);
      mbar_init(bar(Cfg::kVF + i), 4);
      mbar_init(bar(Cfg::kDrain + i), 1);
      mbar_init(bar(Cfg::kQE + i), 1);
    }
    for (int i = 0; i < Cfg::kItems; ++i) mbar_init(bar(Cfg::kQF + i), 8);
    for (int i = 0; i < Cfg::kInfo; ++i) {
      mbar_init(bar(Cfg::kIF + i), 1);
      mbar_init(bar(Cfg::kIE + i), 8 + 8 + 2);  // converters, softmax, issuers
    }
    mbar_init(bar(Cfg::kJoin), 8);
    err[0] = err[1] = 0;
    fence_mbar_init();
    if (blockIdx.x == 0 && p.status != nullptr) *p.status = 0;
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  cache_split<Cfg::kThreads>(units, reinterpret_cast<long long*>(smem + Cfg::kOffScan),
                             reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    setmaxnreg_dec<Cfg::kRegCtl>();
    // The test knob ends one of these roles before it begins; the others' waits run out.
    if (warp == 0) {
      if (lane == 0 && p.expire_site != kSiteMmaStage) tile_mma_s<D>(smem, tmem, ctl);
    } else if (warp == 1) {
      if (lane == 0 && p.expire_site != kSiteMmaPFull) tile_mma_pv<D>(smem, tmem, ctl);
    } else if (warp == 2) {
      if (p.expire_site != kSiteCacheInfo) tile_lookup<D>(p, smem, units, ctl);
    }
  } else if (warp < 12) {
    setmaxnreg_inc<Cfg::kRegSoft>();
    tile_softmax<A, D, FOLD, DIFF>(p, smem, tmem, parts, err + 1, ctl);
  } else {
    setmaxnreg_dec<Cfg::kRegConv>();
    tile_convert<A, C, D, DIFF>(p, smem, warp >= 16, ctl);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // A wait gives up long after CTA 0 has cleared the word.
  if (threadIdx.x == 0 && err[0] != 0) atomicMax(p.status != nullptr ? p.status : parts.status, err[0]);
}

template <class A, class C, int D, bool FOLD, bool DIFF>
cudaError_t launch_tile_as(const CacheFwdParams& p, void* workspace, int sms,
                           cudaStream_t stream) {
  using Cfg = TileCfg<D>;
  auto* kernel = bsa_cache_tile_kernel<A, C, D, FOLD, DIFF>;
  static int done[64];
  const cudaError_t e = set_smem_once(kernel, Cfg::kLaunchSmem, done);
  if (e != cudaSuccess) return e;
  kernel<<<sms, Cfg::kThreads, Cfg::kLaunchSmem, stream>>>(p, workspace);
  return cudaGetLastError();
}

template <class A, class C, int D, bool DIFF>
cudaError_t launch_tile(const CacheFwdParams& p, void* workspace, int sms, cudaStream_t stream) {
  return p.softcap_log2 == 0.f && p.scale_log2 > 0.f
             ? launch_tile_as<A, C, D, true, DIFF>(p, workspace, sms, stream)
             : launch_tile_as<A, C, D, false, DIFF>(p, workspace, sms, stream);
}

}  // namespace bsa
