// bsa_cache_tile.cuh -- attention over the paged 8-bit cache for many query rows: tiles of
// 128 rows (queries of a tile times query heads of a kv head), prompts and their chunks.
//
// Bound: the tensor pipe (4 D flops a row and key), with the conversion of the cache beside
// it.  Products are tcgen05.mma kind::f16 on fp16 operands, in which every stored number is
// exact; e4m3 operands (kind::f8f6f4) would need the queries and the weights rounded to 8
// bits, and int8 has no such kind.  A step is 128 keys, two pieces of 64 from anywhere in the
// cache; work is split on the device (bsa_cache_sched.cuh), one persistent CTA per SM:
//   warp 0      S issuer (one thread): S(t) = Q K(t)^T into one of three TMEM buffers.
//   warp 1      PV issuer: O += P(t) V(t), P read from the S buffer it was written over.
//   warp 2      looks pages and scales up, two steps and more ahead (ring of 8 steps).
//   softmax     warps 4-11.  Lanes t and t + 16 hold the two pieces of one row.  The K scale
//               of a page belongs to 16 keys at least, so it is folded into the exponent's
//               multiplier per group of 16, and log2 of the V scale into its addend, as in
//               the decode kernel: w = exp2(s + log2 vs - m), the sum takes w / vs, weights
//               are rounded to fp16 relative to the largest (2^-11).  An item's O is read out
//               at the next item's first step.
//   converter   warps 12-15.  Stored numbers from global memory (16 bytes a lane, a step ahead
//               in registers) to fp16 tiles in shared memory, in the 128-byte-swizzled layout
//               that the products read; also the queries, bf16 ones scaled per row by a power
//               of two into fp16's range.
// Shared memory holds two tiles each of Q, K and V (192 KB); a step writes 64 KB into it and
// the products read 96 KB of it, which bounds a step at about 1,280 cycles against the 1,024
// of its products.
//
// Every wait is bounded (WaitCtl): one that runs out records a timeout, and all roles leave
// their loops, let the products in flight finish, free TMEM and return.
#pragma once

#include "bsa_cache_decode.cuh"

namespace bsa {

template <int D>
struct TileCfg {
  static constexpr int kThreads = 512;
  static constexpr int kRows = 128;
  static constexpr int kLaunchRegs = 128;
  static constexpr int kRegCtl = 88, kRegSoft = 160, kRegConv = 104;
  static_assert(kRegCtl + 2 * kRegSoft + kRegConv == 4 * kLaunchRegs, "register split");
  static constexpr int kTileB = 128 * D * 2;   // one fp16 tile of Q, K or V
  static constexpr int kHalfB = 128 * 128;     // its 64-column halves, [128][64] swizzled
  static constexpr int kInfo = 8;              // steps looked up ahead
  static constexpr int kItems = 8;             // items whose row factors are kept
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTileB;
  static constexpr int kOffV = kOffK + 2 * kTileB;
  static constexpr int kOffFactor = kOffV + 2 * kTileB;          // [kItems][128] fp32
  static constexpr int kOffInfo = kOffFactor + kItems * 128 * 4;
  static constexpr int kInfoB = 240;
  static constexpr int kOffBar = kOffInfo + kInfo * kInfoB;
  // barriers
  static constexpr int kSF = 0;                 // [3] S(t) computed
  static constexpr int kPVD = 3;                // [3] PV(t) complete
  static constexpr int kPF = 6;                 // [3] P(t) written (softmax warps)
  static constexpr int kKF = 9;                 // [2] K(t) converted (converter warps)
  static constexpr int kVF = 11;                // [2] V(t) converted
  static constexpr int kQF = 13;                // [kItems] Q of an item converted
  static constexpr int kIF = kQF + kItems;      // [kInfo] step looked up
  static constexpr int kIE = kIF + kInfo;       // [kInfo] step no longer needed
  static constexpr int kDrain = kIE + kInfo;    // [2] S, PV issuers' last products
  static constexpr int kJoin = kDrain + 2;      // softmax warps
  static constexpr int kNumBars = kJoin + 1;
  static constexpr int kOffScan = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffWalk = kOffScan + 16 * 8;
  static constexpr int kOffCtl = kOffWalk + 96;  // TMEM address, status, abort flag, join
  static constexpr int kSmemB = kOffCtl + 16 + 1024;
  static_assert(kSmemB <= 232448, "shared memory");
  // Two CTAs never share an SM: each takes all 512 TMEM columns.
  static constexpr int kLaunchSmem = kSmemB > 120 * 1024 ? kSmemB : 120 * 1024;
  static constexpr int kOCol = 384;
  static constexpr uint32_t kIdesc = (1u << 4);  // fp16 inputs, fp32 sums
  static constexpr uint32_t kIdescS = kIdesc | (128u / 8) << 17 | (128u / 16) << 24;
  static constexpr uint32_t kIdescPV = kIdesc | 1u << 16 | (D / 8u) << 17 | (128u / 16) << 24;
};

// What the roles need to know of a step.
struct TileStep {
  CacheSeg seg;   // of every step (13 words)
  int flags;      // DecodeFlags
  int key0[2];    // first key of each piece (kNoKeys: none)
  int64_t off[8]; // per 16 keys: where they start in the cache (bytes), -1: not there
  float ks[8];    // scale of the scores (1 where the keys are not there)
  float lv[8];    // log2 of the value scale (-inf where the keys are not there)
  float rv[8];    // its reciprocal (0 where the keys are not there)
};
static_assert(sizeof(TileStep) <= 240, "step slots");

// ---------------------------------------------------------------------- look-ups

template <int D>
__device__ __forceinline__ void tile_producer(const CacheFwdParams& p, uint8_t* smem,
                                              const CacheUnits& units, const WaitCtl& ctl) {
  using Cfg = TileCfg<D>;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  CacheWalk walk = *reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk);
  CacheSeg seg;
  int t = 0;
  for (;;) {
    walk.next(units, seg);
    const int steps = seg.nq == 0 ? 1 : max(1, (seg.s1 - seg.s0 + 1) / 2);
    // Four steps at a time: lane 8 i + j looks up group j of step i.
    for (int s = 0; s < steps; s += 4) {
      const int piece = seg.s0 + 2 * s + (lane >> 2);
      int key = kNoKeys, tile = -1;
      int64_t off = -1;
      float ks = 1.f, lv = -INFINITY;
      if (seg.nq > 0 && piece < seg.s1) {
        key = piece << 6;
        if (p.row_ptr != nullptr) {
          const int sub = p.block_shift - 6;
          key = (p.col_idx[seg.rp + (piece >> sub)] << p.block_shift) + ((piece & ((1 << sub) - 1)) << 6);
        }
        const int k = key + 16 * (lane & 3);
        if (k < seg.pos0 + seg.nq && k + 16 > seg.lo_key) {
          const int pid = p.table[static_cast<int64_t>(seg.b) * p.max_pages + (k >> p.page_shift)];
          if (pid >= 0 && pid < p.n_pages) {
            tile = pid * p.Hkv + seg.h;
            ks = p.k_scale[tile];
            lv = log2_scale(p.v_scale[tile]);
            off = ((static_cast<int64_t>(tile) << p.page_shift) + (k & ((1 << p.page_shift) - 1))) * D;
          }
        }
      }
      for (int i = 0; i < 4 && s + i < steps; ++i, ++t) {
        const int slot = t % Cfg::kInfo;
        if (t >= Cfg::kInfo &&
            !mbar_wait_inl(bar(Cfg::kIE + slot), (t / Cfg::kInfo - 1) & 1, ctl, kSiteProdKEmpty))
          return;
        TileStep& st = *reinterpret_cast<TileStep*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
        const int j = lane - 8 * i;
        if (j >= 0 && j < 8) {
          st.off[j] = off;
          st.ks[j] = ks;
          st.lv[j] = lv;
          st.rv[j] = tile < 0 ? 0.f : ex2_approx(-lv);
          if ((j & 3) == 0) st.key0[j >> 2] = key;
        }
        if (lane == 0) {
          st.seg = seg;
          st.flags = seg.nq == 0 ? kStageEnd
                                 : (s + i == 0 ? kStageFirst : 0) | (s + i + 1 == steps ? kStageLast : 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Cfg::kIF + slot));
      }
    }
    if (seg.nq == 0) return;
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
__device__ __forceinline__ void tile_mma_s(uint8_t* smem, uint32_t tmem, const WaitCtl& ctl) {
  using Cfg = TileCfg<D>;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const TileDescs<D> md(sbase);
  int item = -1;
  for (int t = 0;; ++t) {
    const int slot = t % Cfg::kInfo;
    if (!mbar_wait_inl(bar(Cfg::kIF + slot), (t / Cfg::kInfo) & 1, ctl, kSiteCacheInfo)) break;
    const int flags = reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB)->flags;
    mbar_arrive(bar(Cfg::kIE + slot));
    if (flags & kStageEnd) break;
    if (flags & kStageFirst) {
      ++item;
      if (!mbar_wait_inl(bar(Cfg::kQF + item % Cfg::kItems), (item / Cfg::kItems) & 1, ctl, kSiteMmaStage))
        break;
    }
    if (!mbar_wait_inl(bar(Cfg::kKF + (t & 1)), (t >> 1) & 1, ctl, kSiteMmaStage)) break;
    // S[t % 3] was last read by PV(t - 3).
    if (t >= 3 && !mbar_wait_inl(bar(Cfg::kPVD + t % 3), ((t - 3) / 3) & 1, ctl, kSiteMmaPvDone)) break;
    tc_fence_after();
    const uint32_t s = tmem + (t % 3) * 128;
    const uint32_t q = md.q0 + (item & 1) * (Cfg::kTileB >> 4);
    const uint32_t k = md.k0 + (t & 1) * (Cfg::kTileB >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * Cfg::kHalfB + (kk & 3) * 32) >> 4;
      tc_mma_ss_lh(s, q + off, md.hi, k + off, md.hi, Cfg::kIdescS, kk > 0 ? 1u : 0u);
    }
    tc_commit(bar(Cfg::kSF + t % 3));
  }
  tc_commit(bar(Cfg::kDrain));
  mbar_drain_wait(bar(Cfg::kDrain), 0);
}

template <int D>
__device__ __forceinline__ void tile_mma_pv(uint8_t* smem, uint32_t tmem, const WaitCtl& ctl) {
  using Cfg = TileCfg<D>;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const TileDescs<D> md(sbase);
  for (int t = 0;; ++t) {
    const int slot = t % Cfg::kInfo;
    if (!mbar_wait_inl(bar(Cfg::kIF + slot), (t / Cfg::kInfo) & 1, ctl, kSiteCacheInfo)) break;
    const int flags = reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB)->flags;
    mbar_arrive(bar(Cfg::kIE + slot));
    if (flags & kStageEnd) break;
    // P(t) written (at an item's first step: the previous item's O read out before that).
    if (!mbar_wait_inl(bar(Cfg::kPF + t % 3), (t / 3) & 1, ctl, kSiteMmaPFull)) break;
    if (!mbar_wait_inl(bar(Cfg::kVF + (t & 1)), (t >> 1) & 1, ctl, kSiteMmaStage)) break;
    tc_fence_after();
    const uint32_t ps = tmem + (t % 3) * 128;
    const uint32_t v = md.v0 + (t & 1) * (Cfg::kTileB >> 4);
    const bool first = flags & kStageFirst;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)  // 16 keys each
      tc_mma_ts_lh(tmem + Cfg::kOCol, ps + kk * 8, v + ((kk * 16 * 128) >> 4), md.hi, Cfg::kIdescPV,
                   kk == 0 && first ? 0u : 1u);
    tc_commit(bar(Cfg::kPVD + t % 3));
  }
  tc_commit(bar(Cfg::kDrain + 1));
  mbar_drain_wait(bar(Cfg::kDrain + 1), 0);
}

// --------------------------------------------------------------------- converter

// 16 bytes, or zeros: a predicated load (as a branch, each of a thread's loads would wait
// for the address of the one before).
__device__ __forceinline__ uint4 load16_if(const void* ptr, bool on) {
  uint4 x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w)
      : "l"(ptr), "r"(static_cast<int>(on)));
  return x;
}

template <class A, class C, int D>
__device__ __forceinline__ void tile_convert(const CacheFwdParams& p, uint8_t* smem, const WaitCtl& ctl) {
  using Cfg = TileCfg<D>;
  constexpr int RPP = 128 * 16 / D;   // rows of a pass of the 128 threads, 16 numbers each
  constexpr int NP = 128 / RPP;       // passes of a tile
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  // Row of a pass and 16-number piece of it.  Eight neighbouring lanes have four pieces each of
  // an even and an odd row, which the swizzle puts on different banks.
  const int piece = (lane & 3) | (D == 128 ? (lane >> 1) & 4 : 0);
  const int r0 = warp * (RPP / 4) + (D == 128 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2);
  auto info = [&](int t) -> const TileStep& {
    return *reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + (t % Cfg::kInfo) * Cfg::kInfoB);
  };
  auto wait_warp = [&](int b, int parity, int site) {
    return __all_sync(0xffffffffu, mbar_wait_inl(bar(b), parity, ctl, site)) != 0;
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  uint4 kr[NP], vr[NP];
  // A step's stored numbers of one side into registers; what no query of the tile sees is
  // zero (the cache may hold anything there).
  const int64_t mine = (r0 & 15) * D + piece * 16;
  auto load = [&](const TileStep& st, const uint8_t* cache, uint4 (&x)[NP]) {
    // Rows of the two pieces of the step that some query of the tile sees.
    const int last = st.seg.pos0 + st.seg.nq - 1, lo = st.seg.lo_key;
    const int lo0 = lo - st.key0[0], hi0 = last - st.key0[0], lo1 = lo - st.key0[1], hi1 = last - st.key0[1];
    int64_t off[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) off[i] = st.off[(i * RPP + r0) >> 4];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = (i * RPP + r0) & 63;
      const bool seen = i < NP / 2 ? r >= lo0 && r <= hi0 : r >= lo1 && r <= hi1;
      x[i] = load16_if(cache + mine + off[i], off[i] >= 0 && seen);
    }
  };
  // 16 stored numbers to fp16, two 16-byte pieces of a swizzled row.
  uint8_t* const dst0 = smem + (piece >> 2) * Cfg::kHalfB + r0 * 128 + (((2 * (piece & 3)) ^ (r0 & 7)) << 4);
  uint8_t* const dst1 = smem + (piece >> 2) * Cfg::kHalfB + r0 * 128 + (((2 * (piece & 3) + 1) ^ (r0 & 7)) << 4);
  auto store = [&](int tile, const uint4 (&x)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      uint32_t h[8];
      stored4_to_half2<C>(x[i].x, h[0], h[1]);
      stored4_to_half2<C>(x[i].y, h[2], h[3]);
      stored4_to_half2<C>(x[i].z, h[4], h[5]);
      stored4_to_half2<C>(x[i].w, h[6], h[7]);
      *reinterpret_cast<uint4*>(dst0 + tile + i * RPP * 128) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(dst1 + tile + i * RPP * 128) = make_uint4(h[4], h[5], h[6], h[7]);
    }
  };

  // Iteration t stores K(t) and V(t - 1), then requests K(t + 1) and V(t).
  int item = -1;
  for (int t = -1;; ++t) {
    const int flags = t < 0 ? 0 : info(t).flags;
    const bool end = flags & kStageEnd;
    if (t >= 0 && !end) {
      // S(t - 2) read the K tile that this step overwrites, and the Q tile of the item before
      // the last one (whose last step it is at the latest).
      if (t >= 2 && !wait_warp(Cfg::kSF + (t - 2) % 3, ((t - 2) / 3) & 1, kSiteProdKEmpty)) break;
      if (flags & kStageFirst) {
        ++item;
        // Row tid of the tile: query and head, scaled into fp16's range.
        const CacheSeg& s = info(t).seg;
        const int qi = static_cast<int>((tid * p.group_inv) >> 16);
        const bool live = qi < s.nq;
        const A* q = static_cast<const A*>(p.q) + (s.q0 + qi) * p.q_token_stride +
                     (s.h * p.group + tid - qi * p.group) * p.q_head_stride;
        float up = 1.f, back = 1.f;
        if constexpr (!std::is_same<A, __half>::value) {
          float top = 0.f;
          if (live) {
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(q + 8 * c);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = act_to_float2<A>(w[i]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
          }
          const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
          const int k = max(-113, min(120, 14 - e));
          up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
          back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        }
        uint8_t* row = smem + Cfg::kOffQ + (item & 1) * Cfg::kTileB + tid * 128;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (live) {
            x = *reinterpret_cast<const uint4*>(q + 8 * c);
            if constexpr (!std::is_same<A, __half>::value) {
              uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = act_to_float2<A>(w[i]);
                w[i] = float2_to_act<__half>(f.x * up, f.y * up);
              }
              x = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          *reinterpret_cast<uint4*>(row + (c >> 3) * Cfg::kHalfB + (((c & 7) ^ (tid & 7)) << 4)) = x;
        }
        reinterpret_cast<float*>(smem + Cfg::kOffFactor)[(item % Cfg::kItems) * 128 + tid] = back;
        fence_proxy_async_smem();
        arrive(Cfg::kQF + item % Cfg::kItems);
      }
      store(Cfg::kOffK + (t & 1) * Cfg::kTileB, kr);
    }
    if (t > 0) {
      // PV(t - 3) read the V tile that V(t - 1) overwrites.
      if (t >= 3 && !wait_warp(Cfg::kPVD + (t - 3) % 3, ((t - 3) / 3) & 1, kSiteProdVEmpty)) break;
      store(Cfg::kOffV + ((t - 1) & 1) * Cfg::kTileB, vr);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && t >= 0) {
      if (!end) mbar_arrive(bar(Cfg::kKF + (t & 1)));
      if (t > 0) mbar_arrive(bar(Cfg::kVF + ((t - 1) & 1)));
    }
    if (end) break;
    const int nx = t + 1;
    if (!wait_warp(Cfg::kIF + nx % Cfg::kInfo, (nx / Cfg::kInfo) & 1, kSiteCacheInfo)) break;
    if (!(info(nx).flags & kStageEnd)) load(info(nx), p.k_cache, kr);
    if (t >= 0) {
      load(info(t), p.v_cache, vr);
      arrive(Cfg::kIE + t % Cfg::kInfo);
    }
  }
}

// ----------------------------------------------------------------------- softmax

// FOLD: positive scale and no soft-cap, so that the scores' factor goes into the exponent's
// multiplier; else they are transformed first.
template <class A, int D, bool FOLD>
__device__ __forceinline__ void tile_softmax(const CacheFwdParams& p, uint8_t* smem, uint32_t tmem,
                                             const CacheParts& parts, int* join_flag, const WaitCtl& ctl) {
  using Cfg = TileCfg<D>;
  constexpr int NC = 64;
  constexpr int R = Cfg::kRows;
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  const int w8 = (threadIdx.x >> 5) - 4, wg = w8 >> 2, wq = w8 & 3;
  const int lane = threadIdx.x & 31, half = lane >> 4;
  const int row = wq * 32 + wg * 16 + (lane & 15);
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32 + wg * 16) << 16);
  const uint32_t to = tl + Cfg::kOCol;
  const int qi = static_cast<int>((row * p.group_inv) >> 16);
  auto wait_bar = [&](int b, int parity, int site) -> bool {
    const bool w = __all_sync(0xffffffffu, mbar_wait_inl(bar(b), parity, ctl, site));
    if (w) tc_fence_after();
    return w;
  };
  auto warp_arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  ConsumerBarrierInl cb{bar(Cfg::kJoin), 0};

  CacheSeg seg{};          // of the item whose O is pending
  float m = -INFINITY, l = 0.f, rf = 1.f;
  int qpos = -1, item = -1;
  bool live = false;

  // The finished item's rows: its O (this thread's columns 64 c + 32 half + ..) scaled and
  // stored, or left as a piece of a cut unit.
  auto finish = [&](int last_step) -> bool {
    if (!wait_bar(Cfg::kPVD + last_step % 3, (last_step / 3) & 1, kSiteSoftItemDone)) return false;
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
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t r[32];
      tmem_ld_16x32bx2_x32<32>(to + c * 64, r);
      tmem_ld_wait(r);
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
    if (!cb.sync(lane, ctl)) return false;
    if (w8 == 0 && lane == 0) {
      __threadfence();
      int* count = parts.count + (blockIdx.x - seg.before);
      const bool now = atomic_add_acq_rel(count, 1) == seg.before + seg.more;
      if (now) *count = 0;
      *join_flag = now;
    }
    if (!cb.sync(lane, ctl)) return false;
    if (*reinterpret_cast<volatile int*>(join_flag)) {
#pragma unroll 1
      for (int r = w8; r < seg.nq * p.group; r += 8)
        join_row<A, D, R>(p, parts, seg, blockIdx.x - seg.before, seg.before + seg.more, r, lane);
    }
    return cb.sync(lane, ctl);
  };

  bool pending = false;
  for (int t = 0;; ++t) {
    const int slot = t % Cfg::kInfo;
    if (!wait_bar(Cfg::kIF + slot, (t / Cfg::kInfo) & 1, kSiteCacheInfo)) break;
    const TileStep& st = *reinterpret_cast<const TileStep*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
    const int flags = st.flags;
    const bool first = flags & kStageFirst;
    if (flags & (kStageFirst | kStageEnd)) {
      // The previous item's O goes out before this step's P is handed over (the product that
      // reads it overwrites O).
      if (pending && !(finish(t - 1) && join())) break;
      if (flags & kStageEnd) break;
      pending = true;
      ++item;
      if (!wait_bar(Cfg::kQF + item % Cfg::kItems, (item / Cfg::kItems) & 1, kSiteSoftSFull)) break;
      seg = st.seg;
      live = qi < seg.nq;
      qpos = live ? seg.pos0 + qi : -1;
      rf = reinterpret_cast<const float*>(smem + Cfg::kOffFactor)[(item % Cfg::kItems) * 128 + row] *
           (FOLD || p.softcap_log2 == 0.f ? p.scale_log2 : p.softcap_inv);
      m = -INFINITY;
      l = 0.f;
    }
    if (!wait_bar(Cfg::kSF + t % 3, (t / 3) & 1, kSiteSoftSFull)) break;
    float x[NC];
    const uint32_t ts = tl + (t % 3) * 128;
    {
      uint32_t a[32], b[32];
      tmem_ld_16x32bx2_x32<64>(ts, a);
      tmem_ld_16x32bx2_x32<64>(ts + 32, b);
      tmem_ld_wait(a);
      tmem_ld_wait(b);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        x[i] = __uint_as_float(a[i]);
        x[32 + i] = __uint_as_float(b[i]);
      }
    }
    const int key0 = st.key0[half];
    float c[4], a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = rf * st.ks[half * 4 + i];
      a[i] = st.lv[half * 4 + i];
    }
    if constexpr (!FOLD) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        x[i] *= c[i >> 4];
        if (p.softcap_log2 > 0.f) x[i] = softcap(x[i], p.softcap_log2);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = 1.f;
    } else {
      // A zero factor would turn a masked score into a NaN.
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = fmaxf(c[i], 1.17549435e-38f);
    }
    {
      int lo = 0, hi = min(NC - 1, qpos - key0);
      if (p.window >= 0) lo = max(lo, qpos - p.window - key0);
      if (__any_sync(0xffffffffu, lo > 0 || hi < NC - 1)) {
        // Bit i: score i is seen.
        uint64_t seen = hi < lo ? 0ull : (~0ull >> (63 - (hi - lo))) << lo;
        const uint32_t s0 = static_cast<uint32_t>(seen), s1 = static_cast<uint32_t>(seen >> 32);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = (s0 >> i) & 1 ? x[i] : -INFINITY;
          x[32 + i] = (s1 >> i) & 1 ? x[32 + i] : -INFINITY;
        }
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float t0 = fmax3(x[16 * g], x[16 * g + 1], x[16 * g + 2]);
      float t1 = fmax3(x[16 * g + 3], x[16 * g + 4], x[16 * g + 5]);
      t0 = fmax3(t0, x[16 * g + 6], x[16 * g + 7]);
      t1 = fmax3(t1, x[16 * g + 8], x[16 * g + 9]);
      t0 = fmax3(t0, x[16 * g + 10], x[16 * g + 11]);
      t1 = fmax3(t1, x[16 * g + 12], x[16 * g + 13]);
      t0 = fmax3(t0, x[16 * g + 14], x[16 * g + 15]);
      mx = fmaxf(mx, fmaf(fmaxf(t0, t1), c[g], a[g]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    float alpha = 1.f;
    const float m_new = fmaxf(m, mx);
    if (first) {
      m = m_new;
    } else if (m_new > m + 8.f) {
      alpha = ex2_approx(m - m_new);
      m = m_new;
    }
    const float neg_m = m == -INFINITY ? 0.f : -m;
    float sum = 0.f;
    {
      uint32_t pk[32];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint64_t c2 = f2_pack(c[g], c[g]), m2 = f2_pack(a[g] + neg_m, a[g] + neg_m);
        uint64_t s2 = 0ull, s3 = 0ull;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t y = f2_fma(f2_pack(x[16 * g + 2 * i], x[16 * g + 2 * i + 1]), c2, m2);
          const uint64_t e = f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y)));
          if (i & 1) s3 = f2_add(s3, e);
          else s2 = f2_add(s2, e);
          pk[8 * g + i] = float2_to_act<__half>(f2_lo(e), f2_hi(e));
        }
        s2 = f2_add(s2, s3);
        // w / vs
        sum = fmaf(f2_lo(s2) + f2_hi(s2), st.rv[half * 4 + g], sum);
      }
      tmem_st_16x32bx2_x32<32>(ts, pk);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    l = l * alpha + sum;
    if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
      // PV(t - 1) must be complete before O is rescaled.
      if (!wait_bar(Cfg::kPVD + (t - 1) % 3, ((t - 1) / 3) & 1, kSiteSoftPvDone)) break;
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        uint32_t r[32];
        tmem_ld_16x32bx2_x32<32>(to + g * 64, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
        tmem_st_16x32bx2_x32<32>(to + g * 64, r);
      }
    }
    tmem_st_wait();
    warp_arrive(Cfg::kPF + t % 3);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Cfg::kIE + slot));
  }
}

// ------------------------------------------------------------------------ kernel

template <class A, class C, int D, bool FOLD>
__global__ void __launch_bounds__(512, 1) bsa_cache_tile_kernel(const CacheFwdParams p, void* workspace) {
  using Cfg = TileCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffCtl);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);  // status, abort flag, join flag
  const WaitCtl ctl{err + 1, err, kCacheWaitNs, 0};
  const CacheParts parts = cache_parts(workspace, gridDim.x, Cfg::kRows, D);
  const CacheUnits units{p, 31 - __clz(static_cast<int>((128u * p.group_inv) >> 16)), 6, 2};
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
    }
    for (int i = 0; i < Cfg::kItems; ++i) mbar_init(bar(Cfg::kQF + i), 4);
    for (int i = 0; i < Cfg::kInfo; ++i) {
      mbar_init(bar(Cfg::kIF + i), 1);
      mbar_init(bar(Cfg::kIE + i), 4 + 8 + 2);  // converter and softmax warps, two issuers
    }
    mbar_init(bar(Cfg::kJoin), 8);
    err[0] = err[1] = err[2] = 0;
    fence_mbar_init();
    if (blockIdx.x == 0) *p.status = 0;
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  cache_split<Cfg::kThreads>(units, 4, reinterpret_cast<long long*>(smem + Cfg::kOffScan),
                             reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    setmaxnreg_dec<Cfg::kRegCtl>();
    if (warp == 0) {
      if (lane == 0) tile_mma_s<D>(smem, tmem, ctl);
    } else if (warp == 1) {
      if (lane == 0) tile_mma_pv<D>(smem, tmem, ctl);
    } else if (warp == 2) {
      tile_producer<D>(p, smem, units, ctl);
    }
  } else if (warp < 12) {
    setmaxnreg_inc<Cfg::kRegSoft>();
    tile_softmax<A, D, FOLD>(p, smem, tmem, parts, err + 2, ctl);
  } else {
    setmaxnreg_dec<Cfg::kRegConv>();
    tile_convert<A, C, D>(p, smem, ctl);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // A wait gives up long after CTA 0 has cleared the word.
  if (threadIdx.x == 0 && err[0] != 0) atomicMax(p.status, err[0]);
}

template <class A, class C, int D, bool FOLD>
cudaError_t launch_tile_as(const CacheFwdParams& p, void* workspace, int sms, cudaStream_t stream) {
  using Cfg = TileCfg<D>;
  auto* kernel = bsa_cache_tile_kernel<A, C, D, FOLD>;
  static int done[64], regs = 0;
  cudaError_t e = set_smem_once(kernel, Cfg::kLaunchSmem, done);
  if (e != cudaSuccess) return e;
  if (regs == 0) {
    // setmaxnreg.inc waits for registers that the other warpgroups gave back: the shares
    // only add up when the kernel is launched at exactly kLaunchRegs.
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs != Cfg::kLaunchRegs) return cudaErrorInvalidConfiguration;
  kernel<<<sms, Cfg::kThreads, Cfg::kLaunchSmem, stream>>>(p, workspace);
  return cudaGetLastError();
}

template <class A, class C, int D>
cudaError_t launch_tile(const CacheFwdParams& p, void* workspace, int sms, cudaStream_t stream) {
  return p.softcap_log2 == 0.f && p.scale_log2 > 0.f
             ? launch_tile_as<A, C, D, true>(p, workspace, sms, stream)
             : launch_tile_as<A, C, D, false>(p, workspace, sms, stream);
}

}  // namespace bsa
