// bsa_cache_decode.cuh -- attention over the paged 8-bit cache for few query rows: at most
// 8 * NT rows (queries of a tile times query heads of a kv head).
//
// Bound: memory.  A key costs 2 D bytes and 4 D R flops, R <= 16, so the kernel has to keep
// the loads in flight and spend few instructions a byte.
//   * Work is split evenly on the device (bsa_cache_sched.cuh).  One CTA per SM: a producer
//     warp walks its segments, looks pages and scales up and brings the keys in by TMA, a
//     second one the values, 256 keys a stage, about 190 KB ahead of the eight consumer warps;
//     joining a segment's warps thus stalls no load.
//   * A consumer warp takes two 16-key slices of a stage (two chains that overlap), with a
//     running maximum and sum of its own; the warps are joined when the segment ends.
//   * Products on mma.m16n8k16 (fp16 inputs, fp32 sums), transposed so that the keys (then
//     the head dim) fill the 16 rows and the few query rows the 8 columns: S^T = K Q^T and
//     O^T = V^T P^T.  The order of d inside S and of the columns of V is free, so both
//     fragments come from contiguous bytes: a lane's 16-byte pieces of a key row give it
//     four k-steps of K each, and its 16-byte pieces of four value rows, interleaved by byte
//     permutes, give 8 row pairs of V^T.  With the 128-byte swizzle of the boxes all of these
//     shared-memory reads are free of bank conflicts (d = 64: the values' are two-way).  The
//     tensor pipe is nearly idle here; tcgen05 would need the operands converted into shared
//     memory first, a second trip for every byte.
//   * Stored numbers are exact in fp16.  bf16 queries are scaled per row by a power of two
//     into fp16's range (exact but for numbers 2^-28 of the row's largest).  The V scale
//     is folded into the exponent, w = exp2(s + log2 vs - m), so that weights are rounded
//     to fp16 relative to the largest weight times scale, and the sum takes w / vs: both
//     sums are held in fp32, with m following the running maximum of s + log2 vs.
//   * Weights are taken relative to a reference m, set 2^7 below the running maximum and moved
//     only when a score passes that maximum by 2^8 (one vote a stage), so the usual stage needs
//     no shuffles.  They stay below 2^15, and one in 2^21 of the largest is still a normal fp16
//     number (with m at the maximum one in 2^14: behind a key that leads by 2^24 with values
//     near zero, or beside a page of 2^24 times the V scale, nothing was left of the others).
//
// Measured, 32 query and 8 kv heads, d = 128, e4m3: 64 requests of 2,048 to 8,192 tokens 111 us,
// 6.0 TB/s (0.88 of a copy; the loads alone, without the products, 0.93); 4 of 65,536 tokens 91
// us, 5.9 TB/s; one of 1,000 tokens 10.8 us, almost all of it the way of one CTA: the launch, the
// split (1.6 us), the first look-ups (0.8), a stage (1.2), the join of its warps (1) and of the
// unit's pieces (1).  Four queries of 16 requests with a window of 1,000 (d = 64, int8, pages of
// 16, soft-cap, sinks) 21 us.  Smaller stages wait for a look-up each (128 keys: 157 us where 256
// took 125, before the split weighed its units); per-lane loads instead of TMA 170.
#pragma once

#include <type_traits>

#include "bsa_cache.cuh"
#include "bsa_cache_sched.cuh"
#include "bsa_ptx.cuh"

namespace bsa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// log2 of the largest weight when a row's reference is set, and how far (in log2) scores may
// pass that maximum before it is set again: weights reach 2^(kLift + kSlack), below fp16's 65504.
constexpr float kLift = 7.f, kSlack = 8.f;

// Four stored numbers (one word) as two fp16 pairs: (0, 1) and (2, 3).
template <class C>
__device__ __forceinline__ void stored4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (C::kInt8) {
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const half2 off = __float2half2_rn(1152.f);
    const half2 x = __hsub2(*reinterpret_cast<const half2*>(&a), off);
    const half2 y = __hsub2(*reinterpret_cast<const half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// d += a (16 x 16) * b (16 x 8), fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit numbers held as mma fragments.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * log2(e) * tanh(z) of two scores.  From e^(2z) (exact limits for large |z|), which near
// zero would leave half an ulp of 1 instead of one of z: there the series of tanh up to z^9,
// 2e-8 off at 0.3.  Both are taken and one is chosen: neighbours differ.
__device__ __forceinline__ void softcap2(float& a, float& b, float cap_log2) {
  auto both = [](float x) { return f2_pack(x, x); };
  const uint64_t zero = 0x8000000080000000ull;  // -0: a sum with it changes nothing
  const uint64_t z = f2_pack(a, b), w = f2_fma(z, z, zero);
  uint64_t y = f2_fma(w, both(62.f / 2835.f), both(-17.f / 315.f));
  y = f2_fma(w, y, both(2.f / 15.f));
  y = f2_fma(w, y, both(-1.f / 3.f));
  y = f2_fma(f2_fma(w, z, zero), y, z);
  const uint64_t t = f2_fma(z, both(2.f * kLog2e), zero);
  const uint64_t d = f2_add(f2_pack(ex2_approx(f2_lo(t)), ex2_approx(f2_hi(t))), both(1.f));
  const uint64_t far = f2_fma(f2_pack(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d))), both(-2.f), both(1.f));
  a = cap_log2 * (fabsf(a) > 0.3f ? f2_lo(far) : f2_lo(y));
  b = cap_log2 * (fabsf(b) > 0.3f ? f2_hi(far) : f2_hi(y));
}

// log2 of a V scale inside the range that the exponents take (NaN and zero count as its
// lower end); exact for powers of two.
__device__ __forceinline__ float log2_scale(float s) {
  s = fminf(fmaxf(s, 0x1p-60f), 0x1p+60f);
  static_assert(kScaleLogMin == -60 && kScaleLogMax == 60, "range");
  const uint32_t u = __float_as_uint(s);
  const float e = static_cast<float>(static_cast<int>(u >> 23) - 127);
  return e + lg2_approx(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u));
}

template <int D, int NT>
struct DecodeCfg {
  static constexpr int kWarps = 8;  // consumers; the producer and the values' copier come after
  // 16 rows of d = 128 take more registers than ten warps leave each (168): the producer gets a
  // warpgroup of its own, whose registers go to the consumers.  64 requests of 8,192 tokens, 4
  // queries each: 219 us; 297 with 168 registers for each of nine warps.
  static constexpr bool kSplitRegs = NT * D == 256;
  static constexpr int kThreads = kSplitRegs ? 384 : 32 * (kWarps + 2);
  static constexpr int kRegs = 168, kRegProd = 72, kRegCons = 216;
  static_assert(128 * kRegProd + 256 * kRegCons <= 384 * kRegs, "register split");
  static constexpr int kRows = 8 * NT;
  static constexpr int kSub = 2;                      // slices of a stage per warp
  static constexpr int kSlices = kWarps * kSub;       // slices of a stage
  static constexpr int kStages = 192 * 1024 / (2 * kSlices * 16 * D);
  static constexpr int kVB = D / 8;                   // bytes of a value row per lane
  static constexpr int kSliceB = 16 * D;              // one slice of K or of V
  static constexpr int kSideB = kSlices * kSliceB;
  static constexpr int kStageB = 2 * kSideB;          // K boxes, then V boxes
  static constexpr int kJoinB = (kWarps / 2) * 32 * (D / 4) * 4;  // half the warps' O, one NT
  static constexpr int kInfoB = 64 + 16 + 16 * 16 + 16 * 8;  // DecodeStage
  static_assert(kSlices <= 16, "boxes of a DecodeStage");
  static constexpr int kOffJoin = kStages * kStageB;
  static constexpr int kOffStats = kOffJoin + kJoinB;  // (reference, sum) of each warp's rows
  static constexpr int kOffSegs = kOffStats + kWarps * kRows * 8;
  static constexpr int kOffInfo = kOffSegs + 64 * static_cast<int>(sizeof(CacheSeg));
  static constexpr int kOffBar = kOffInfo + kStages * kInfoB;  // full, empty, values to copy
  static constexpr int kOffScan = kOffBar + (3 * kStages + 1) * 8;  // and the consumers' barrier
  static constexpr int kOffWalk = kOffScan + 16 * 8;
  static constexpr int kOffCtl = kOffWalk + 96;       // status, abort flag, last piece, join's word
  static constexpr int kSmemB = kOffCtl + 16 + 1024;  // + align slack
  static_assert(sizeof(CacheSeg) <= 64 && sizeof(CacheWalk) <= 96, "slots");
  static_assert(kThreads / 32 <= 16, "scan scratch");
  static_assert(kOffInfo % 16 == 0 && kOffBar % 8 == 0 && kOffScan % 8 == 0, "alignment");
  static_assert(kSmemB <= 232448, "shared memory");
};

// A box of a stage: its first key (kNoKeys: nothing of it is seen), the scale of its
// scores and log2 of its values' scale.
struct DecodeBox {
  int key0;
  float ks, lv;
  int pad;
};
constexpr int kNoKeys = kMaxPositions;  // past every position, so that the masks cover it

enum DecodeFlags { kStageFirst = 1, kStageLast = 2, kStageEnd = 4 };

// What the producer says about a stage.
struct DecodeStage {
  CacheSeg seg;
  int seg_pad[(64 - sizeof(CacheSeg)) / 4];
  int flags, pad[3];
  DecodeBox boxes[16];
  int2 copies[16];  // page and head, first row of each box (-1: none; -2 in the first: the end)
};

// Barriers of the consumer warps.  A warp whose wait on a copy gave up leaves the loop, so
// the warps first meet with a bounded wait and settle whether the join takes place
// (ConsumerBarrier); if it does, none leaves before its end, and the hardware barrier does.
template <int kThreads>
__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
// A bounded wait; INLINE: nothing out of line, where registers are split.
template <bool INLINE>
__device__ __forceinline__ bool decode_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl, int site) {
  if constexpr (INLINE) return mbar_wait_inl(bar, parity, ctl, site);
  else return mbar_wait(bar, parity, ctl, site);
}

// A warp's arrival stays counted when its wait gives up, so a slower one may find everybody
// there after that: the wait alone does not say who goes on.  A word in shared memory, WORD bytes
// behind the barrier, does: it holds the parity of the joins so far, the first warp behind its
// wait flips it (the wait held, so all have arrived and all come here) or leaves -1, and every
// warp, whatever its own wait said, goes by the word.  None can meet a later join's flip: that
// join needs its arrival.
template <bool INLINE, int WORD>
struct ConsumerBarrier {
  uint32_t bar, phase;
  __device__ __forceinline__ bool sync(int lane, const WaitCtl& ctl) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    const bool ok = __all_sync(0xffffffffu, decode_wait<INLINE>(bar, phase, ctl, kSiteCacheJoin));
    const uint32_t was = phase;
    phase ^= 1;
    uint32_t says = 0;
    if (lane == 0) {
      const uint32_t mine = ok ? phase : 0xffffffffu;
      asm volatile("atom.relaxed.cta.shared::cta.cas.b32 %0, [%1], %2, %3;"
                   : "=r"(says)
                   : "r"(bar + WORD), "r"(was), "r"(mine)
                   : "memory");
      if (says == was) says = mine;
    }
    return __shfl_sync(0xffffffffu, says, 0) == phase;
  }
};

template <class C, int D, int NT>
__device__ __forceinline__ void decode_producer(const CacheFwdParams& p, const CUtensorMap* tm_k,
                                                uint8_t* smem, const CacheUnits& units,
                                                const WaitCtl& ctl) {
  using Cfg = DecodeCfg<D, NT>;
  constexpr int S = Cfg::kStages;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  auto empty = [&](int i) { return sbase + Cfg::kOffBar + 8 * (S + i); };
  auto go = [&](int i) { return sbase + Cfg::kOffBar + 8 * (2 * S + i); };
  CacheWalk walk = *reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk);
  const int sl = units.sl, per_stage = (16 * Cfg::kSlices) >> sl;
  const int box_b = D << sl;
  CacheSeg* ring = reinterpret_cast<CacheSeg*>(smem + Cfg::kOffSegs);  // two batches' segments

  // A box's lookups depend on one another (layout block, page, scales), each a trip to
  // memory.  They are made for 32 boxes at a time, one a lane, over as many segments as
  // those lie in, and a batch ahead of the copies: between two stages of one batch the next
  // batch gets one lookup further, and none is waited for.
  struct Batch {
    int n;            // boxes (0: the share has ended)
    int seg;          // this lane's box: place of its segment in the ring,
    int first, last;  // whether it is the segment's first, last box
    int key;          // first key (kNoKeys: nothing of it is seen)
    int pid, tile;
    float ks, vs;
  };
  CacheSeg seg;
  int pos = 0, segs = 0;  // next piece of seg; segments so far
  bool open = false;      // seg has pieces left
  auto place = [&](Batch& x) {
    x.n = 0;
    x.key = kNoKeys;
    while (x.n < 32) {
      if (!open) {
        walk.next(units, seg);  // every lane walks the same way
        if (seg.nq == 0) break;
        pos = seg.s0;
        if (lane == 0) ring[segs % 64] = seg;
        ++segs;
      }
      // A segment without a piece still takes a place: its rows are written.
      const int left = max(1, seg.s1 - pos), take = min(left, 32 - x.n), i = lane - x.n;
      if (i >= 0 && i < take) {
        x.seg = (segs - 1) % 64;
        x.first = pos + i == seg.s0;
        x.last = i == left - 1;
        if (pos + i < seg.s1)
          x.key = p.row_ptr != nullptr ? p.col_idx[seg.rp + ((pos + i) >> (p.block_shift - sl))]
                                       : (pos + i) << sl;
        x.pid = pos + i;
      }
      x.n += take;
      pos += take;
      open = take < left;
    }
    __syncwarp();
  };
  auto find_page = [&](Batch& x) {
    if (x.key == kNoKeys) return;
    const CacheSeg& s = ring[x.seg];
    if (p.row_ptr != nullptr) {
      const int sub = p.block_shift - sl;
      x.key = (x.key << p.block_shift) + ((x.pid & ((1 << sub) - 1)) << sl);
    }
    if (x.key > s.pos0 + s.nq - 1 || x.key + (1 << sl) <= s.lo_key) {
      x.key = kNoKeys;
      return;
    }
    x.pid = p.table[static_cast<int64_t>(s.b) * p.max_pages + (x.key >> p.page_shift)];
  };
  auto find_scales = [&](Batch& x) {
    if (x.key == kNoKeys) return;
    if (x.pid < 0 || x.pid >= p.n_pages) {
      x.key = kNoKeys;
      return;
    }
    x.tile = x.pid * p.Hkv + ring[x.seg].h;
    x.ks = p.k_scale[x.tile];
    x.vs = p.v_scale[x.tile];
  };

  Batch cur{}, next{};
  place(cur);
  find_page(cur);
  find_scales(cur);
  int at = 0, step = 0, issued = 0;  // boxes of cur that are copied; lookups of next made
  for (int g = 0;; ++g) {
    const int slot = g % S;
    if (at >= cur.n && cur.n > 0) {
      if (step < 1) place(next);
      if (step < 2) find_page(next);
      if (step < 3) find_scales(next);
      cur = next;
      at = step = 0;
    }
    const bool end = cur.n == 0;
    // The stage: boxes [at, at + n) of the batch, of one segment.
    const int who = __shfl_sync(0xffffffffu, cur.seg, at);
    const uint32_t same = __ballot_sync(0xffffffffu, lane < cur.n && cur.seg == who) >> at;
    const int n = end ? 0 : min(per_stage, __ffs(~same) == 0 ? 32 - at : __ffs(~same) - 1);
    const bool mine = lane >= at && lane < at + n;
    const int flags = end ? kStageEnd
                          : (__any_sync(0xffffffffu, mine && cur.first) ? kStageFirst : 0) |
                                (__any_sync(0xffffffffu, mine && cur.last) ? kStageLast : 0);
    // One answer for the warp: lanes that saw the slot freed must not go on without lanes that
    // saw the abort flag first.
    if (g >= S && !__all_sync(0xffffffffu, decode_wait<Cfg::kSplitRegs>(empty(slot), (g / S - 1) & 1, ctl,
                                                                        kSiteProdKEmpty)))
      break;
    DecodeStage& st = *reinterpret_cast<DecodeStage*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
    const bool load = mine && cur.key != kNoKeys;
    const int loads = __popc(__ballot_sync(0xffffffffu, load));
    const int row = cur.key & ((1 << p.page_shift) - 1);
    if (lane < Cfg::kSlices) st.copies[lane] = make_int2(end ? -2 : -1, 0);
    __syncwarp();
    if (load) st.copies[lane - at] = make_int2(cur.tile, row);
    __syncwarp();
    if (lane == 0) {
      mbar_arrive_expect_tx(full(slot), loads * 2 * box_b);
      mbar_arrive(go(slot));
    }
    __syncwarp();
    if (load) tma_load_3d(sbase + slot * Cfg::kStageB + (lane - at) * box_b, tm_k, full(slot), 0, row, cur.tile);
    // The scales may still be on their way: described after the copies have begun.
    if (lane < Cfg::kSlices) st.boxes[lane] = DecodeBox{kNoKeys, 0.f, 0.f, 0};
    __syncwarp();
    if (mine) st.boxes[lane - at] = DecodeBox{cur.key, cur.ks, log2_scale(cur.vs), 0};
    if (lane == 0) st.flags = flags;
    if ((flags & kStageFirst) && lane < static_cast<int>(sizeof(CacheSeg) / 4))
      reinterpret_cast<int*>(&st.seg)[lane] = reinterpret_cast<const int*>(&ring[who])[lane];
    __syncwarp();
    if (lane == 0) mbar_arrive(full(slot));
    issued = g + 1;
    if (end) break;
    at += n;
    if (step == 0) place(next);
    else if (step == 1) find_page(next);
    else if (step == 2) find_scales(next);
    step = min(step + 1, 3);
  }
  // Every copy lands before the CTA leaves (also when the consumers have given up).  One limit for
  // all: where the values' copier has given up, no stage fills any more.
  const uint64_t t0 = globaltimer_ns();
  for (int j = max(0, issued - S); j < issued; ++j) {
    const uint64_t gone = globaltimer_ns() - t0;
    mbar_drain_wait(full(j % S), (j / S) & 1, gone < kDrainLimitNs ? kDrainLimitNs - gone : 0);
  }
}

// The values' copies, beside the producer, which the issue of small boxes' copies keeps busy
// (64 requests of 2,048 to 8,192 tokens in pages of 16: 140 us, 170 with all in the producer; in
// pages of 64 no difference).  One warp.
template <int D, int NT>
__device__ __forceinline__ void decode_values(const CUtensorMap* tm_v, uint8_t* smem, int box_b,
                                              const WaitCtl& ctl) {
  using Cfg = DecodeCfg<D, NT>;
  constexpr int S = Cfg::kStages;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  for (int g = 0;; ++g) {
    const int slot = g % S;
    const uint32_t full = sbase + Cfg::kOffBar + 8 * slot;
    if (!__all_sync(0xffffffffu, decode_wait<Cfg::kSplitRegs>(full + 16 * S, (g / S) & 1, ctl, kSiteProdVEmpty)))
      break;
    const DecodeStage& st =
        *reinterpret_cast<const DecodeStage*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
    const int2 c = lane < Cfg::kSlices ? st.copies[lane] : make_int2(-1, 0);
    if (c.x >= 0)
      tma_load_3d(sbase + slot * Cfg::kStageB + Cfg::kSideB + lane * box_b, tm_v, full, 0, c.y, c.x);
    const bool end = __any_sync(0xffffffffu, c.x == -2);
    if (lane == 0) mbar_arrive(full);
    if (end) break;
  }
}

// Adds and returns what was there; the warp's earlier writes (after a __syncwarp) are seen by
// whoever sees the sum, and this thread sees the others'.
__device__ __forceinline__ int atomic_add_acq_rel(int* p, int x) {
  int r;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;"
               : "=r"(r)
               : "l"(p), "r"(x)
               : "memory");
  return r;
}

// Rows r0, r0 + step, .. (N of them, fewer at the unit's end) of a cut unit: pieces 0 .. more,
// the first at the end of CTA root's share, piece i at the start of CTA root + i's.  One warp;
// the rows' loads overlap.
template <class A, int D, int R, int N>
__device__ __forceinline__ void join_rows(const CacheFwdParams& p, const CacheParts& parts,
                                          const CacheSeg& s, int root, int more, int r0, int step,
                                          int lane) {
  constexpr int E = D / 32, U = N > 1 ? 2 : 4;
  const int rows = s.nq * p.group;
  int64_t row[N];  // of the output
  float top[N], z[N], o[N][E] = {};
  auto row_of = [&](int j) { return min(r0 + j * step, rows - 1); };
  auto slot = [&](int i, int j) {
    return static_cast<int64_t>(i == 0 ? 2 * root + 1 : 2 * (root + i)) * R + row_of(j);
  };
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int qi = static_cast<int>((row_of(j) * p.group_inv) >> 16);
    const int head = s.h * p.group + row_of(j) - qi * p.group;
    row[j] = static_cast<int64_t>(s.q0 + qi) * p.Hq + head;
    z[j] = p.sinks != nullptr ? p.sinks[head] * kLog2e : -INFINITY;
    top[j] = z[j];
  }
#pragma unroll 1
  for (int i = lane; i <= more; i += 32)
#pragma unroll
    for (int j = 0; j < N; ++j) top[j] = fmaxf(top[j], __ldcg(&parts.ml[slot(i, j)]).x);
#pragma unroll
  for (int k = 1; k < 32; k *= 2)
#pragma unroll
    for (int j = 0; j < N; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], k));
#pragma unroll
  for (int j = 0; j < N; ++j) z[j] = z[j] == -INFINITY ? 0.f : ex2_approx(z[j] - top[j]);
#pragma unroll U
  for (int i = 0; i <= more; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t at = slot(i, j);
      const float2 x = __ldcg(&parts.ml[at]);
      const float f = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top[j]);
      const float* src = parts.o + at * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
        o[j][0] += f * v.x;
        o[j][1] += f * v.y;
        o[j][2] += f * v.z;
        o[j][3] += f * v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
        o[j][0] += f * v.x;
        o[j][1] += f * v.y;
      }
      z[j] += f * x.y;
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (r0 + j * step >= rows) continue;
    const float inv = z[j] == 0.f ? 0.f : 1.f / z[j];
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<A*>(p.out) + row[j] * D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      dst[i] = float2_to_act<A>(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
    if (lane == 0) p.lse[row[j]] = z[j] == 0.f ? -INFINITY : (top[j] + log2f(z[j])) * kLn2;
  }
}

template <class A, class C, int D, int NT>
__global__ void __launch_bounds__(DecodeCfg<D, NT>::kThreads, 1)
    bsa_cache_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const CacheFwdParams p,
                            void* workspace) {
  using Cfg = DecodeCfg<D, NT>;
  constexpr int W = Cfg::kWarps, R = Cfg::kRows, S = Cfg::kStages, VB = Cfg::kVB;
  constexpr int KT = D / 64;  // 16-byte pieces of a key row per lane
  constexpr int SUB = Cfg::kSub;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;  // fragment row and column of this lane
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int i) { return sbase + Cfg::kOffBar + 8 * i; };
  auto empty = [&](int i) { return sbase + Cfg::kOffBar + 8 * (S + i); };
  int* err = reinterpret_cast<int*>(smem + Cfg::kOffCtl);
  const WaitCtl ctl{err + 1, err, kCacheWaitNs, p.expire_site};
  const CacheParts parts = cache_parts(workspace, gridDim.x, R, D);
  auto group_div = [&](int r) { return static_cast<int>((r * p.group_inv) >> 16); };

  // A unit's fixed work (joining its warps, its rows, the next unit's queries) counts like 512
  // keys: 64 requests of 2,048 to 8,192 tokens 117.4 us with 64 keys, 116 with 256, 111 with 512.
  const CacheUnits units{p, 31 - __clz(group_div(R)), p.box_shift, 512 >> p.box_shift,
                         128 >> p.box_shift};
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full(i), 3);  // copies announced, boxes described, values' copies begun
      mbar_init(empty(i), W);
      mbar_init(sbase + Cfg::kOffBar + 8 * (2 * S + i), 1);
    }
    mbar_init(sbase + Cfg::kOffBar + 8 * (3 * S), W);
    err[0] = err[1] = err[3] = 0;
    fence_mbar_init();
    if (blockIdx.x == 0 && p.status != nullptr) *p.status = 0;
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  cache_split<Cfg::kThreads>(units, reinterpret_cast<long long*>(smem + Cfg::kOffScan),
                             reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk));

  if (warp >= W) {
    if constexpr (Cfg::kSplitRegs) setmaxnreg_dec<Cfg::kRegProd>();
    if (warp == W) decode_producer<C, D, NT>(p, &tm_k, smem, units, ctl);
    else if (warp == W + 1) decode_values<D, NT>(&tm_v, smem, D << p.box_shift, ctl);
  } else {
    if constexpr (Cfg::kSplitRegs) setmaxnreg_inc<Cfg::kRegCons>();
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    uint32_t qf[NT][KT][8];  // Q fragments: row 8n + g, the columns of this lane's pieces
    float rf[NT][2];         // factor of the scores of rows 8n + 2t, 8n + 2t + 1
    int hi[NT][2];           // their positions (-1: no such row)
    auto load_q = [&](const CacheSeg& seg) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g, qi = group_div(row);
        if (row < seg.nq * p.group) {
          const A* q = static_cast<const A*>(p.q) + (seg.q0 + qi) * p.q_token_stride +
                       (seg.h * p.group + row - qi * p.group) * p.q_head_stride + t * (16 * KT);
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const uint4 a = *reinterpret_cast<const uint4*>(q + c * 16);
            const uint4 b = *reinterpret_cast<const uint4*>(q + c * 16 + 8);
            qf[n][c][0] = a.x; qf[n][c][1] = a.y; qf[n][c][2] = a.z; qf[n][c][3] = a.w;
            qf[n][c][4] = b.x; qf[n][c][5] = b.y; qf[n][c][6] = b.z; qf[n][c][7] = b.w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < KT; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) qf[n][c][i] = 0;
        }
      }
    };
    CacheSeg s{};
    // The first segment's queries are requested before its keys have landed.
    CacheWalk walk = *reinterpret_cast<CacheWalk*>(smem + Cfg::kOffWalk);
    walk.next(units, s);
    load_q(s);
    int last = 0;  // last position of the tile
    constexpr int kJoinBar = Cfg::kOffBar + 8 * (3 * S);
    ConsumerBarrier<Cfg::kSplitRegs, Cfg::kOffCtl + 12 - kJoinBar> cb{sbase + kJoinBar, 0};
    bool gone = false;
    for (int gs = 0;; ++gs) {
      const int slot = gs % S;
      // A warp whose wait gave up leaves; the abort flag ends the others' waits too.
      if (!__all_sync(0xffffffffu, decode_wait<Cfg::kSplitRegs>(full(slot), (gs / S) & 1, ctl, kSiteMmaStage)))
        break;
      const DecodeStage& st =
          *reinterpret_cast<const DecodeStage*>(smem + Cfg::kOffInfo + slot * Cfg::kInfoB);
      const int flags = st.flags;
      if (flags & kStageEnd) break;
      if (flags & kStageFirst) {
        s = st.seg;
        last = s.pos0 + s.nq - 1;
        if (gs > 0) load_q(s);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
          float back = 1.f;
          if constexpr (!std::is_same<A, __half>::value) {
            // bf16: largest magnitude of the row to [2^14, 2^15), then fp16.
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < KT; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = act_to_float2<A>(qf[n][c][i]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            const int k = max(-113, min(120, 14 - e));
            const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
            back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
            for (int c = 0; c < KT; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = act_to_float2<A>(qf[n][c][i]);
                qf[n][c][i] = float2_to_act<__half>(f.x * up, f.y * up);
              }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            rf[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + e)) *
                       (p.softcap_log2 > 0.f ? p.softcap_inv : p.scale_log2);
            hi[n][e] = r < s.nq * p.group ? s.pos0 + group_div(r) : -1;
          }
        }
      }
      // This warp's slices: warp and warp + W, so that few slices spread over the warps.
      DecodeBox sl[SUB];
      bool any = false;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const int i = warp + u * W, sub = p.box_shift - 4;
        sl[u] = st.boxes[i >> sub];
        any |= sl[u].key0 != kNoKeys;
        sl[u].key0 += (i & ((1 << sub) - 1)) << 4;  // kNoKeys stays past every position
      }
      if (any) {
        const uint8_t* kbox = smem + slot * Cfg::kStageB;
        const uint8_t* vbox = kbox + Cfg::kSideB;
        // S^T: keys g and g + 8 (rows) by query rows 2t, 2t + 1 (columns).
        float x[SUB][NT][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) x[u][n][0] = x[u][n][1] = x[u][n][2] = x[u][n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KT; ++c) {
          uint32_t wa[SUB][4], wb[SUB][4];
          const int piece = D == 128 ? ((2 * t + c) ^ g) : (t ^ (g >> 1));
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            const uint8_t* src = kbox + (warp + u * W) * Cfg::kSliceB + g * D + piece * 16;
            const uint4 a = *reinterpret_cast<const uint4*>(src);
            const uint4 b = *reinterpret_cast<const uint4*>(src + 8 * D);
            wa[u][0] = a.x; wa[u][1] = a.y; wa[u][2] = a.z; wa[u][3] = a.w;
            wb[u][0] = b.x; wb[u][1] = b.y; wb[u][2] = b.z; wb[u][3] = b.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
              uint32_t a0, a1, a2, a3;
              stored4_to_half2<C>(wa[u][i], a0, a2);
              stored4_to_half2<C>(wb[u][i], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816(x[u][n], a0, a1, a2, a3, qf[n][c][2 * i], qf[n][c][2 * i + 1]);
            }
        }
        bool grow = false, whole[SUB];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][n][e] *= rf[n][e & 1] * sl[u].ks;
        if (p.softcap_log2 > 0.f)
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; e += 2) softcap2(x[u][n][e], x[u][n][e + 1], p.softcap_log2);
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          whole[u] = sl[u].key0 + 15 <= s.pos0 && (p.window < 0 || sl[u].key0 >= last - p.window);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float y = x[u][n][e] + sl[u].lv;
              if (!whole[u]) {
                const int key = sl[u].key0 + g + (e >> 1) * 8, top = hi[n][e & 1];
                if (key > top || (p.window >= 0 && key < top - p.window)) y = -INFINITY;
              }
              x[u][n][e] = y;
              grow |= y > m[n][e & 1] + (kLift + kSlack);
            }
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(x[0][n][e], x[0][n][e + 2]);
#pragma unroll
              for (int u = 1; u < SUB; ++u) top = fmaxf(top, fmaxf(x[u][n][e], x[u][n][e + 2]));
#pragma unroll
              for (int k = 4; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
              top = fmaxf(top - kLift, m[n][e]);
              const float f = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - top);
              m[n][e] = top;
              l[n][e] *= f;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[n][j][e] *= f;
                o[n][j][e + 2] *= f;
              }
            }
        }
        uint32_t pf[SUB][NT][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const float rv = ex2_approx(-sl[u].lv);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float top = m[n][e & 1];
              x[u][n][e] = ex2_approx(x[u][n][e] - (top == -INFINITY ? 0.f : top));
            }
            l[n][0] = fmaf(x[u][n][0] + x[u][n][2], rv, l[n][0]);
            l[n][1] = fmaf(x[u][n][1] + x[u][n][3], rv, l[n][1]);
            pf[u][n][0] = transpose8x8(float2_to_act<__half>(x[u][n][0], x[u][n][1]));
            pf[u][n][1] = transpose8x8(float2_to_act<__half>(x[u][n][2], x[u][n][3]));
          }
        }
        // O^T: columns VB * g + 2j, 2j + 1 of the values (rows) by the query rows.
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          uint32_t vw[4][VB / 4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * t + (i & 1) + (i >> 1) * 8;
            const uint8_t* src = vbox + (warp + u * W) * Cfg::kSliceB + r * D;
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(src + (g ^ (2 * t + (i & 1))) * 16);
              vw[i][0] = w.x; vw[i][1] = w.y; vw[i][2] = w.z; vw[i][3] = w.w;
            } else {
              const uint2 w =
                  *reinterpret_cast<const uint2*>(src + ((g >> 1) ^ t) * 16 + (g & 1) * 8);
              vw[i][0] = w.x; vw[i][1] = w.y;
            }
          }
          if (!whole[u]) {
            // Values that no row sees may be anything, a NaN among it: zero.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = sl[u].key0 + 2 * t + (i >> 1) * 8 + (i & 1);
              if (key > last || key < s.lo_key)
#pragma unroll
                for (int w = 0; w < VB / 4; ++w) vw[i][w] = 0;
            }
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
            const uint32_t w01 = __byte_perm(vw[0][j / 2], vw[1][j / 2], sel);
            const uint32_t w23 = __byte_perm(vw[2][j / 2], vw[3][j / 2], sel);
            uint32_t a0, a1, a2, a3;
            stored4_to_half2<C>(w01, a0, a1);
            stored4_to_half2<C>(w23, a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[n][j], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
      if (!(flags & kStageLast)) continue;

      // ---- join the warps: halves onto halves, each warp's accumulator scaled to the common
      // maximum by its reader (pass 1: the row statistics come with it).  Slot i of the
      // buffer is read by warp i in pass 1, so warp i may write it again after that.
      float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffStats);
      float4* join = reinterpret_cast<float4*>(smem + Cfg::kOffJoin);
      auto give = [&](int n, int slot) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          join[(slot * (D / 16) + j) * 32 + lane] =
              make_float4(o[n][j][0], o[n][j][1], o[n][j][2], o[n][j][3]);
      };
      auto take = [&](int n, int slot, float f0, float f1) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float4 x = join[(slot * (D / 16) + j) * 32 + lane];
          o[n][j][0] = fmaf(x.x, f0, o[n][j][0]);
          o[n][j][1] = fmaf(x.y, f1, o[n][j][1]);
          o[n][j][2] = fmaf(x.z, f0, o[n][j][2]);
          o[n][j][3] = fmaf(x.w, f1, o[n][j][3]);
        }
      };
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 4; k < 32; k *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
          if (g == 0) ml[warp * R + 8 * n + 2 * t + e] = make_float2(m[n][e], l[n][e]);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n > 0) consumer_sync<32 * W>();  // the buffer of the columns before
        if (warp >= W / 2) give(n, warp - W / 2);
        if (n > 0) {
          consumer_sync<32 * W>();
        } else if (!cb.sync(lane, ctl)) {
          gone = true;
          break;
        }
        if (warp < W / 2) {
          float f[2], fo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * R + r].x);
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const float2 x = ml[w * R + r];
              sum += x.y * (x.x == -INFINITY ? 0.f : ex2_approx(x.x - top));  // a NaN stays
            }
            const float mo = ml[(warp + W / 2) * R + r].x;
            f[e] = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - top);
            fo[e] = mo == -INFINITY ? 0.f : ex2_approx(mo - top);
            m[n][e] = top;
            l[n][e] = sum;
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[n][j][0] *= f[0];
            o[n][j][1] *= f[1];
            o[n][j][2] *= f[0];
            o[n][j][3] *= f[1];
          }
          take(n, warp, fo[0], fo[1]);
        }
#pragma unroll
        for (int half = W / 4; half >= 1; half /= 2) {
          if (warp >= half && warp < 2 * half) give(n, warp);
          consumer_sync<32 * W>();
          if (warp < half) take(n, warp + half, 1.f, 1.f);
        }
      }
      if (gone) break;
      // ---- warp 0 has the segment's sums: final rows, or a partial result of a cut unit
      const bool whole_unit = s.starts && s.ends;
      if (warp == 0) {
        const int piece = 2 * blockIdx.x + (s.starts ? 1 : 0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            if (r >= s.nq * p.group) continue;
            if (whole_unit) {
              const int qi = group_div(r), head = s.h * p.group + r - qi * p.group;
              const int64_t row = static_cast<int64_t>(s.q0 + qi) * p.Hq + head;
              float top = m[n][e], z = l[n][e], f = 1.f;
              if (p.sinks != nullptr) {
                const float sink = p.sinks[head] * kLog2e;
                const float mx = fmaxf(top, sink);
                f = top == -INFINITY ? 0.f : ex2_approx(top - mx);
                z = z * f + (sink == -INFINITY ? 0.f : ex2_approx(sink - mx));
                top = mx;
              }
              const float inv = z == 0.f ? 0.f : f / z;
              uint32_t w[D / 16];
#pragma unroll
              for (int j = 0; j < D / 16; ++j)
                w[j] = float2_to_act<A>(o[n][j][e] * inv, o[n][j][e + 2] * inv);
              uint4* dst = reinterpret_cast<uint4*>(static_cast<A*>(p.out) + row * D + g * VB);
#pragma unroll
              for (int i = 0; i < D / 64; ++i)
                dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              if (g == 0) p.lse[row] = z == 0.f ? -INFINITY : (top + log2f(z)) * kLn2;
            } else {
              float4* dst = reinterpret_cast<float4*>(
                  parts.o + (static_cast<int64_t>(piece) * R + r) * D + g * VB);
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                dst[i] = make_float4(o[n][2 * i][e], o[n][2 * i][e + 2], o[n][2 * i + 1][e],
                                     o[n][2 * i + 1][e + 2]);
              if (g == 0)
                parts.ml[static_cast<int64_t>(piece) * R + r] = make_float2(m[n][e], l[n][e]);
            }
          }
        if (!whole_unit) {
          // The CTA that leaves a unit's last piece joins them (in their order, whoever it is).
          __syncwarp();
          if (lane == 0) {
            int* count = parts.count + (blockIdx.x - s.before);
            const int pieces = s.before + 1 + s.more;
            const bool join_now = atomic_add_acq_rel(count, 1) == pieces - 1;
            if (join_now) *count = 0;  // as the next call wants it
            err[2] = join_now;
          }
        }
      }
      consumer_sync<32 * W>();  // the join buffer is free again
      if (!whole_unit) {
        if (err[2]) {
          // At most two rows a warp.
          if (warp < s.nq * p.group)
            join_rows<A, D, R, R / W>(p, parts, s, blockIdx.x - s.before, s.before + s.more, warp, W, lane);
        }
        consumer_sync<32 * W>();  // err[2] has been read
      }
    }
  }
  __syncthreads();
  // A wait gives up long after CTA 0 has cleared the word.
  if (tid == 0 && err[0] != 0) atomicMax(p.status != nullptr ? p.status : parts.status, err[0]);
}

template <class A, class C, int D, int NT>
cudaError_t launch_decode(const CUtensorMap& k, const CUtensorMap& v, const CacheFwdParams& p,
                          void* workspace, int sms, cudaStream_t stream) {
  using Cfg = DecodeCfg<D, NT>;
  auto* kernel = bsa_cache_decode_kernel<A, C, D, NT>;
  static int done[64];
  const cudaError_t e = set_smem_once(kernel, Cfg::kSmemB, done);
  if (e != cudaSuccess) return e;
  kernel<<<sms, Cfg::kThreads, Cfg::kSmemB, stream>>>(k, v, p, workspace);
  return cudaGetLastError();
}

template <class C, int D>
cudaError_t launch_decode(bool fp16, int rows, const CUtensorMap& k, const CUtensorMap& v,
                          const CacheFwdParams& p, void* workspace, int sms, cudaStream_t stream) {
  if (fp16)
    return rows <= 8 ? launch_decode<__half, C, D, 1>(k, v, p, workspace, sms, stream)
                     : launch_decode<__half, C, D, 2>(k, v, p, workspace, sms, stream);
  return rows <= 8 ? launch_decode<__nv_bfloat16, C, D, 1>(k, v, p, workspace, sms, stream)
                   : launch_decode<__nv_bfloat16, C, D, 2>(k, v, p, workspace, sms, stream);
}

}  // namespace bsa
