// bsa_diff_fwd_kernel.cuh -- forward of block-sparse differential attention for sm_103a:
//     out = (P_0 - lam P_1) V,   P_m = softmax over the active keys of scale q_m . k
//
// A work item is 64 queries of one head, both maps as 128 rows (bsa_diff.cuh): row 32 w + 16 m
// + r is query 16 w + r under map m, so that the two rows of a query sit 16 lanes apart in one
// warp's TMEM lanes.  Everything up to the epilogue is the plain forward's pipeline at 128 query
// rows (bsa_fwd_kernel.cuh: roles, barriers, S buffers, register split): warp 0 loads keys and
// values, warp 3 queries, warp 1 issues S = Q K^T, warp 2 O += P V, softmax warps 4-7 hold the
// rows of map 0 and 8-11 those of map 1 (each with its own running maximum and sum), and the
// epilogue warps read O out, half the columns of both of a query's rows a lane, divide them by
// their sums and store O_0 - lam O_1 (and, for a training step, O_1, which the backward needs).
//
// P is rounded to bf16 for its product, as in the plain forward; maxima, sums, O and the
// difference of the maps are fp32, and out is rounded once.
//
// Bound: as the plain forward the softmax warps' chain of TMEM loads, maxima and exponentials;
// a step of 128 keys is 128 x 128 scores whichever map they belong to.
// Measured: 16 heads of 128 on 4 kv heads, 16,384 tokens, block 128, a band and a stride: 255 us,
// 1,400 TFLOP/s (0.74 of a cuBLAS bf16 product; the plain forward on 32 such heads takes 255 too);
// 8,192 tokens 109 us; 2 x 8 heads of 64, 2,999 tokens, block 64, a window and a global block: 21
// us; 4 heads of 64, 512 tokens: 6.8 us, an item's way.  The tensor pipe works 59 % of the time,
// the exponentials' unit 30 %.
// What counted: both maps in one tile rather than two passes over the keys; queries by a warp of
// their own, an item ahead (306 us with the keys' warp); O released before the output's stores,
// which are spaced out (316); masks tested once a warp (286); items dealt forwards and backwards
// in turn (3 % against dealing forwards).  And the size of the code: the roles' loops together
// passed the instruction cache, and the SMs of a GPC share the one behind it, which was busy 75 %
// of the time.  An epilogue whose lanes read both rows of a query instead of exchanging columns,
// in packed arithmetic, list places by products instead of divisions, the queries' copies in a
// loop and waits of one loop made 59 KB of 82, and 255 us of 282.
#pragma once

#include "bsa_diff.cuh"

namespace bsa {

// The plain forward's layout of shared memory and barriers, with barriers of their own for Q.
template <int KB, int D>
struct DiffFwdCfg : FwdCfg<128, KB, D> {
  using Base = FwdCfg<128, KB, D>;
  static constexpr int kBarQF = Base::kNumBars;       // [2] Q of an item landed
  static constexpr int kBarQE = Base::kNumBars + 2;   // [2] the item's last S complete
  static constexpr int kNumBars = Base::kNumBars + 4;
  static constexpr int kBarBytes = 256;
  static_assert(kNumBars * 8 + 8 <= kBarBytes, "barrier area");
  static constexpr int kOffStats = Base::kOffBar + kBarBytes;
  static constexpr int kSmemBytes = kOffStats + 128 * 8 + 1024;  // + align slack
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kLaunchSmem = kSmemBytes > 120 * 1024 ? kSmemBytes : 120 * 1024;
};

// ---------------------------------------------------------------- producers

// Queries, by a warp of their own: an item's are eight or sixteen copies, which would hold up the
// keys', and go out as soon as the item before the last has had its last product.
template <int KB, int D, bool SPLIT>
__device__ __forceinline__ void diff_query_producer(const DiffFwdParams& p, const CUtensorMap* tm_q,
                                                    uint32_t sbase, const WaitCtl& ctl) {
  using C = DiffFwdCfg<KB, D>;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  int n = 0;  // items armed
  ItemStream is;
  for (is.init<true>(p); !is.done(); is.next<true>(p), ++n) {
    if (n >= 2 && !mbar_wait_inl(bar(C::kBarQE + (n & 1)), ((n - 2) / 2) & 1, ctl, kSiteProdKEmpty)) break;
    const uint32_t fb = bar(C::kBarQF + (n & 1)), qd = sbase + C::kOffQ + (n & 1) * C::kQTile;
    mbar_arrive_expect_tx(fb, SPLIT ? C::kQTile / 2 : C::kQTile);
#pragma unroll 1
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int z = 0; z < (SPLIT ? 1 : D / 64); ++z)
          tma_load_4d(qd + (SPLIT ? m : z) * C::kQRegion + (32 * w + 16 * m) * 128, tm_q, fb, 0,
                      is.cur.y * 64 + 16 * w, z, 2 * is.cur.x + m);
  }
  for (int j = (n > 2 ? n - 2 : 0); j < n; ++j) mbar_drain_wait(bar(C::kBarQF + (j & 1)), (j / 2) & 1);
}

template <int KB, int D>
__device__ __forceinline__ void diff_producer(const DiffFwdParams& p, const CUtensorMap* tm_k,
                                              const CUtensorMap* tm_v, uint32_t sbase, const WaitCtl& ctl) {
  using C = DiffFwdCfg<KB, D>;
  constexpr int G = C::kG;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  struct StepKeys {
    int col[G];
    int head, nblk;
  };
  StepCursor<G> c;
  c.init(p);
  int colv[G];  // column blocks of the cursor's step, loaded one step ahead
  auto fetch_cols = [&]() {
    if (!c.valid()) return;
    const int nb = c.nblk();
    const int* cols = p.col_idx + c.is.cur.z + c.s * G;
#pragma unroll
    for (int g = 0; g < G; ++g) colv[g] = (g < nb) ? cols[g] : 0;
  };
  fetch_cols();

  StepKeys h1{}, h2{};  // steps t-1, t-2
  h1.nblk = h2.nblk = 0;
  int nsteps = -1;  // known once the cursor runs out
  int nk = 0, nv = 0;  // K and V loads armed
  for (int t = 0;; ++t) {
    StepKeys r0{};
    r0.nblk = 0;
    if (c.valid()) {
      r0.nblk = c.nblk();
      r0.head = diff_over(c.is.cur.x, p.pairs_mul, p.pairs_shift);
#pragma unroll
      for (int g = 0; g < G; ++g) r0.col[g] = colv[g];
      c.advance(p);
      fetch_cols();  // the next step's columns, consumed one iteration later
    } else {
      if (nsteps < 0) nsteps = t;
      if (nsteps == 0 || t >= nsteps + 2) break;
    }
    if (r0.nblk > 0) {
      // K slot t % 3 held K(t-3), read by S(t-3).
      static_assert(C::kNQ == 2 && C::kNK == 3, "slot reuse is tied to the S buffers");
      if (t >= 3 && !mbar_wait_inl(bar(C::kBarSF + t % 3), ((t - 3) / 3) & 1, ctl, kSiteProdKEmpty)) break;
      const uint32_t fb = bar(C::kBarKF + t % 3);
      mbar_arrive_expect_tx(fb, r0.nblk * C::kBlkB);
      ++nk;
      const uint32_t kdst = sbase + C::kOffK + (t % 3) * C::kKVTile;
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (g < r0.nblk) tma_load_4d(kdst + g * C::kBlkB, tm_k, fb, 0, r0.col[g] * KB, 0, r0.head);
    }
    const StepKeys rv = h2;
    if (rv.nblk > 0) {
      const int g = t - 2;
      const int gv = g - C::kNV;
      if (gv >= 0 && !mbar_wait_inl(bar(C::kBarPVD + gv % 3), (gv / 3) & 1, ctl, kSiteProdVEmpty))
        break;
      const uint32_t fb = bar(C::kBarVF + g % 3);
      mbar_arrive_expect_tx(fb, rv.nblk * C::kBlkB);
      ++nv;
      const uint32_t vdst = sbase + C::kOffV + (g % C::kNV) * C::kKVTile;
#pragma unroll
      for (int b = 0; b < G; ++b)
        if (b < rv.nblk) tma_load_4d(vdst + b * C::kBlkB, tm_v, fb, 0, rv.col[b] * KB, 0, rv.head);
    }
    h2 = h1;
    h1 = r0;
  }
  // Wait until every copy this thread issued has landed (immediate on the normal path).
  for (int j = (nk > 3 ? nk - 3 : 0); j < nk; ++j)
    mbar_drain_wait(bar(C::kBarKF + j % 3), (j / 3) & 1);
  for (int j = (nv > 3 ? nv - 3 : 0); j < nv; ++j)
    mbar_drain_wait(bar(C::kBarVF + j % 3), (j / 3) & 1);
}

// -------------------------------------------------------------- S issuer

// S(t) = Q K(t)^T into S[t % 3], as in the plain forward.
template <int KB, int D>
__device__ __forceinline__ void diff_mma_s(const DiffFwdParams& p, uint32_t sbase, uint32_t tmem,
                                           const WaitCtl& ctl) {
  using C = DiffFwdCfg<KB, D>;
  constexpr int G = C::kG;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const MmaDescs<128, KB, D> md(sbase);
  StepCursor<G> c;
  c.init(p);
  for (int t = 0; c.valid(); ++t) {
    const int nblk = c.nblk(), n = c.is.n;
    const bool first = c.s == 0, last = c.s == c.nsteps - 1;
    c.advance(p);
    if (first && !mbar_wait_inl(bar(C::kBarQF + (n & 1)), (n / 2) & 1, ctl, kSiteMmaStage)) break;
    if (!mbar_wait_inl(bar(C::kBarKF + t % 3), (t / 3) & 1, ctl, kSiteMmaStage)) break;
    // S[t % 3] was last read by PV(t-3).
    if (t >= 3 && !mbar_wait_inl(bar(C::kBarPVD + t % 3), ((t - 3) / 3) & 1, ctl, kSiteMmaPvDone)) break;
    tc_fence_after();
    const uint32_t sb = tmem + (t % 3) * 128;
    const uint32_t qlo = md.q0 + (n & 1) * (C::kQTile >> 4);
    const uint32_t klo = md.k0 + (t % 3) * (C::kKVTile >> 4);
    auto s_mmas = [&](int nb) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t qa = qlo + (((kk >> 2) * C::kQRegion + (kk & 3) * 32) >> 4);
        const uint32_t kb = klo + (((kk >> 2) * C::kHalfB + (kk & 3) * 32) >> 4);
        if (KB == 128) {
          tc_mma_ss_lh(sb, qa, md.hi, kb, md.hi, C::kIdescS, kk > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int g = 0; g < nb; ++g)
            tc_mma_ss_lh(sb + g * KB, qa, md.hi, kb + ((g * C::kBlkB) >> 4), md.hi, C::kIdescS1,
                         kk > 0 ? 1u : 0u);
        }
      }
    };
    if (KB == 64 && nblk > 1)  // a branch between two MMAs slows their issue
      s_mmas(2);
    else
      s_mmas(1);
    tc_commit(bar(C::kBarSF + t % 3));
    if (last) tc_commit(bar(C::kBarQE + (n & 1)));
  }
  tc_commit(bar(C::kBarDrainS));
  mbar_drain_wait(bar(C::kBarDrainS), 0);
}

// ------------------------------------------------------------------ softmax

template <int KB, int D>
__device__ __forceinline__ void diff_softmax(const DiffFwdParams& p, uint32_t sbase, uint8_t* smem,
                                             uint32_t tmem, const WaitCtl& ctl) {
  using C = DiffFwdCfg<KB, D>;
  constexpr int G = C::kG;
  constexpr int NC = 64;  // score columns per thread
  constexpr int NA = 8;   // independent max chains
  constexpr int NS = 4;   // packed sum accumulators
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const int map = ((threadIdx.x >> 5) - C::kSoftWarp) >> 2;
  const int wq = (threadIdx.x >> 5) & 3;  // TMEM lane quadrant of this warp
  const int lane = threadIdx.x & 31;
  const int half = lane >> 4;
  const int row = wq * 32 + map * 16 + (lane & 15);  // of the tile
  const int qin = wq * 16 + (lane & 15);             // query of the tile
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32 + map * 16) << 16);
  const uint32_t to = tl + C::kOCol;
  const int kbase = (KB == 128) ? 64 * half : 0;  // first key of this half in its block
  float2* stats = reinterpret_cast<float2*>(smem + C::kOffStats);
  // scale > 0: the row max of the raw scores gives the max of the scaled ones and the exponent
  // is one FFMA; otherwise the scores are scaled first.
  const bool pos_scale = p.scale_log2 > 0.f;
  const float cs = pos_scale ? p.scale_log2 : 1.f;
  const bool ragged = p.L % KB != 0;
  int g = 0;
  bool ok = true;
  bool s_next = false;  // S(g+1) already complete, as seen by a probe issued during step g

  auto warp_arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  auto wait_bar = [&](int b, int parity, int site) -> bool {
    bool w = mbar_wait_inl(bar(b), parity, ctl, site);
    w = __all_sync(0xffffffffu, w);
    if (w) tc_fence_after();
    return w;
  };

  ItemStream is;
  for (is.init<true>(p); ok && !is.done(); is.next<true>(p)) {
    const int nnz = is.nnz();
    const int dpos = p.causal_diag ? is.dpos() : -1;  // position of the diagonal block in the row
    // Position of a block that the end of the sequence cuts: only the last one can be.
    const int cut = ragged && p.col_idx[is.cur.z + nnz - 1] == p.L / KB ? nnz - 1 : -1;
    // The query's place in its layout block: block 128 has two tiles.
    const int qblk = qin + (KB == 128 ? (is.cur.y & 1) * 64 : 0);
    const int nsteps = (nnz + G - 1) / G;
    float m_used = -INFINITY;
    float l = 0.f;
    for (int s = 0; s < nsteps; ++s, ++g) {
      const int nblk = step_blocks<G>(nnz, s);
      const bool valid = (KB == 128) || (half < nblk);
      const int blk = (KB == 128) ? s : s * 2 + half;  // the half's place in the row
      const uint32_t ts = tl + (g % 3) * 128;
      if (__all_sync(0xffffffffu, s_next)) {
        tc_fence_after();
      } else {
        ok = wait_bar(C::kBarSF + g % 3, (g / 3) & 1, kSiteSoftSFull);
        if (!ok) break;
      }
      float x[NC];
      {
        uint32_t r0[32], r1[32];
        tmem_ld_16x32bx2_x32<64>(ts + 0, r0);
        tmem_ld_16x32bx2_x32<64>(ts + 32, r1);
        tmem_ld_wait(r0);
        tmem_ld_wait(r1);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = __uint_as_float(r0[i]);
          x[32 + i] = __uint_as_float(r1[i]);
        }
      }
      if (!pos_scale) {
#pragma unroll
        for (int c = 0; c < NC; ++c) x[c] *= p.scale_log2;
      }
      if (!valid || blk == dpos || blk == cut) {  // KB = 128: the same for the whole warp
        // Last key of this half's 64 that the row sees: before the diagonal's and the sequence's end.
        int lim = valid ? NC - 1 : -1;
        if (blk == dpos) lim = min(lim, qblk - kbase);
        if (blk == cut) lim = min(lim, (p.L - 1) % KB - kbase);
#pragma unroll
        for (int c = 0; c < NC; ++c) x[c] = mask_gt(x[c], c, lim);
      }
      // Row max: NA chains of three-input maxima, then the other half of the row (lane ^ 16).
      float mr[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        mr[a] = x[a];
#pragma unroll
        for (int c = a + NA; c < NC; c += 2 * NA)
          mr[a] = (c + NA < NC) ? fmax3(mr[a], x[c], x[c + NA]) : fmaxf(mr[a], x[c]);
      }
#pragma unroll
      for (int w = NA / 2; w >= 1; w /= 2)
#pragma unroll
        for (int a = 0; a < w; ++a) mr[a] = fmaxf(mr[a], mr[a + w]);
      float mx = mr[0] * cs;  // -inf stays -inf (cs > 0)
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      float alpha = 1.f;
      const float m_new = fmaxf(m_used, mx);
      if (s == 0) {
        m_used = m_new;
      } else if (m_new > m_used + 8.f) {
        alpha = ex2_approx(m_used - m_new);
        m_used = m_new;
      }
      const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;

      // exp2(x*c - m) on pairs; packed row sums; P (bf16 pairs) over the S columns just read.
      uint64_t sr2[NS];
#pragma unroll
      for (int a = 0; a < NS; ++a) sr2[a] = 0ull;
      const uint64_t c2 = f2_pack(cs, cs), m2 = f2_pack(neg_m, neg_m);
      {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint64_t y = f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), c2, m2);
          const uint64_t e = f2_pack(ex2_approx(f2_lo(y)), ex2_approx(f2_hi(y)));
          sr2[i % NS] = f2_add(sr2[i % NS], e);
          pk[i] = pack_bf16x2(f2_lo(e), f2_hi(e));
        }
        tmem_st_16x32bx2_x32<32>(ts, pk);
      }
      // S(g+4) needs this step's P, so the barrier of S(g+1) cannot be a phase ahead.
      s_next = mbar_test_wait(bar(C::kBarSF + (g + 1) % 3), ((g + 1) / 3) & 1);
      sr2[0] = f2_add(f2_add(sr2[0], sr2[1]), f2_add(sr2[2], sr2[3]));
      float rs = f2_lo(sr2[0]) + f2_hi(sr2[0]);
      rs += __shfl_xor_sync(0xffffffffu, rs, 16);
      l = l * alpha + rs;

      // O rescale (rare): PV(g-1) must be complete first.
      if (s > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        ok = wait_bar(C::kBarPVD + (g - 1) % 3, ((g - 1) / 3) & 1, kSiteSoftPvDone);
        if (!ok) break;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r[32];
          load_o32(to, c, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
          store_o32(to, c, r);
        }
      }
      tmem_st_wait();
      warp_arrive(C::kBarPF + g % 3);
    }
    if (!ok) break;
    // Row statistics to the epilogue, once it has read the previous item's.
    if (is.n > 0) {
      ok = wait_bar(C::kBarStFree, (is.n - 1) & 1, kSiteSoftStatsFree);
      if (!ok) break;
    }
    if (half == 0) stats[row] = make_float2(m_used, l);
    __threadfence_block();
    warp_arrive(C::kBarStFull);
  }
  tmem_st_wait();  // a loop left early leaves no store under way when TMEM is freed
}

// ----------------------------------------------------------------- epilogue

template <int KB, int D>
__device__ __forceinline__ void diff_epilogue(const DiffFwdParams& p, uint32_t sbase,
                                              const uint8_t* smem, uint32_t tmem,
                                              const WaitCtl& ctl) {
  using C = DiffFwdCfg<KB, D>;
  constexpr int G = C::kG;
  constexpr int HC = D / 2;  // output columns of each of a query's two lanes, 16 apart
  constexpr float kLn2 = 0.6931471805599453f;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const int wq = (threadIdx.x >> 5) & 3;
  const int lane = threadIdx.x & 31;
  const int half = lane >> 4;  // of the query's columns; and the map whose lse this lane stores
  const int qin = wq * 16 + (lane & 15);
  const uint32_t to = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::kOCol;
  const float2* stats = reinterpret_cast<const float2*>(smem + C::kOffStats);
  const bool v8 = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.out2)) & 31) == 0;
  auto wait_bar = [&](int b, int parity, int site) -> bool {
    bool w = mbar_wait_inl(bar(b), parity, ctl, site);
    w = __all_sync(0xffffffffu, w);
    if (w) tc_fence_after();
    return w;
  };
  auto warp_arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  // 32 columns as bf16: whole sectors where the bases allow it.
  auto store32 = [&](__nv_bfloat16* dst, const uint32_t (&w)[16], unsigned gap) {
    if (v8) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        __nanosleep(gap);  // a burst of stores stalls the softmax warps
        st_global_v8(dst + 16 * q, w[8 * q], w[8 * q + 1], w[8 * q + 2], w[8 * q + 3], w[8 * q + 4],
                     w[8 * q + 5], w[8 * q + 6], w[8 * q + 7]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        reinterpret_cast<uint4*>(dst)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  };

  int g = 0;  // first step of the current item
  ItemStream is;
  for (is.init<false>(p); !is.done(); is.next<false>(p)) {
    const int nnz = is.nnz();
    const int q = is.cur.y * 64 + qin;
    const bool live = q < p.L;
    const int64_t pair = is.cur.x;
    const int64_t orow = (pair * p.L + q) * D + half * HC;  // this lane's first output number
    float* lse = p.lse + (2 * pair + half) * p.L + q;
    if (nnz == 0) {
      if (live) {
#pragma unroll 1
        for (int c = 0; c < HC; c += 8) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow + c) = zero;
          if (p.out2 != nullptr) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out2) + orow + c) = zero;
        }
        *lse = -INFINITY;
      }
      continue;
    }
    float lam = 0.f;
    if (live) lam = p.lam_rows ? p.lam[pair * p.L + q] : p.lam[static_cast<unsigned>(is.cur.x) % p.H];
    const int gl = g + (nnz + G - 1) / G - 1;  // the item's last step
    g = gl + 1;
    if (!wait_bar(C::kBarStFull, is.n & 1, kSiteEpiStats)) break;
    const float2 ml0 = stats[wq * 32 + (lane & 15)], ml1 = stats[wq * 32 + 16 + (lane & 15)];
    const float2 ml = half ? ml1 : ml0;
    warp_arrive(C::kBarStFree);
    if (!wait_bar(C::kBarPVD + gl % 3, (gl / 3) & 1, kSiteSoftItemDone)) break;
    auto twice = [](float x) { return f2_pack(x, x); };
    const uint64_t inv0 = twice((ml0.y > 0.f) ? 1.f / ml0.y : 0.f), weight = twice(-lam);
    const uint64_t inv1 = twice((ml1.y > 0.f) ? 1.f / ml1.y : 0.f);
    uint32_t w[HC / 32][16], w2[HC / 32][16];
#pragma unroll
    for (int c = 0; c < HC / 32; ++c) {
      uint32_t r0[32], r1[32];  // this lane's columns of its query's two rows
      tmem_ld_16x32bx2_x32<HC>(to + 32 * c, r0);
      tmem_ld_16x32bx2_x32<HC>(to + (16u << 16) + 32 * c, r1);
      tmem_ld_wait(r0);
      tmem_ld_wait(r1);
      if (c == HC / 32 - 1) warp_arrive(C::kBarOFree);  // O may be overwritten now
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint64_t a = f2_pack(__uint_as_float(r0[2 * i]), __uint_as_float(r0[2 * i + 1]));
        const uint64_t b = f2_pack(__uint_as_float(r1[2 * i]), __uint_as_float(r1[2 * i + 1]));
        const uint64_t o2 = f2_mul(b, inv1), o = f2_fma(o2, weight, f2_mul(a, inv0));
        w[c][i] = pack_bf16x2(f2_lo(o), f2_hi(o));
        w2[c][i] = pack_bf16x2(f2_lo(o2), f2_hi(o2));
      }
    }
    const unsigned gap = is.nx1.w < 0 ? 0 : C::kStoreGapNs;  // none behind the last item
    if (live) {
#pragma unroll
      for (int c = 0; c < HC / 32; ++c) {
        store32(static_cast<__nv_bfloat16*>(p.out) + orow + 32 * c, w[c], gap);
        if (p.out2 != nullptr) store32(static_cast<__nv_bfloat16*>(p.out2) + orow + 32 * c, w2[c], gap);
      }
    }
    if (live) *lse = (ml.y > 0.f) ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
  }
}

// ------------------------------------------------------------------- kernel

template <int KB, int D, bool SPLIT>
__global__ void __launch_bounds__(DiffFwdCfg<KB, D>::kThreads, 1)
    bsa_diff_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const DiffFwdParams p) {
  using C = DiffFwdCfg<KB, D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
    for (int x = 0; x < 3; ++x) {
      mbar_init(bar(C::kBarSF + x), 1);
      mbar_init(bar(C::kBarPVD + x), 1);
      mbar_init(bar(C::kBarKF + x), 1);
      mbar_init(bar(C::kBarVF + x), 1);
      mbar_init(bar(C::kBarPF + x), 4 * C::kNumWG);
    }
    mbar_init(bar(C::kBarDrainS), 1);
    mbar_init(bar(C::kBarDrainP), 1);
    mbar_init(bar(C::kBarOFree), 4);
    mbar_init(bar(C::kBarStFull), 4 * C::kNumWG);
    mbar_init(bar(C::kBarStFree), 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(C::kBarQF + x), 1);
      mbar_init(bar(C::kBarQE + x), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    wait_before();  // TMEM is not held across it (launch_after)
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if constexpr (SPLIT) {  // the column halves that no copy writes
    for (int i = threadIdx.x; i < C::kNQ * C::kQTile / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, p.expire_site};
  wait_before();

  if (warp < C::kSoftWarp) {
    setmaxnreg_dec<C::kRegCtl>();
    if (warp == 0) {
      if (lane == 0) diff_producer<KB, D>(p, &tm_k, &tm_v, sbase, ctl);
    } else if (warp == 1) {
      if (lane == 0) diff_mma_s<KB, D>(p, sbase, tmem, ctl);
    } else if (warp == 2) {
      if (lane == 0) fwd_mma_pv<128, KB, D>(p, sbase, tmem, ctl);
    } else {
      if (lane == 0) diff_query_producer<KB, D, SPLIT>(p, &tm_q, sbase, ctl);
    }
  } else if (warp < C::kEpiWarp) {
    setmaxnreg_inc<C::kRegSoft>();
    diff_softmax<KB, D>(p, sbase, smem, tmem, ctl);
  } else {
    setmaxnreg_dec<C::kRegEpi>();
    diff_epilogue<KB, D>(p, sbase, smem, tmem, ctl);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int KB, int D, bool SPLIT>
cudaError_t launch_diff_fwd(const DiffFwdParams& p, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, int grid, cudaStream_t stream) {
  using C = DiffFwdCfg<KB, D>;
  static_assert(C::kEpi && C::kSplitRegs, "roles");
  auto* kernel = bsa_diff_fwd_kernel<KB, D, SPLIT>;
  static int done[64] = {0}, split_ok[64] = {0};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = set_smem_once(kernel, C::kLaunchSmem, done);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !split_ok[dev]) {
    // setmaxnreg.inc waits for registers that the other warpgroups gave back: the shares only
    // add up when the kernel is launched at exactly kLaunchRegs.
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != C::kLaunchRegs) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) split_ok[dev] = 1;
  }
  return launch_after(kernel, dim3(grid), C::kThreads, C::kLaunchSmem, stream, q, k, v, p);
}

}  // namespace bsa
