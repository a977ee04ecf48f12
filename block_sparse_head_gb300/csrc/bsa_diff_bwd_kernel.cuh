// bsa_diff_bwd_kernel.cuh -- backward of block-sparse differential attention for sm_103a.
//
// With P_m = exp(scale q_m . k - lse_m) on the active entries, w = (1, -lam), dP = dO V^T and
// D_m = rowsum(dO * O_m):
//     dS_m = w_m P_m (dP - D_m),   dQ_m = scale dS_m K_m,   dK_m = scale dS_m^T Q_m,
//     dV = (P_0 - lam P_1)^T dO,   dlam = -D_1.
// K, V and their gradients are shared by both maps and by the heads of a kv head.
//
// The row terms are bsa_diff_rows.cu's; the two walks here are dQ over the layout's rows and dK and
// dV over its columns.
// Both are the plain backward's pipelines (bsa_bwd_kernel.cuh: roles, barriers, TMEM regions) on
// tiles of 64 queries with both maps as 128 rows, row 64 a + 32 m + r being query 32 a + r under
// map m:
//   dQ walk    item: such a tile, A = its Q, B = its dO (each row twice).  Step: 128 keys,
//              X = K, Y = V.  T1 = A X^T, T2 = B Y^T, E = dS, acc += E X.  The row sums of
//              P_m dP, in fp32 throughout, are D_m without the rounding of the bf16 outputs:
//              they give dlam, and the dK/dV walk takes them instead of the row terms' D.
//   dK/dV walk item: a key block, A = K, B = V (rows: keys).  Step: 64 queries of one head of
//              the kv head, X = Q of both maps (128 rows), Y = dO (64 rows).  T1 = A X^T (128
//              columns), T2 = B Y^T (64 columns, for both maps).  A thread's 64 columns of T1
//              are 32 queries under both maps, so that E1 = P_0^T - lam P_1^T, combined in fp32
//              and rounded once, takes 64 columns (half the product of two maps apart), and
//              E2 = dS^T 128.  acc1 += E1 Y = dV,  acc2 += E2 X = dK / scale: the sum over maps
//              and heads stays in TMEM.  A column's steps are its entries times heads times
//              halves, and columns differ widely (a global one is seen by every row), so that
//              the CTAs share the steps, not the columns out: of a column that
//              is cut, each CTA but the last one there leaves an fp32 piece, which that one joins.
// Queries of d / 2 numbers are laid out over d columns, zero in the other map's half
// (bsa_diff.cuh): E2 X then puts each map's dK into its own columns.
// Rows past the end of the sequence read as zero and carry -lse = -inf, so that their P is 0;
// keys past it have K = V = 0: the dQ walk masks them, the dK/dV walk does not store them.
// P, dS and their combinations are rounded to bf16 for their products; scores, dP, D, the sums
// over keys, rows, maps and heads and dlam's sum are fp32 or more, and each gradient is rounded
// once.  Every wait is bounded (WaitCtl), as in the plain kernels.
//
// Bound: the chain of a step, products -> TMEM loads -> exponentials and dS -> TMEM stores ->
// products; the tensor pipe works 52 % of the dQ walk's time and 49 % of the other's.  Timing copies
// without one part each: no row terms -1 %, no exponentials -2 %, a quarter of the first products
// -14 %, of the second ones -7 %.
// Measured (dQ + dK/dV): 16 heads of 128 on 4 kv heads, 8,192 tokens, block 128, a band and a
// stride: 185 + 205 us, 1,090 TFLOP/s (0.58 of a cuBLAS bf16 product; 0.39 without the scores and
// dP that the second walk computes again); 2 x 8 heads of 64, 2,999 tokens, block 64, a window
// and a global block: 27 + 37 us; 2 x 2 heads, 333 tokens: 10 + 16 us, one CTA's way.  What
// counted, at the first: columns' steps shared by the CTAs (whole columns: 510 and 230 us);
// packed fp32 arithmetic, masks only in the blocks that need them, dP's buffer released once it
// is loaded (dQ 232 -> 192); cut columns joined by the last CTA there rather than by a kernel of
// their own (15 to 30 us); three stages of queries and dP over the scores' second half, so that
// the next scores run ahead (dK/dV 218 -> 209); at block 64 two groups of warps in turn (41 ->
// 37); masks as a pass of their own instead of a second copy of a step's code, which competes for
// the instruction cache (dQ 196 -> 181, dK/dV 207 -> 205); the end of the sequence masked in the
// dQ walk costs 4 us of these (dQ 185).
#pragma once

#include "bsa_bwd_kernel.cuh"
#include "bsa_diff.cuh"

namespace bsa {

__device__ __forceinline__ int2 stream_range(const DiffBwdParams& p) {
  return stream_range(static_cast<const DiffList&>(p));
}
__device__ __forceinline__ int4 stream_item(const DiffBwdParams& p, int u) {
  return stream_item(static_cast<const DiffList&>(p), u);
}
__device__ __forceinline__ int4 stream_place(const DiffBwdParams& p, int u, const int4& r) {
  return stream_place(static_cast<const DiffList&>(p), u, r);
}

// Row terms of 64 queries: two groups of 32, each [-lse_0, -lse_1 (log2 units), -D_0, -D_1, -lam]
// of 32 fp32 (negated: they are added) and 16 bytes of room, so that the two half-warps, which
// read the same places of different groups, hit different banks.
constexpr int kDiffVecHalf = 5 * 32 + 4;
constexpr int kDiffVec = 2 * kDiffVecHalf;
static_assert(kDiffVec == kDiffVecFloats, "workspace");

template <int BLK, int D, bool KV>
struct DiffBwdCfg {
  static constexpr int kRows = KV ? BLK : 128;         // rows of an item tile
  static constexpr int kEwWarps = 8;                   // elementwise warps
  // Those of one step: eight for 128 rows; for 64 rows (dK/dV, block 64) four, and the two groups
  // take steps in turn.
  static constexpr int kStepWarps = kRows / 16;
  static constexpr int kGroups = kEwWarps / kStepWarps;
  static constexpr int kMma2Warp = 2 + kEwWarps;
  static constexpr int kThreads = 32 * (3 + kEwWarps);
  static constexpr int kG = KV ? 1 : 128 / BLK;        // key blocks of a step (dQ walk)
  static constexpr int kHalves = BLK / 64;             // query tiles of a block
  static constexpr int kItemTile = kRows * D * 2;
  static constexpr int kItemPlane = kRows * 128;       // 64 columns of an item tile
  static constexpr int kXTile = 128 * D * 2;           // dQ: K of a step; dK/dV: Q of both maps
  static constexpr int kXBlk = KV ? 128 : BLK;         // rows that one plane of X holds
  static constexpr int kXPlane = kXBlk * 128;
  static constexpr int kXBlkB = kXBlk * D * 2;
  static constexpr int kYTile = (KV ? 64 : 128) * D * 2;
  static constexpr int kYPlane = (KV ? 64 : BLK) * 128;
  static constexpr int kNX = 3;             // X slots (dK/dV: stages of X, Y and the row terms)
  static constexpr int kNY = KV ? 3 : 2;
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kItemTile;
  static constexpr int kOffX = 2 * kItemTile;
  static constexpr int kOffY = kOffX + kNX * kXTile;
  static constexpr int kVecB = kDiffVec * 4;
  static constexpr int kOffVec = kOffY + kNY * kYTile;
  static constexpr int kOffBar = kOffVec + (KV ? kNX * kVecB : 0);
  // barriers
  static constexpr int kBarIF = 0;     // item tiles landed (dK/dV: A's)
  static constexpr int kBarIE = 1;     // item tiles free (dK/dV: A's)
  static constexpr int kBarXF = 2;     // [3] X landed (dK/dV: X, Y and the row terms)
  static constexpr int kBarXE = 5;     // [3] X free
  static constexpr int kBarYF = 8;     // [2] dQ: Y landed
  static constexpr int kBarYE = 10;    // [2] dQ: Y free
  // By the step's parity, so that one who waits for a step's phase (the second issuer, a group of
  // warps) cannot miss it: the next one needs that step's second products.
  static constexpr int kBarTF = 12;    // [2] T1 (dQ: and T2) computed
  static constexpr int kBarDF = 14;    // [2] dK/dV: T2 computed
  static constexpr int kBarEF1 = 16;   // [2] dK/dV: E1 written (a step's warps)
  static constexpr int kBarEF = 18;    // [2] E (E2) written (a step's warps)
  static constexpr int kBarAD = 20;    // [2] a step's second products done
  static constexpr int kBarDL = 22;    // dQ: T2 loaded; dK/dV: T1 loaded (a step's warps)
  static constexpr int kBarAR = 23;    // accumulators read out (a step's warps)
  static constexpr int kBarIFV = 24;   // dK/dV: item tile B landed
  static constexpr int kBarIEV = 25;   // dK/dV: item tile B free
  static constexpr int kBarDrain = 26, kBarDrain2 = 27, kNumBars = 28;
  static constexpr int kBarBytes = 256;
  static_assert(kNumBars * 8 + 8 <= kBarBytes && kOffBar % 8 == 0 && kOffVec % 16 == 0, "barrier area");
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static constexpr int kLaunchSmem = kSmemBytes > 120 * 1024 ? kSmemBytes : 120 * 1024;
  // TMEM columns.  dQ: T1 at 0 or 256 (E over it), T2 at 128, acc at 384.  dK/dV: a step's T1 at 0
  // or 128, T2 (and E2) over its second half, E1 over its first; acc at 256.
  static constexpr int kT1 = 0, kT2 = 128, kT1b = 256;
  static constexpr int kAcc1 = KV ? 256 : 384, kAcc2 = 256 + D;
  static constexpr uint32_t kIdescT1 = idesc_bf16_f32(kRows, KV ? 128 : BLK, false, false);
  static constexpr uint32_t kIdescT2 = idesc_bf16_f32(kRows, KV ? 64 : BLK, false, false);
  static constexpr uint32_t kIdescAcc = idesc_bf16_f32(kRows, D, false, true);  // B MN-major
};

// This CTA's steps of the dK/dV walk (see DiffBwdParams), a column's end loaded one column ahead.
struct DiffKvWalk {
  long long left;    // steps still to go, this one among them
  int per;           // steps of a column's entry: heads of the kv head times halves
  int b, x, rest;    // batch, entry of row_idx, head * halves + half
  int col, begin, end, next_end;  // column and its entries; the next column's end
  bool first, head;  // first step of the piece; the piece begins the column
  __device__ __forceinline__ int end_of(const DiffBwdParams& p, int c) const {
    return c < p.cols ? p.col_ptr[c + 1] : 0;
  }
  __device__ __forceinline__ void init(const DiffBwdParams& p) {
    const long long at = blockIdx.x * p.share;
    left = p.steps - at < p.share ? p.steps - at : p.share;
    if (left <= 0) return;
    per = p.pairs * p.halves;
    const long long entry = diff_div(at, per);
    rest = static_cast<int>(at - entry * per);
    b = static_cast<int>(diff_div(entry, p.nnz));
    x = static_cast<int>(entry - static_cast<long long>(b) * p.nnz);
    col = diff_column(p, x);
    begin = p.col_ptr[col];
    end = p.col_ptr[col + 1];
    next_end = end_of(p, col + 1);
    first = true;
    head = x == begin && rest == 0;
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ bool tail() const { return x + 1 == end && rest + 1 == per; }
  __device__ __forceinline__ bool last() const { return left == 1 || tail(); }
  __device__ __forceinline__ void advance(const DiffBwdParams& p) {
    --left;
    first = false;
    if (++rest < per) return;
    rest = 0;
    if (++x < end || left <= 0) return;
    first = head = true;
    do {  // the next column with entries
      if (++col == p.cols) {
        col = 0;
        ++b;
        x = 0;
        begin = 0;
        end = p.col_ptr[1];
      } else {
        begin = end;
        end = next_end;
      }
      next_end = end_of(p, col + 1);
    } while (begin == end);
  }
};

// Both maps' rows of 64 queries of head `pair`, 32 at a time, into a tile of 128 rows.
// `tile` planes are 128 rows apart.  SPLIT: one plane a map.
template <int D, bool SPLIT>
__device__ __forceinline__ void diff_load_q(uint32_t tile, const CUtensorMap* tm, uint32_t bar,
                                            int q0, int pair) {
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int z = 0; z < (SPLIT ? 1 : D / 64); ++z)
        tma_load_4d(tile + (SPLIT ? m : z) * (128 * 128) + (64 * a + 32 * m) * 128, tm, bar, 0,
                    q0 + 32 * a, z, 2 * pair + m);
}

// ----------------------------------------------------------------- producers

template <int BLK, int D, bool SPLIT>
__device__ __forceinline__ void diff_dq_producer(const DiffBwdParams& p, const CUtensorMap* tm_q,
                                                 const CUtensorMap* tm_do, const CUtensorMap* tm_k,
                                                 const CUtensorMap* tm_v, uint32_t sbase,
                                                 const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, false>;
  constexpr int G = C::kG;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  StepCursor<G> c;
  c.init(p);
  int n = -1;          // items whose tiles were armed
  int nx = 0, ny = 0;  // steps whose X (Y) copies were armed
  for (int t = 0; c.valid(); ++t) {
    const int nblk = c.nblk();
    const int pair = c.is.cur.x, q0 = c.is.cur.y * 64, head = diff_over(pair, p.pairs_mul, p.pairs_shift);
    int cols[G];
#pragma unroll
    for (int g = 0; g < G; ++g) cols[g] = (g < nblk) ? p.col_idx[c.is.cur.z + c.s * G + g] : 0;
    if (c.s == 0) {
      // Free once the previous item's last T1 and T2 are complete.
      if (n >= 0 && !mbar_wait(bar(C::kBarIE), n & 1, ctl, kSiteProdKEmpty)) break;
      const uint32_t fb = bar(C::kBarIF);
      mbar_arrive_expect_tx(fb, (SPLIT ? C::kItemTile / 2 : C::kItemTile) + C::kItemTile);
      ++n;
      diff_load_q<D, SPLIT>(sbase + C::kOffA, tm_q, fb, q0, pair);
#pragma unroll 1
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int z = 0; z < D / 64; ++z)
            tma_load_4d(sbase + C::kOffB + z * C::kItemPlane + (64 * a + 32 * m) * 128, tm_do, fb, 0,
                        q0 + 32 * a, z, pair);
    }
    c.advance(p);
    // X slot t % 3 held K(t-3), read by the dQ product of t-3; Y slot t % 2 held V(t-2), read
    // by T2(t-2).
    if (t >= 3 && !mbar_wait(bar(C::kBarXE + t % 3), ((t - 3) / 3) & 1, ctl, kSiteProdKEmpty)) break;
    const uint32_t fx = bar(C::kBarXF + t % 3);
    mbar_arrive_expect_tx(fx, nblk * C::kXBlkB);
    const uint32_t xd = sbase + C::kOffX + (t % 3) * C::kXTile;
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < nblk) tma_load_4d(xd + g * C::kXBlkB, tm_k, fx, 0, cols[g] * BLK, 0, head);
    ++nx;
    if (t >= 2 && !mbar_wait(bar(C::kBarYE + t % 2), ((t - 2) / 2) & 1, ctl, kSiteProdVEmpty)) break;
    const uint32_t fy = bar(C::kBarYF + t % 2);
    mbar_arrive_expect_tx(fy, nblk * C::kXBlkB);
    const uint32_t yd = sbase + C::kOffY + (t % 2) * C::kYTile;
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (g < nblk) tma_load_4d(yd + g * C::kXBlkB, tm_v, fy, 0, cols[g] * BLK, 0, head);
    ++ny;
  }
  // Wait for every copy this thread issued (immediate on the normal path).
  for (int j = (nx > 3 ? nx - 3 : 0); j < nx; ++j) mbar_drain_wait(bar(C::kBarXF + j % 3), (j / 3) & 1);
  for (int j = (ny > 2 ? ny - 2 : 0); j < ny; ++j) mbar_drain_wait(bar(C::kBarYF + j % 2), (j / 2) & 1);
  if (n >= 0) mbar_drain_wait(bar(C::kBarIF), n & 1);
}

template <int BLK, int D, bool SPLIT>
__device__ __forceinline__ void diff_kv_producer(const DiffBwdParams& p, const CUtensorMap* tm_k,
                                                 const CUtensorMap* tm_v, const CUtensorMap* tm_q,
                                                 const CUtensorMap* tm_do, uint32_t sbase,
                                                 const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, true>;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  DiffKvWalk c;
  c.init(p);
  const int tiles = (p.L + 63) / 64;
  int n = -1, t = 0;  // pieces whose A was armed; steps armed
  int nv = 0;         // pieces whose B was armed
  int head = 0, key0 = 0;
  for (; c.valid(); ++t) {
    if (c.first) {
      const int kv = c.col / p.nb;
      head = c.b * (p.cols / p.nb) + kv;
      key0 = (c.col - kv * p.nb) * BLK;
    }
    const int pair = head * p.pairs + c.rest / C::kHalves;
    const int q64 = p.row_idx[c.x] * C::kHalves + c.rest % C::kHalves;
    const bool item_first = c.first;
    if (item_first) {
      // A is free once the previous piece's last T1 is complete.
      if (n >= 0 && !mbar_wait(bar(C::kBarIE), n & 1, ctl, kSiteProdKEmpty)) break;
      const uint32_t fb = bar(C::kBarIF);
      mbar_arrive_expect_tx(fb, C::kItemTile);
      ++n;
      tma_load_4d(sbase + C::kOffA, tm_k, fb, 0, key0, 0, head);
    }
    c.advance(p);
    // Stage t % 3 held step t-3, read by its dV and dK products.
    if (t >= 3 && !mbar_wait(bar(C::kBarXE + t % 3), ((t - 3) / 3) & 1, ctl, kSiteProdVEmpty)) break;
    const uint32_t fb = bar(C::kBarXF + t % 3);
    mbar_arrive_expect_tx(fb, (SPLIT ? C::kXTile / 2 : C::kXTile) + C::kYTile + C::kVecB);
    diff_load_q<D, SPLIT>(sbase + C::kOffX + (t % 3) * C::kXTile, tm_q, fb, q64 * 64, pair);
    tma_load_4d(sbase + C::kOffY + (t % 3) * C::kYTile, tm_do, fb, 0, q64 * 64, 0, pair);
    // A block's second half may lie past the sequence; the row terms have room for it.
    bulk_load(sbase + C::kOffVec + (t % 3) * C::kVecB,
              p.vec + (static_cast<int64_t>(pair) * diff_vec_tiles(tiles) + q64) * kDiffVec, C::kVecB, fb);
    if (item_first) {
      // B (V) after the step's tiles: the previous item's last T2 completes later.
      if (nv > 0 && !mbar_wait(bar(C::kBarIEV), (nv - 1) & 1, ctl, kSiteProdKEmpty)) {
        ++t;
        break;
      }
      const uint32_t fv = bar(C::kBarIFV);
      mbar_arrive_expect_tx(fv, C::kItemTile);
      tma_load_4d(sbase + C::kOffB, tm_v, fv, 0, key0, 0, head);
      ++nv;
    }
  }
  for (int j = (t > 3 ? t - 3 : 0); j < t; ++j) mbar_drain_wait(bar(C::kBarXF + j % 3), (j / 3) & 1);
  if (n >= 0) mbar_drain_wait(bar(C::kBarIF), n & 1);
  if (nv > 0) mbar_drain_wait(bar(C::kBarIFV), (nv - 1) & 1);
}

// ---------------------------------------------------------------- MMA issuers

// td = item tile x step tile^T over d; rows of the step in blocks of N (idesc), nb of them.
template <int D, int PLANE_I, int PLANE_S, int BLOCK_B, int NCOL>
__device__ __forceinline__ void diff_issue_first(uint32_t td, uint32_t it, uint32_t st, uint32_t hi,
                                                 uint32_t idesc, int nb) {
  auto mmas = [&](int n) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t ia = ((kk >> 2) * PLANE_I + (kk & 3) * 32) >> 4;
      const uint32_t is = ((kk >> 2) * PLANE_S + (kk & 3) * 32) >> 4;
#pragma unroll
      for (int g = 0; g < n; ++g)
        tc_mma_ss_lh(td + g * NCOL, it + ia, hi, st + is + ((g * BLOCK_B) >> 4), hi, idesc,
                     kk > 0 ? 1u : 0u);
    }
  };
  // A branch between two MMAs slows their issue.
  if (nb > 1)
    mmas(2);
  else
    mmas(1);
}

template <int BLK, int D>
__device__ __forceinline__ void diff_dq_mma(const DiffBwdParams& p, uint32_t sbase, uint32_t tmem,
                                            const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, false>;
  constexpr int G = C::kG;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const uint64_t a_desc = sdesc_sw128(sbase + C::kOffA, 16, 1024);
  const uint32_t hi = static_cast<uint32_t>(a_desc >> 32);
  const uint32_t a0 = static_cast<uint32_t>(a_desc);
  const uint32_t b0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffB, 16, 1024));
  const uint32_t x0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffX, 16, 1024));
  const uint32_t y0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffY, 16, 1024));
  StepCursor<G> c;
  c.init(p);
  int n = -1;
  for (int t = 0; c.valid(); ++t) {
    const int nblk = G == 1 ? 1 : c.nblk();
    const bool first = c.s == 0, last = c.s == c.nsteps - 1;
    c.advance(p);
    if (first) {
      ++n;
      if (!mbar_wait(bar(C::kBarIF), n & 1, ctl, kSiteMmaStage)) break;
    }
    if (!mbar_wait(bar(C::kBarXF + t % 3), (t / 3) & 1, ctl, kSiteMmaStage)) break;
    // This T1 region held step t-2, whose dQ product read E from it.
    if (t >= 2 && !mbar_wait(bar(C::kBarAD + (t & 1)), ((t - 2) / 2) & 1, ctl, kSiteMmaPvDone)) break;
    tc_fence_after();
    diff_issue_first<D, C::kItemPlane, C::kXPlane, C::kXBlkB, BLK>(
        tmem + ((t & 1) ? C::kT1b : C::kT1), a0, x0 + (t % 3) * (C::kXTile >> 4), hi, C::kIdescT1, nblk);
    // T2 is free once the elementwise warps have loaded that of step t-1.
    if (t >= 1 && !mbar_wait(bar(C::kBarDL), (t - 1) & 1, ctl, kSiteMmaPFull)) break;
    if (!mbar_wait(bar(C::kBarYF + t % 2), (t / 2) & 1, ctl, kSiteMmaStage)) break;
    tc_fence_after();
    diff_issue_first<D, C::kItemPlane, C::kYPlane, C::kXBlkB, BLK>(
        tmem + C::kT2, b0, y0 + (t % 2) * (C::kYTile >> 4), hi, C::kIdescT2, nblk);
    tc_commit(bar(C::kBarTF + (t & 1)));
    tc_commit(bar(C::kBarYE + t % 2));
    if (last) tc_commit(bar(C::kBarIE));
  }
  tc_commit(bar(C::kBarDrain));
  mbar_drain_wait(bar(C::kBarDrain), 0);
}

// dQ walk, second issuing thread: acc += dS K of step u once the warps have written dS.
template <int BLK, int D>
__device__ __forceinline__ void diff_dq_mma2(const DiffBwdParams& p, uint32_t sbase, uint32_t tmem,
                                             const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, false>;
  constexpr int G = C::kG;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const uint64_t x_desc = sdesc_sw128(sbase + C::kOffX, C::kXPlane, 1024);
  const uint32_t hi = static_cast<uint32_t>(x_desc >> 32);
  const uint32_t x0 = static_cast<uint32_t>(x_desc);
  StepCursor<G> c;
  c.init(p);
  int n = -1;
  for (int u = 0; c.valid(); ++u) {
    const int nblk = c.nblk();
    const bool first = c.s == 0;
    c.advance(p);
    if (first) ++n;
    if (!mbar_wait(bar(C::kBarEF + (u & 1)), (u / 2) & 1, ctl, kSiteMmaPFull)) break;
    if (first && n > 0 && !mbar_wait(bar(C::kBarAR), (n - 1) & 1, ctl, kSiteMmaPFull)) break;
    tc_fence_after();
    const uint32_t te = tmem + ((u & 1) ? C::kT1b : C::kT1), xs = x0 + (u % 3) * (C::kXTile >> 4);
    auto one = [&](int kk) {
      const uint32_t bo = ((((kk * 16) / BLK) * C::kXBlkB + ((kk * 16) % BLK) * 128) >> 4);
      tc_mma_ts_lh(tmem + C::kAcc1, te + kk * 8, xs + bo, hi, C::kIdescAcc, (first && kk == 0) ? 0u : 1u);
    };
#pragma unroll
    for (int kk = 0; kk < (G == 1 ? 8 : 4); ++kk) one(kk);
    if (G == 2 && nblk > 1) {
#pragma unroll
      for (int kk = 4; kk < 8; ++kk) one(kk);
    }
    tc_commit(bar(C::kBarAD + (u & 1)));
    tc_commit(bar(C::kBarXE + u % 3));
  }
  tc_commit(bar(C::kBarDrain2));
  mbar_drain_wait(bar(C::kBarDrain2), 0);
}

// dK/dV walk: T1 and T2.  Steps alternate between two regions of 128 columns.  T1(t) fills one;
// once every elementwise warp has loaded it, T2(t) goes into its second half; E1(t) and then E2(t)
// (over T2(t)) are written there as well.  So T1(t+1) needs the products of t-1 only, and runs
// while the warps are at step t.  Per step, here: T2(t), then T1(t+1).
template <int BLK, int D>
__device__ __forceinline__ void diff_kv_mma(const DiffBwdParams& p, uint32_t sbase, uint32_t tmem,
                                            const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, true>;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const uint64_t a_desc = sdesc_sw128(sbase + C::kOffA, 16, 1024);
  const uint32_t hi = static_cast<uint32_t>(a_desc >> 32);
  const uint32_t a0 = static_cast<uint32_t>(a_desc);
  const uint32_t b0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffB, 16, 1024));
  const uint32_t x0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffX, 16, 1024));
  const uint32_t y0 = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffY, 16, 1024));
  auto issue1 = [&](int t) {
    diff_issue_first<D, C::kItemPlane, C::kXPlane, 0, 128>(tmem + ((t & 1) ? C::kT2 : C::kT1), a0,
                                                           x0 + (t % 3) * (C::kXTile >> 4), hi,
                                                           C::kIdescT1, 1);
  };
  DiffKvWalk c;
  c.init(p);
  if (c.valid()) {
    int n = 0;
    bool first = true, last = c.last();
    c.advance(p);
    bool ok = mbar_wait(bar(C::kBarIF), 0, ctl, kSiteMmaStage) &&
              mbar_wait(bar(C::kBarXF), 0, ctl, kSiteMmaStage);
    if (ok) {
      tc_fence_after();
      issue1(0);  // S^T = K Q^T
      tc_commit(bar(C::kBarTF));
      if (last) tc_commit(bar(C::kBarIE));
    }
    for (int t = 0; ok; ++t) {
      if (first && !mbar_wait(bar(C::kBarIFV), n & 1, ctl, kSiteMmaStage)) break;
      if (!mbar_wait(bar(C::kBarDL), t & 1, ctl, kSiteMmaPFull)) break;
      tc_fence_after();
      diff_issue_first<D, C::kItemPlane, C::kYPlane, 0, 64>(
          tmem + ((t & 1) ? C::kT2 : C::kT1) + 64, b0, y0 + (t % 3) * (C::kYTile >> 4), hi,
          C::kIdescT2, 1);  // dP^T = V dO^T
      tc_commit(bar(C::kBarDF + (t & 1)));
      if (last) tc_commit(bar(C::kBarIEV));
      if (!c.valid()) break;
      first = c.first;
      last = c.last();
      c.advance(p);
      if (first && !mbar_wait(bar(C::kBarIF), (n + 1) & 1, ctl, kSiteMmaStage)) break;
      if (!mbar_wait(bar(C::kBarXF + (t + 1) % 3), ((t + 1) / 3) & 1, ctl, kSiteMmaStage)) break;
      // Two barriers, by region: the next phase of this one is step t+1's own.
      if (t >= 1 && !mbar_wait(bar(C::kBarAD + ((t + 1) & 1)), ((t - 1) / 2) & 1, ctl, kSiteMmaPvDone))
        break;
      tc_fence_after();
      issue1(t + 1);
      tc_commit(bar(C::kBarTF + ((t + 1) & 1)));
      if (last) tc_commit(bar(C::kBarIE));
      if (first) ++n;
    }
  }
  tc_commit(bar(C::kBarDrain));
  mbar_drain_wait(bar(C::kBarDrain), 0);
}

// dK/dV walk, second issuing thread: dV += E1 dO once E1 is written, dK += E2 Q once E2 is.
template <int BLK, int D>
__device__ __forceinline__ void diff_kv_mma2(const DiffBwdParams& p, uint32_t sbase, uint32_t tmem,
                                             const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, true>;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const uint64_t x_desc = sdesc_sw128(sbase + C::kOffX, C::kXPlane, 1024);
  const uint64_t y_desc = sdesc_sw128(sbase + C::kOffY, C::kYPlane, 1024);
  const uint32_t hi = static_cast<uint32_t>(x_desc >> 32);
  const uint32_t x0 = static_cast<uint32_t>(x_desc), y0 = static_cast<uint32_t>(y_desc);
  DiffKvWalk c;
  c.init(p);
  int n = -1;
  for (int t = 0; c.valid(); ++t) {
    const bool first = c.first;
    c.advance(p);
    if (first) ++n;
    const uint32_t t1 = tmem + ((t & 1) ? C::kT2 : C::kT1);
    if (!mbar_wait(bar(C::kBarEF1 + (t & 1)), (t / 2) & 1, ctl, kSiteMmaPFull)) break;
    if (first && n > 0 && !mbar_wait(bar(C::kBarAR), (n - 1) & 1, ctl, kSiteMmaPFull)) break;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      tc_mma_ts_lh(tmem + C::kAcc1, t1 + kk * 8, y0 + (t % 3) * (C::kYTile >> 4) + ((kk * 16 * 128) >> 4),
                   hi, C::kIdescAcc, (first && kk == 0) ? 0u : 1u);
    if (!mbar_wait(bar(C::kBarEF + (t & 1)), (t / 2) & 1, ctl, kSiteMmaPFull)) break;
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      tc_mma_ts_lh(tmem + C::kAcc2, t1 + 64 + kk * 8,
                   x0 + (t % 3) * (C::kXTile >> 4) + ((kk * 16 * 128) >> 4), hi, C::kIdescAcc,
                   (first && kk == 0) ? 0u : 1u);
    tc_commit(bar(C::kBarAD + (t & 1)));
    tc_commit(bar(C::kBarXE + t % 3));
  }
  tc_commit(bar(C::kBarDrain2));
  mbar_drain_wait(bar(C::kBarDrain2), 0);
}

// dlam[h], by the second issuing warp of CTA h, h + grid, .. before its first product is due: the
// sums of 16 rows that the dQ walk left, added in fp64 and a fixed order.
__device__ __forceinline__ void diff_sum_lam(const DiffBwdParams& p, int lane) {
  const int per = 4 * diff_vec_tiles((p.L + 63) / 64), live = 4 * ((p.L + 63) / 64);
  for (int h = blockIdx.x; h < p.H; h += gridDim.x) {
    double s = 0.0;
    for (int b = 0; b < p.B; ++b) {
      const float* x = p.lam_sums + (static_cast<int64_t>(b) * p.H + h) * per;
      for (int i = lane; i < live; i += 8 * 32) {
        float y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) y[u] = i + 32 * u < live ? x[i + 32 * u] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += static_cast<double>(y[u]);
      }
    }
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) s += __shfl_xor_sync(0xffffffffu, s, w);
    if (lane == 0) p.dlam[h] = static_cast<float>(s);
  }
}

// ----------------------------------------------------------- elementwise warps

template <int BLK, int D, bool SPLIT>
__device__ __forceinline__ void diff_dq_elementwise(const DiffBwdParams& p, uint32_t sbase,
                                                    uint32_t tmem, const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, false>;
  constexpr int G = C::kG, DQ = SPLIT ? D / 2 : D;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const int wg = ((threadIdx.x >> 5) - 2) >> 2;
  const int wq = (threadIdx.x >> 5) & 3;
  const int lane = threadIdx.x & 31;
  const int half = lane >> 4;
  // Row 64 a + 32 m + r of the tile is query 32 a + r under map m.
  const int map = wq & 1;
  const int qin = 32 * (wq >> 1) + wg * 16 + (lane & 15);
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32 + wg * 16) << 16);
  const int kbase = (BLK == 128) ? 64 * half : 0;
  const int tiles = diff_vec_tiles((p.L + 63) / 64);
  auto warp_arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  auto wait_bar = [&](int b, int parity, int site) -> bool {
    bool w = mbar_wait(bar(b), parity, ctl, site);
    w = __all_sync(0xffffffffu, w);
    if (w) tc_fence_after();
    return w;
  };
  // This thread's 32-column groups of an accumulator row (read_o's) that are the row's dQ: all
  // of them, or (SPLIT) its map's half.
  auto store_dq = [&](int64_t pair, int q, const uint32_t (&pk)[D / 4]) {
    if (q >= p.L) return;
    __nv_bfloat16* r = static_cast<__nv_bfloat16*>(p.dq) + ((2 * pair + map) * p.L + q) * DQ + half * 32;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      if (SPLIT && c != map) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(r + (SPLIT ? 0 : c * 64) + i * 8) =
            make_uint4(pk[16 * c + 4 * i], pk[16 * c + 4 * i + 1], pk[16 * c + 4 * i + 2],
                       pk[16 * c + 4 * i + 3]);
    }
  };
  // dlam of the second map's rows: one number each, or (one weight a head) sums of 16 rows, which
  // the dK/dV walk's kernel adds up.
  auto store_lam = [&](int64_t pair, int tile, float x) {
    if (map == 0) return;
    if (p.lam_rows) {
      const int q = tile * 64 + qin;
      if (half == 0 && q < p.L) p.dlam[pair * p.L + q] = x;
      return;
    }
    if (tile * 64 + qin >= p.L) x = 0.f;
#pragma unroll
    for (int k = 1; k < 16; k *= 2) x += __shfl_xor_sync(0xffffffffu, x, k);
    if (lane == 0) p.lam_sums[(pair * tiles + tile) * 4 + (qin >> 4)] = x;
  };
  // The previous item's accumulator goes out at the next item's first step, once that step's E
  // is handed over.
  bool pending = false;
  int ppair = 0, pq = 0, pg = 0;  // its query and last step
  auto read_pending = [&]() -> bool {
    if (!wait_bar(C::kBarAD + (pg & 1), (pg / 2) & 1, kSiteSoftItemDone)) return false;
    uint32_t pk[D / 4];
    read_o<D>(tl + C::kAcc1, p.scale, pk);
    warp_arrive(C::kBarAR);
    store_dq(ppair, pq, pk);
    pending = false;
    return true;
  };

  int g = 0;
  bool ok = true;
  ItemStream is;
  for (is.init<false>(p); ok && !is.done(); is.next<false>(p)) {
    const int cnt = is.nnz();
    const int pair = is.cur.x;
    const int q = is.cur.y * 64 + qin;
    if (cnt == 0) {
      const uint32_t zero[D / 4] = {};
      store_dq(pair, q, zero);
      store_lam(pair, is.cur.y, 0.f);
      continue;
    }
    float* v = p.vec + (static_cast<int64_t>(pair) * tiles + is.cur.y) * kDiffVec + (qin >> 5) * kDiffVecHalf +
               (qin & 31);
    // dS = P (w dP - w D) with the row's weight w
    const float w = map ? v[128] : 1.f, wd = w * v[64 + 32 * map];
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), l2 = f2_pack(v[32 * map], v[32 * map]);
    const uint64_t w2 = f2_pack(w, w);
    uint64_t wd2 = f2_pack(wd, wd);
    const int dpos = p.causal_diag ? is.dpos() : -1;
    // Does the end of the sequence cut the last block?  Keys behind the end score 0, and exp(0 - lse)
    // may be more than fp32 holds.
    const bool cut = p.L % BLK != 0 && p.col_idx[is.cur.z + cnt - 1] == p.L / BLK;
    const int qblk = qin + (BLK == 128 ? (is.cur.y & 1) * 64 : 0);
    const int nsteps = (cnt + G - 1) / G;
    float rsum = 0.f;  // of P dP
    for (int s = 0; s < nsteps; ++s, ++g) {
      const int nblk = step_blocks<G>(cnt, s);
      const bool valid = (BLK == 128) || (half < nblk);
      const int place = (BLK == 128) ? s : s * 2 + half;
      if (!wait_bar(C::kBarTF + (g & 1), (g / 2) & 1, kSiteSoftSFull)) {
        ok = false;
        break;
      }
      const uint32_t t1 = tl + ((g & 1) ? C::kT1b : C::kT1);
      uint32_t rs[64], rp[64];
      tmem_ld_16x32bx2_x32<64>(t1, *reinterpret_cast<uint32_t(*)[32]>(rs));
      tmem_ld_16x32bx2_x32<64>(t1 + 32, *reinterpret_cast<uint32_t(*)[32]>(rs + 32));
      tmem_ld_16x32bx2_x32<64>(tl + C::kT2, *reinterpret_cast<uint32_t(*)[32]>(rp));
      tmem_ld_16x32bx2_x32<64>(tl + C::kT2 + 32, *reinterpret_cast<uint32_t(*)[32]>(rp + 32));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(rs));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(rs + 32));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(rp));
      tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(rp + 32));
      warp_arrive(C::kBarDL);  // T2 may now take the next step's dP
      // Keys behind the query in the diagonal block or behind the end, and a block that is not there,
      // are masked: after the exponentials, so that the steps without a mask run no second copy of
      // the code.
      int hi = valid ? (place == dpos ? qblk - kbase : 63) : -1;
      if (cut && place == cnt - 1) hi = min(hi, (p.L - 1) % BLK - kbase);
      auto pair_of = [](const uint32_t (&r)[64], int i) {
        return f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      };
#pragma unroll
      for (int i = 0; i < 32; ++i) {  // P, over the scores
        const uint64_t y = f2_fma(pair_of(rs, i), c2, l2);
        rs[2 * i] = __float_as_uint(ex2_approx(f2_lo(y)));
        rs[2 * i + 1] = __float_as_uint(ex2_approx(f2_hi(y)));
      }
      if (__any_sync(0xffffffffu, hi < 63)) {
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          rs[c] = c > hi ? 0u : rs[c];
          rp[c] = c > hi ? 0u : rp[c];
        }
      }
      uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int i = 0; i < 32; ++i) sums[i & 3] = f2_fma(pair_of(rs, i), pair_of(rp, i), sums[i & 3]);
      sums[0] = f2_add(f2_add(sums[0], sums[1]), f2_add(sums[2], sums[3]));
      const float part = f2_lo(sums[0]) + f2_hi(sums[0]);
      rsum += part;
      if (nsteps == 1) {
        // All of the row is here: D from P dP itself instead of from the rounded outputs, whose
        // error is largest in rows of few keys.
        const float all = -w * (part + __shfl_xor_sync(0xffffffffu, part, 16));
        wd2 = f2_pack(all, all);
      }
      uint32_t pk1[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint64_t ds = f2_mul(pair_of(rs, i), f2_fma(pair_of(rp, i), w2, wd2));
        pk1[i] = pack_bf16x2(f2_lo(ds), f2_hi(ds));
      }
      tmem_st_16x32bx2_x32<32>(t1, pk1);
      tmem_st_wait();
      warp_arrive(C::kBarEF + (g & 1));
      if (s == 0 && pending && !read_pending()) {
        ok = false;
        break;
      }
    }
    if (!ok) break;
    rsum += __shfl_xor_sync(0xffffffffu, rsum, 16);
    store_lam(pair, is.cur.y, -rsum);
    // For the dK/dV walk, which comes after this one.
    if (half == 0) v[64 + 32 * map] = -rsum;
    pending = true;
    ppair = pair;
    pq = q;
    pg = g - 1;
  }
  if (ok && pending) read_pending();
  tmem_st_wait();
}

template <int BLK, int D>
__device__ __forceinline__ void diff_kv_elementwise(const DiffBwdParams& p, uint32_t sbase,
                                                    const uint8_t* smem, uint32_t tmem,
                                                    const WaitCtl& ctl) {
  using C = DiffBwdCfg<BLK, D, true>;
  auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
  const int wg = ((threadIdx.x >> 5) - 2) >> 2;
  const int group = C::kGroups == 2 ? wg : 0;  // takes steps group, group + kGroups, ..
  const int gwarp = ((threadIdx.x >> 5) - 2) % C::kStepWarps;
  const int wq = (threadIdx.x >> 5) & 3;
  const int lane = threadIdx.x & 31;
  const int half = lane >> 4;
  const int row = (BLK == 128) ? (wq * 32 + wg * 16 + (lane & 15)) : (wq * 16 + (lane & 15));
  const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32 + (BLK == 128 ? wg * 16 : 0)) << 16);
  auto warp_arrive = [&](int b) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  auto wait_bar = [&](int b, int parity, int site) -> bool {
    bool w = mbar_wait(bar(b), parity, ctl, site);
    w = __all_sync(0xffffffffu, w);
    if (w) tc_fence_after();
    return w;
  };

  auto pair_of = [](const uint32_t (&r)[32], int i) {
    return f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
  };
  const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
  DiffKvWalk c;
  c.init(p);
  if (group == 1 && c.valid()) c.advance(p);
  int dpos = -1, dcol = -1;  // the diagonal block's place in column dcol
  for (int g = group; c.valid(); g += C::kGroups) {
    const uint32_t t1 = tl + ((g & 1) ? C::kT2 : C::kT1);
    if (c.col != dcol && p.causal_diag) {
      dcol = c.col;
      dpos = p.diag_pos[dcol];
    }
    // Of this half's 32 queries those before the key are masked in the diagonal block.
    const int lo = (c.x - c.begin == dpos) ? row - 64 * (c.rest % C::kHalves) - 32 * half : -(1 << 30);
    const float4* vec = reinterpret_cast<const float4*>(smem + C::kOffVec + (g % 3) * C::kVecB +
                                                        half * (kDiffVecHalf * 4));
    if (!wait_bar(C::kBarTF + (g & 1), (g / 2) & 1, kSiteSoftSFull)) break;
    uint32_t rs[2][32];  // S^T, then P^T, of each map
    tmem_ld_16x32bx2_x32<64>(t1, rs[0]);
    tmem_ld_16x32bx2_x32<64>(t1 + 32, rs[1]);
    tmem_ld_wait(rs[0]);
    tmem_ld_wait(rs[1]);
    warp_arrive(C::kBarDL);  // T2 may go over the second half
    // E1 = P_0^T - lam P_1^T, handed over on its own so that dV's product runs while dS^T is
    // formed.  The second map's P is kept with its weight -lam.
    {
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 l0 = vec[i >> 1], l1 = vec[8 + (i >> 1)], lm = vec[32 + (i >> 1)];
        auto two = [&](const float4& f) { return i & 1 ? f2_pack(f.z, f.w) : f2_pack(f.x, f.y); };
        const uint64_t y0 = f2_fma(pair_of(rs[0], i), c2, two(l0)), y1 = f2_fma(pair_of(rs[1], i), c2, two(l1));
        const uint64_t p1 = f2_mul(f2_pack(ex2_approx(f2_lo(y1)), ex2_approx(f2_hi(y1))), two(lm));
        const uint64_t p0 = f2_pack(ex2_approx(f2_lo(y0)), ex2_approx(f2_hi(y0)));
        rs[0][2 * i] = __float_as_uint(f2_lo(p0));
        rs[0][2 * i + 1] = __float_as_uint(f2_hi(p0));
        rs[1][2 * i] = __float_as_uint(f2_lo(p1));
        rs[1][2 * i + 1] = __float_as_uint(f2_hi(p1));
        const uint64_t w = f2_add(p0, p1);
        pk[i] = pack_bf16x2(f2_lo(w), f2_hi(w));
      }
      if (c.x - c.begin == dpos) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 32; ++i) rs[m][i] = i < lo ? 0u : rs[m][i];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint64_t w = f2_add(pair_of(rs[0], i), pair_of(rs[1], i));
          pk[i] = pack_bf16x2(f2_lo(w), f2_hi(w));
        }
      }
      tmem_st_16x32bx2_x16<16>(t1, pk);
    }
    tmem_st_wait();
    warp_arrive(C::kBarEF1 + (g & 1));
    if (!wait_bar(C::kBarDF + (g & 1), (g / 2) & 1, kSiteSoftSFull)) break;
    uint32_t rp[32];  // dP^T
    tmem_ld_16x32bx2_x32<32>(t1 + 64, rp);
    tmem_ld_wait(rp);
    {
      uint32_t pk[32];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 dd = vec[16 + 8 * m + (i >> 1)];
          const uint64_t t = f2_add(pair_of(rp, i), i & 1 ? f2_pack(dd.z, dd.w) : f2_pack(dd.x, dd.y));
          const uint64_t ds = f2_mul(pair_of(rs[m], i), t);
          pk[16 * m + i] = pack_bf16x2(f2_lo(ds), f2_hi(ds));
        }
      tmem_st_16x32bx2_x32<32>(t1 + 64, pk);
    }
    tmem_st_wait();
    warp_arrive(C::kBarEF + (g & 1));
    const bool whole = c.head && c.tail();
    if (c.last()) {
      // The piece is complete once its last step's products are.
      if (!wait_bar(C::kBarAD + (g & 1), (g / 2) & 1, kSiteSoftItemDone)) break;
      const int kv = c.col / p.nb, key = (c.col - kv * p.nb) * BLK + row;
      if (whole) {
        uint32_t pk[D / 4], pk2[D / 4];
        read_o<D>(tl + C::kAcc1, 1.f, pk);
        read_o<D>(tl + C::kAcc2, p.scale, pk2);
        warp_arrive(C::kBarAR);
        if (key < p.L) {
          const int64_t orow = static_cast<int64_t>(c.b * (p.cols / p.nb) + kv) * p.L + key;
          store_row_bf16<D>(static_cast<__nv_bfloat16*>(p.dv) + orow * D, 0, half, pk);
          store_row_bf16<D>(static_cast<__nv_bfloat16*>(p.dk) + orow * D, 0, half, pk2);
        }
      } else {
        // A cut column.  Its pieces lie in the CTAs root .. end; this warp's rows of them meet on
        // their own.  Who finds all others' pieces there adds them to what it holds; else it leaves
        // its own, and joins them if another has been as late.  The sum goes in the CTAs' order in
        // any case.
        const long long base = static_cast<long long>(c.b) * p.nnz;
        const int root = static_cast<int>(diff_div((base + c.begin) * c.per, p.share));
        const int end = static_cast<int>(diff_div((base + c.end) * c.per - 1, p.share));
        const int me = blockIdx.x;
        int* count = p.count + root * C::kEwWarps + gwarp;
        // A piece is laid out as its readers, the same warps elsewhere, take it: lanes side by side.
        auto piece = [&](int i, int g) {
          const int64_t slot = i == root ? 2 * static_cast<int64_t>(root) + 1 : 2 * static_cast<int64_t>(i);
          return reinterpret_cast<float4*>(p.parts) + slot * (BLK * 2 * D / 4) +
                 (gwarp * (D / 32) + g) * (8 * 32) + lane;
        };
        const int64_t orow = static_cast<int64_t>(c.b * (p.cols / p.nb) + kv) * p.L + key;
        // Columns 64 g + 32 half .. of dV | dK: the pieces' sum (own: this CTA's) to bf16.
        auto sum_pieces = [&](int g, const uint32_t* own) {
          float4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i = root; i <= end; ++i) {
            float4 y[8];
            if (own != nullptr && i == me) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                y[u] = make_float4(__uint_as_float(own[4 * u]), __uint_as_float(own[4 * u + 1]),
                                   __uint_as_float(own[4 * u + 2]), __uint_as_float(own[4 * u + 3]));
            } else {
              const float4* from = piece(i, g);
#pragma unroll
              for (int u = 0; u < 8; ++u) y[u] = __ldcg(from + 32 * u);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              x[u].x += y[u].x;
              x[u].y += y[u].y;
              x[u].z += y[u].z;
              x[u].w += y[u].w;
            }
          }
          if (key >= p.L) return;
          const bool is_k = g >= D / 64;
          const float f = is_k ? p.scale : 1.f;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_k ? p.dk : p.dv) + orow * D +
                               (is_k ? g - D / 64 : g) * 64 + half * 32;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            reinterpret_cast<uint4*>(out)[u] =
                make_uint4(pack_bf16x2(x[2 * u].x * f, x[2 * u].y * f), pack_bf16x2(x[2 * u].z * f, x[2 * u].w * f),
                           pack_bf16x2(x[2 * u + 1].x * f, x[2 * u + 1].y * f),
                           pack_bf16x2(x[2 * u + 1].z * f, x[2 * u + 1].w * f));
        };
        const bool late = warp_load_acquire(count, lane) == end - root;
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t r[32];
          load_o32(tl + C::kAcc1, i, r);
          tmem_ld_wait(r);
          if (i == D / 32 - 1) warp_arrive(C::kBarAR);
          if (late) {
            sum_pieces(i, r);
          } else {
            float4* to = piece(me, i);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              to[32 * u] = make_float4(__uint_as_float(r[4 * u]), __uint_as_float(r[4 * u + 1]),
                                       __uint_as_float(r[4 * u + 2]), __uint_as_float(r[4 * u + 3]));
          }
        }
        if (!late && warp_add_acq_rel(count, 1, lane) == end - root) {
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) sum_pieces(i, nullptr);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < C::kGroups; ++i)
      if (c.valid()) c.advance(p);
  }
  tmem_st_wait();
}

// ------------------------------------------------------------------- kernel

// a, b: the item tiles' tensors (dQ: q, dO; dK/dV: k, v), x, y the step tiles' (dQ: k, v;
// dK/dV: q, dO).
template <int BLK, int D, bool SPLIT, bool KV>
__global__ void __launch_bounds__(DiffBwdCfg<BLK, D, KV>::kThreads, 1)
    bsa_diff_bwd_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                        const DiffBwdParams p) {
  using C = DiffBwdCfg<BLK, D, KV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    auto bar = [&](int i) { return sbase + C::kOffBar + 8 * i; };
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), (i >= C::kBarEF1 && i < C::kBarEF + 2) || i == C::kBarAR || i == C::kBarDL
                            ? C::kStepWarps
                            : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) {
    wait_before();  // TMEM is not held across it (launch_after)
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if constexpr (SPLIT) {  // the column halves of Q that no copy writes
    const int bytes = KV ? C::kNX * C::kXTile : C::kItemTile;
    for (int i = threadIdx.x; i < bytes / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(smem + (KV ? C::kOffX : C::kOffA))[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns, p.expire_site};
  wait_before();
  if (warp == 0) {
    if (lane == 0) {
      if constexpr (KV) diff_kv_producer<BLK, D, SPLIT>(p, &tm_a, &tm_b, &tm_x, &tm_y, sbase, ctl);
      else diff_dq_producer<BLK, D, SPLIT>(p, &tm_a, &tm_b, &tm_x, &tm_y, sbase, ctl);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      if constexpr (KV) diff_kv_mma<BLK, D>(p, sbase, tmem, ctl);
      else diff_dq_mma<BLK, D>(p, sbase, tmem, ctl);
    }
  } else if (warp == C::kMma2Warp) {
    if constexpr (KV)
      if (!p.lam_rows) diff_sum_lam(p, lane);
    if (lane == 0) {
      if constexpr (KV) diff_kv_mma2<BLK, D>(p, sbase, tmem, ctl);
      else diff_dq_mma2<BLK, D>(p, sbase, tmem, ctl);
    }
  } else {
    if constexpr (KV) diff_kv_elementwise<BLK, D>(p, sbase, smem, tmem, ctl);
    else diff_dq_elementwise<BLK, D, SPLIT>(p, sbase, tmem, ctl);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int BLK, int D, bool SPLIT, bool KV>
cudaError_t launch_diff_bwd(const DiffBwdParams& p, const CUtensorMap& a, const CUtensorMap& b,
                            const CUtensorMap& x, const CUtensorMap& y, int grid, cudaStream_t stream) {
  using C = DiffBwdCfg<BLK, D, KV>;
  auto* kernel = bsa_diff_bwd_kernel<BLK, D, SPLIT, KV>;
  static int done[64] = {0};
  const cudaError_t e = set_smem_once(kernel, C::kLaunchSmem, done);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(grid), C::kThreads, C::kLaunchSmem, stream, a, b, x, y, p);
}

}  // namespace bsa
