// bsa_cache_decode.cuh -- attention over the paged 8-bit cache for few query rows: at most
// 8 * NT rows (queries of a tile times query heads of a kv head).
//
// Bound: memory.  A key costs 2 D bytes and 4 D R flops, R <= 16, so the kernel has to keep
// the loads in flight and spend few instructions a byte.
//   * Work is split evenly on the device (bsa_cache_sched.cuh); inside a CTA's segment the
//     warps take 16-key slices in turn, each with a running maximum and sum of its own,
//     joined when the segment ends.
//   * A lane copies exactly the bytes that its matrix fragments need (cp.async, 16 bytes at
//     a time, whole 32-byte sectors over the warp), into shared memory that only this lane
//     reads: no barriers, no bank conflicts, kStages - 1 slices in flight a warp.
//   * Products on mma.m16n8k16 (fp16 inputs, fp32 sums), transposed so that the keys (then
//     the head dim) fill the 16 rows and the few query rows the 8 columns: S^T = K Q^T and
//     O^T = V^T P^T.  The order of d inside S and of the columns of V is free, so both
//     fragments come from contiguous bytes: a lane's 16-byte piece of a key row gives it
//     four k-steps of K, and its 16-byte pieces of four value rows, interleaved by byte
//     permutes, give 8 row pairs of V^T.  The tensor pipe is nearly idle here; tcgen05
//     would need the operands converted into shared memory first, a second trip for every
//     byte.
//   * Stored numbers are exact in fp16.  bf16 queries are scaled per row by a power of two
//     into fp16's range (exact but for numbers 2^-28 of the row's largest).  The V scale
//     is folded into the exponent, w = exp2(s + log2 vs - m), so that weights are rounded
//     to fp16 relative to the largest weight times scale, and the sum takes w / vs: both
//     sums are held in fp32, with m the running maximum of s + log2 vs.
//   * The running maximum moves only when a score passes it by 2^8 (one vote a slice; the
//     weights stay below 256), so the usual slice needs no shuffles.
#pragma once

#include <type_traits>

#include "bsa_cache.cuh"
#include "bsa_cache_sched.cuh"
#include "bsa_ptx.cuh"

namespace bsa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// cap * log2(e) * tanh(z), from e^(2z): exact limits for large |z|.
__device__ __forceinline__ float softcap(float z, float cap_log2) {
  return cap_log2 * (1.f - __fdividef(2.f, 1.f + ex2_approx(z * (2.f * kLog2e))));
}

// log2 of a V scale inside the range that the exponents take (NaN and zero count as its
// lower end).
__device__ __forceinline__ float log2_scale(float s) {
  return fminf(fmaxf(lg2_approx(s), static_cast<float>(kScaleLogMin)),
               static_cast<float>(kScaleLogMax));
}

template <int D, int NT>
struct DecodeCfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = 2;               // per SM
  static constexpr int kStages = 3;
  static constexpr int kSL = 4;                 // log2 keys of a slice
  static constexpr int kVB = D / 8;             // bytes of a value row per lane
  static constexpr int kStageB = 2 * 16 * D;    // one warp's K and V slice
  static constexpr int kRingB = kWarps * kStages * kStageB;
  static constexpr int kJoinB = (kWarps / 2) * 32 * (D / 4) * 4;  // half the warps' O, one NT
  static constexpr int kOffJoin = kRingB;
  static constexpr int kOffSeg = kOffJoin + kJoinB;
  static constexpr int kOffScan = kOffSeg + 3 * 64;
  static constexpr int kSmemB = kOffScan + 192;
  static_assert(kWarps * kRows * 8 <= kJoinB, "row statistics share the join buffer");
  static_assert(sizeof(CacheSeg) <= 64, "segment slots");
  static_assert(kCtas * (kSmemB + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Waiting slices of a warp: where the slice's keys start and what scales them.
struct DecodeSlice {
  int key0;  // >= 0: loaded; -1: nothing of it is seen; -2: none was left to load
  float ks, lv;
};

template <class A, class C, int D, int NT>
__global__ void __launch_bounds__(DecodeCfg<D, NT>::kThreads, DecodeCfg<D, NT>::kCtas)
    bsa_cache_decode_kernel(const CacheFwdParams p, void* workspace) {
  using Cfg = DecodeCfg<D, NT>;
  constexpr int W = Cfg::kWarps, R = Cfg::kRows, S = Cfg::kStages, VB = Cfg::kVB;
  constexpr int KT = D / 64;  // 16-byte pieces of a key row per lane
  extern __shared__ __align__(16) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;  // fragment row and column of this lane
  CacheSeg* segs = reinterpret_cast<CacheSeg*>(smem + Cfg::kOffSeg);  // 3 slots of 64 bytes
  auto seg_at = [&](int i) -> CacheSeg& {
    return *reinterpret_cast<CacheSeg*>(reinterpret_cast<uint8_t*>(segs) + 64 * (i % 3));
  };
  const CacheParts parts = cache_parts(workspace, gridDim.x, R, D);
  if (blockIdx.x == 0 && tid == 0) *p.status = 0;

  int tq = R / p.group;
  if (p.row_ptr != nullptr) tq = 1 << (31 - __clz(tq));
  const CacheUnits<Cfg::kSL> units{p, tq};
  CacheWalk<Cfg::kSL>* walk_slot = reinterpret_cast<CacheWalk<Cfg::kSL>*>(smem + Cfg::kOffScan + 128);
  cache_split<Cfg::kSL, Cfg::kThreads>(units, W, reinterpret_cast<long long*>(smem + Cfg::kOffScan),
                                       walk_slot);
  CacheWalk<Cfg::kSL> walk;
  if (tid == 0) {
    walk = *walk_slot;
    walk.next(units, seg_at(0));
    if (seg_at(0).nq > 0) walk.next(units, seg_at(1));
    else seg_at(1).nq = 0;
    parts.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  __syncthreads();

  // ---- this warp's stream of slices: those of the current segment, then of the next one
  const uint32_t ring = smem_u32(smem) + warp * (S * Cfg::kStageB);
  int f_seg = 0, f_idx = 0, f_n = 0;  // segment being loaded, next slice of it, its slices
  int f_key0 = -1, f_pid = 0;         // this lane's slice of the current batch of 32
  float f_ks = 0.f, f_lv = 0.f;
  int stage_in = 0, stage_out = 0;
  auto count_of = [&](const CacheSeg& s) {
    return s.nq == 0 ? 0 : max(0, (s.s1 - s.s0 - warp + W - 1) / W);
  };
  f_n = count_of(seg_at(0));
  // Loads the next slice (limit: the last segment that may be begun) and says which it is.
  auto push = [&](int limit) -> DecodeSlice {
    DecodeSlice r{-2, 0.f, 0.f};
    while (f_idx >= f_n && f_seg < limit) {
      ++f_seg;
      f_idx = 0;
      f_n = count_of(seg_at(f_seg));
    }
    if (f_idx < f_n) {
      const CacheSeg& s = seg_at(f_seg);
      if ((f_idx & 31) == 0) {
        // The places of the next 32 slices, one a lane.
        const int i = s.s0 + warp + (f_idx + lane) * W;
        f_key0 = -1;
        if (i < s.s1) {
          const int last = s.pos0 + s.nq - 1;
          int key = i << Cfg::kSL;
          if (p.row_ptr != nullptr) {
            const int sub = p.block_shift - Cfg::kSL;
            key = (p.col_idx[s.rp + (i >> sub)] << p.block_shift) + ((i & ((1 << sub) - 1)) << Cfg::kSL);
          }
          if (key <= last && key + 15 >= s.lo_key) {
            f_pid = p.table[static_cast<int64_t>(s.b) * p.max_pages + (key >> p.page_shift)];
            if (f_pid >= 0 && f_pid < p.n_pages) {
              f_key0 = key;
              const int64_t tile = static_cast<int64_t>(f_pid) * p.Hkv + s.h;
              f_ks = p.k_scale[tile];
              f_lv = log2_scale(p.v_scale[tile]);
            }
          }
        }
      }
      const int src = f_idx & 31;
      r.key0 = __shfl_sync(0xffffffffu, f_key0, src);
      const int pid = __shfl_sync(0xffffffffu, f_pid, src);
      r.ks = __shfl_sync(0xffffffffu, f_ks, src);
      r.lv = __shfl_sync(0xffffffffu, f_lv, src);
      ++f_idx;
      if (r.key0 >= 0) {
        const int64_t base = (((static_cast<int64_t>(pid) * p.Hkv + s.h) << p.page_shift) +
                              (r.key0 & ((1 << p.page_shift) - 1))) * D;
        const uint32_t dst = ring + stage_in * Cfg::kStageB;
        const uint8_t* k = p.k_cache + base + g * D + t * 16;
#pragma unroll
        for (int i = 0; i < 2 * KT; ++i)  // key g, then key g + 8; pieces t and t + 4
          cp_async16(dst + i * 512 + lane * 16, k + (i / KT) * 8 * D + (i % KT) * 64);
        const uint8_t* v = p.v_cache + base + g * VB;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // keys 2t, 2t + 1, 2t + 8, 2t + 9
          const uint8_t* src_v = v + (2 * t + (i >> 1) * 8 + (i & 1)) * D;
          const uint32_t dst_v = dst + 16 * D + i * (32 * VB) + lane * VB;
          if constexpr (VB == 16) cp_async16(dst_v, src_v);
          else cp_async8(dst_v, src_v);
        }
        stage_in = stage_in + 1 == S ? 0 : stage_in + 1;
      }
    }
    cp_async_commit();
    return r;
  };
  DecodeSlice fifo[S - 1];
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fifo[i] = push(1);

  for (int si = 0;; ++si) {
    const CacheSeg s = seg_at(si);
    if (s.nq == 0) break;
    if (tid == 0) {  // read by the others after this segment's barriers
      if (seg_at(si + 1).nq > 0) walk.next(units, seg_at(si + 2));
      else seg_at(si + 2).nq = 0;
    }
    const int mine = count_of(s);
    if (f_seg < si) {  // a warp without slices in the last segment
      f_seg = si;
      f_idx = 0;
      f_n = mine;
    }
    const int last = s.pos0 + s.nq - 1;
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
    }
    if (mine > 0) {
      // Q fragments: row 8n + g, the columns of this lane's pieces of a key row.
      uint32_t qf[NT][KT][8];
      float rf[NT][2];      // factor of the scores of rows 8n + 2t, 8n + 2t + 1
      int hi[NT][2];        // their positions (-1: no such row)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g;
        const bool live = row < s.nq * p.group;
        const int qi = row / p.group;
        float top = 0.f;
        if (live) {
          const A* q = static_cast<const A*>(p.q) + (s.q0 + qi) * p.q_token_stride +
                       (s.h * p.group + row - qi * p.group) * p.q_head_stride + t * 16;
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const uint4 a = *reinterpret_cast<const uint4*>(q + c * 64);
            const uint4 b = *reinterpret_cast<const uint4*>(q + c * 64 + 8);
            qf[n][c][0] = a.x; qf[n][c][1] = a.y; qf[n][c][2] = a.z; qf[n][c][3] = a.w;
            qf[n][c][4] = b.x; qf[n][c][5] = b.y; qf[n][c][6] = b.z; qf[n][c][7] = b.w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < KT; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) qf[n][c][i] = 0;
        }
        float back = 1.f;
        if constexpr (sizeof(A) == 2 && !std::is_same<A, __half>::value) {
          // bf16: largest magnitude of the row to [2^14, 2^15), then fp16.
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
          hi[n][e] = r < s.nq * p.group ? s.pos0 + r / p.group : -1;
        }
      }
      for (int done = 0; done < mine;) {
        const DecodeSlice cur = fifo[0];
#pragma unroll
        for (int i = 0; i < S - 2; ++i) fifo[i] = fifo[i + 1];
        cp_async_wait<S - 2>();
        // The slice's fragments; then its stage is free for the slice after the next.
        uint4 kw[2 * KT];
        uint32_t vw[4][VB / 4];
        if (cur.key0 >= 0) {
          const uint8_t* src = smem + warp * (S * Cfg::kStageB) + stage_out * Cfg::kStageB;
#pragma unroll
          for (int i = 0; i < 2 * KT; ++i)
            kw[i] = *reinterpret_cast<const uint4*>(src + i * 512 + lane * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* sv = src + 16 * D + i * (32 * VB) + lane * VB;
            if constexpr (VB == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(sv);
              vw[i][0] = x.x; vw[i][1] = x.y; vw[i][2] = x.z; vw[i][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(sv);
              vw[i][0] = x.x; vw[i][1] = x.y;
            }
          }
          stage_out = stage_out + 1 == S ? 0 : stage_out + 1;
        }
        fifo[S - 2] = push(si + 1);
        if (cur.key0 == -2) continue;  // nothing was left to load when this place was filled
        ++done;
        if (cur.key0 < 0) continue;

        // S^T: keys g and g + 8 (rows) by query rows 2t, 2t + 1 (columns).
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KT; ++c) {
          const uint32_t wa[4] = {kw[c].x, kw[c].y, kw[c].z, kw[c].w};
          const uint32_t wb[4] = {kw[KT + c].x, kw[KT + c].y, kw[KT + c].z, kw[KT + c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            stored4_to_half2<C>(wa[i], a0, a2);
            stored4_to_half2<C>(wb[i], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(x[n], a0, a1, a2, a3, qf[n][c][2 * i], qf[n][c][2 * i + 1]);
          }
        }
        const bool whole = cur.key0 + 15 <= s.pos0 &&
                           (p.window < 0 || cur.key0 >= last - p.window);
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = x[n][e] * (rf[n][e & 1] * cur.ks);
            if (p.softcap_log2 > 0.f) y = softcap(y, p.softcap_log2);
            y += cur.lv;
            if (!whole) {
              const int key = cur.key0 + g + (e >> 1) * 8, top = hi[n][e & 1];
              if (key > top || (p.window >= 0 && key < top - p.window)) y = -INFINITY;
            }
            x[n][e] = y;
            grow |= y > m[n][e & 1] + 8.f;
          }
        }
        if (!whole) {
          // Values that no row sees may be anything, a NaN among it: zero.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = cur.key0 + 2 * t + (i >> 1) * 8 + (i & 1);
            if (key > last || key < s.lo_key)
#pragma unroll
              for (int w = 0; w < VB / 4; ++w) vw[i][w] = 0;
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(x[n][e], x[n][e + 2]);
#pragma unroll
              for (int k = 4; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
              top = fmaxf(top, m[n][e]);
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
        const float rv = ex2_approx(-cur.lv);
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float top = m[n][e & 1];
            x[n][e] = ex2_approx(x[n][e] - (top == -INFINITY ? 0.f : top));
          }
          l[n][0] = fmaf(x[n][0] + x[n][2], rv, l[n][0]);
          l[n][1] = fmaf(x[n][1] + x[n][3], rv, l[n][1]);
          pf[n][0] = transpose8x8(float2_to_act<__half>(x[n][0], x[n][1]));
          pf[n][1] = transpose8x8(float2_to_act<__half>(x[n][2], x[n][3]));
        }
        // O^T: columns VB * g + 2j, 2j + 1 of the values (rows) by the query rows.
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
          const uint32_t w01 = __byte_perm(vw[0][j / 2], vw[1][j / 2], sel);
          const uint32_t w23 = __byte_perm(vw[2][j / 2], vw[3][j / 2], sel);
          uint32_t a0, a1, a2, a3;
          stored4_to_half2<C>(w01, a0, a1);
          stored4_to_half2<C>(w23, a2, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(o[n][j], a0, a1, a2, a3, pf[n][0], pf[n][1]);
        }
      }
    }

    // ---- join the warps: row statistics, then the scaled accumulators, halves onto halves
    float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffJoin);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int k = 4; k < 32; k *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
        if (g == 0) ml[warp * R + 8 * n + 2 * t + e] = make_float2(m[n][e], l[n][e]);
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * R + 8 * n + 2 * t + e].x);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 x = ml[w * R + 8 * n + 2 * t + e];
          sum += x.y * (x.x == -INFINITY ? 0.f : ex2_approx(x.x - top));  // a NaN stays
        }
        const float f = m[n][e] == -INFINITY ? 0.f : ex2_approx(m[n][e] - top);
        m[n][e] = top;
        l[n][e] = sum;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[n][j][e] *= f;
          o[n][j][e + 2] *= f;
        }
      }
    float4* join = reinterpret_cast<float4*>(smem + Cfg::kOffJoin);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int half = W / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (warp >= half && warp < 2 * half) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            join[((warp - half) * (D / 16) + j) * 32 + lane] =
                make_float4(o[n][j][0], o[n][j][1], o[n][j][2], o[n][j][3]);
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const float4 x = join[(warp * (D / 16) + j) * 32 + lane];
            o[n][j][0] += x.x;
            o[n][j][1] += x.y;
            o[n][j][2] += x.z;
            o[n][j][3] += x.w;
          }
        }
      }
    // ---- warp 0 has the segment's sums: final rows, or a partial result of a cut unit
    if (warp == 0) {
      const bool whole_unit = s.starts && s.ends;
      const int slot = 2 * blockIdx.x + (s.starts ? 1 : 0);
      if (lane == 0 && s.starts && !s.ends)
        parts.meta[blockIdx.x] = make_int4(s.more, s.q0, s.nq, s.h);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e;
          if (r >= s.nq * p.group) continue;
          if (whole_unit) {
            const int qi = r / p.group, head = s.h * p.group + r - qi * p.group;
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
            float4* dst = reinterpret_cast<float4*>(parts.o + (static_cast<int64_t>(slot) * R + r) * D + g * VB);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              dst[i] = make_float4(o[n][2 * i][e], o[n][2 * i][e + 2], o[n][2 * i + 1][e],
                                   o[n][2 * i + 1][e + 2]);
            if (g == 0) parts.ml[static_cast<int64_t>(slot) * R + r] = make_float2(m[n][e], l[n][e]);
          }
        }
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

// Joins the pieces of the unit that was cut at the end of CTA blockIdx.x's share: one warp
// a row.  Launched with every call and early (programmatic dependent launch): it waits for
// the attention kernel's results on the device, and its CTAs leave at once where nothing
// was cut.
template <class A, int D, int R>
__global__ void __launch_bounds__(128) bsa_cache_join_kernel(const CacheFwdParams p, void* workspace) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheParts parts = cache_parts(workspace, gridDim.x, R, D);
  const int4 unit = parts.meta[blockIdx.x];  // pieces that follow, q0, nq, h
  const int r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit.x == 0 || r >= unit.z * p.group) return;
  // Piece 0 ends this CTA's share, piece i begins that of CTA blockIdx.x + i.
  auto slot = [&](int i) {
    return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * R + r;
  };
  const int qi = r / p.group, head = unit.w * p.group + r - qi * p.group;
  const float sink = p.sinks != nullptr ? p.sinks[head] * kLog2e : -INFINITY;
  float top = sink;
  for (int i = lane; i <= unit.x; i += 32) top = fmaxf(top, parts.ml[slot(i)].x);
#pragma unroll
  for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  float z = sink == -INFINITY ? 0.f : ex2_approx(sink - top), o[E] = {};
#pragma unroll 4
  for (int i = 0; i <= unit.x; ++i) {
    const int64_t s = slot(i);
    const float2 x = parts.ml[s];
    const float f = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
    const float* src = parts.o + s * D + lane * E;
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      o[0] += f * v.x;
      o[1] += f * v.y;
      o[2] += f * v.z;
      o[3] += f * v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      o[0] += f * v.x;
      o[1] += f * v.y;
    }
    z += f * x.y;
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  const int64_t row = static_cast<int64_t>(unit.y + qi) * p.Hq + head;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<A*>(p.out) + row * D + lane * E);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dst[i] = float2_to_act<A>(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (lane == 0) p.lse[row] = z == 0.f ? -INFINITY : (top + log2f(z)) * kLn2;
}

template <class A, class C, int D, int NT>
cudaError_t launch_decode(const CacheFwdParams& p, void* workspace, int sms, cudaStream_t stream) {
  using Cfg = DecodeCfg<D, NT>;
  auto* kernel = bsa_cache_decode_kernel<A, C, D, NT>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemB);
  if (e != cudaSuccess) return e;
  const int grid = Cfg::kCtas * sms;
  kernel<<<grid, Cfg::kThreads, Cfg::kSmemB, stream>>>(p, workspace);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, Cfg::kRows / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bsa_cache_join_kernel<A, D, Cfg::kRows>, p, workspace);
}

template <class C, int D>
cudaError_t launch_decode(bool fp16, int rows, const CacheFwdParams& p, void* workspace, int sms,
                          cudaStream_t stream) {
  if (fp16)
    return rows <= 8 ? launch_decode<__half, C, D, 1>(p, workspace, sms, stream)
                     : launch_decode<__half, C, D, 2>(p, workspace, sms, stream);
  return rows <= 8 ? launch_decode<__nv_bfloat16, C, D, 1>(p, workspace, sms, stream)
                   : launch_decode<__nv_bfloat16, C, D, 2>(p, workspace, sms, stream);
}

}  // namespace bsa
