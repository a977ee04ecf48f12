// bsa_rotary.cu -- rotary positions with several axes: every pair of numbers of a head is turned
// by (position on the pair's axis) x (the pair's frequency).  See include/bsa.h.
//
// Bound: memory, each number read and written once.
//   * The angle: the table holds frequencies in turns per position as 64-bit binary fractions, each
//     within 2^-64 turns, and the 64-bit product with an integer position, which wraps at whole
//     turns, adds nothing to that: at position 2^31 it is within 2^-33 turns of the angle.  Its top
//     32 bits are rounded to fp32 for sincospif, by 2^-25 half-turns at most: 1e-7 radians in all.  (An fp32 product would be off by 2^-24 of the angle: at position 2^20 all of a
//     radian's fourth digit.)
//   * A thread keeps one token and one piece of its row (8 numbers, or 8 and their partners) and
//     walks the heads of q and k with it, so that sines and cosines stay in registers: 8 of them
//     for all heads.  Few tokens: the heads are split over threads and CTAs, which then each
//     work them out.
//   * Loads of kRows heads are in flight at once (2, 6 and 8 of them measured the same or worse),
//     all reads and writes streaming, since no number is used twice (59 -> 58 us, 110 -> 109).
// Measured: 32 + 8 heads of 128, 16,384 tokens 58 us, 5.8 TB/s (0.85 of a copy); 2 x 20,280 tokens
// of 16 + 16 heads, adjacent pairs on three axes, 109 us, 6.1 TB/s; 64 packed tokens 3.8 us, the
// launch and two dependent loads (a call takes the host four times that).
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bsa_cache.cuh"
#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;

// N 16-bit numbers, read or written at once.
template <int N>
struct Piece;
template <>
struct Piece<8> {
  using T = uint4;
};
template <>
struct Piece<4> {
  using T = uint2;
};
template <>
struct Piece<2> {
  using T = uint32_t;
};
template <>
struct Piece<1> {
  using T = unsigned short;
};

template <class A>
__device__ __forceinline__ float to_float(uint16_t x);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint16_t x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
template <>
__device__ __forceinline__ float to_float<__half>(uint16_t x) {
  return __half2float(__ushort_as_half(x));
}
template <class A>
__device__ __forceinline__ uint16_t from_float(float x) {
  return static_cast<uint16_t>(float2_to_act<A>(x, 0.f));
}

// HALF: numbers i and i + pairs are a pair; a thread has N of the first and their partners.  Else
// numbers 2i and 2i + 1 are, and a thread has N = 8 numbers.  Pieces behind the last pair are
// copied.
template <class A, bool HALF, int N>
__global__ void __launch_bounds__(kThreads, 3) bsa_rotary_kernel(const RotaryParams p) {
  using T = typename Piece<N>::T;
  constexpr int P = HALF ? N : N / 2;  // pairs of a thread
  const int v = threadIdx.x % p.pieces, row = threadIdx.x / p.pieces;
  const int tok = row & (p.tokens - 1), hsub = row >> p.token_shift;
  const int b = blockIdx.x / p.tiles;
  const int t = (blockIdx.x - b * p.tiles) * p.tokens + tok;
  if (hsub >= p.hsubs || t >= p.L) return;
  // Of the pair's first numbers, this piece's; behind them, the numbers that stay.
  const int rotating = HALF ? p.pairs / N : (2 * p.pairs + N - 1) / N;
  const bool turns = v < rotating;
  const int x0 = (HALF && !turns) ? 2 * p.pairs + (v - rotating) * N : v * N;
  float c[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int pair = HALF ? x0 + i : v * P + i;
    c[i] = 1.f;
    s[i] = 0.f;
    if (turns && pair < p.pairs) {
      const bsa_rotary_pair e = p.table[pair];
      // An axis that the call has no positions of turns nothing.
      const bool on = static_cast<unsigned>(e.axis) < static_cast<unsigned>(p.axes);
      const int32_t pos = on ? p.positions[e.axis * p.pos_axis + b * p.pos_batch + t] : 0;
      const uint64_t angle = e.turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
      sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s[i], &c[i]);
      if (p.inverse) s[i] = -s[i];
    }
  }
  const int step = p.hsubs * gridDim.y;
#pragma unroll 1
  for (int h0 = blockIdx.y * p.hsubs + hsub; h0 < p.heads; h0 += kRows * step) {
    T a[kRows], z[kRows];
    uint16_t* to[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int h = h0 + j * step;
      to[j] = nullptr;
      if (h >= p.heads) continue;
      const RotarySide& side = p.side[h >= p.side[0].heads];
      const int64_t hh = h >= p.side[0].heads ? h - p.side[0].heads : h;
      const uint16_t* from = static_cast<const uint16_t*>(side.in) + b * side.in_batch + hh * side.in_head +
                             t * side.in_token + x0;
      to[j] = static_cast<uint16_t*>(side.out) + b * side.out_batch + hh * side.out_head + t * side.out_token + x0;
      a[j] = __ldcs(reinterpret_cast<const T*>(from));
      if (HALF && turns) z[j] = __ldcs(reinterpret_cast<const T*>(from + p.pairs));
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (to[j] == nullptr) continue;
      uint16_t* x = reinterpret_cast<uint16_t*>(&a[j]);
      if (HALF) {
        uint16_t* y = reinterpret_cast<uint16_t*>(&z[j]);
        if (turns) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float f = to_float<A>(x[i]), g = to_float<A>(y[i]);
            x[i] = from_float<A>(fmaf(f, c[i], -g * s[i]));
            y[i] = from_float<A>(fmaf(f, s[i], g * c[i]));
          }
          __stcs(reinterpret_cast<T*>(to[j] + p.pairs), z[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (v * P + i >= p.pairs) continue;  // stays, bit for bit
          const float f = to_float<A>(x[2 * i]), g = to_float<A>(x[2 * i + 1]);
          x[2 * i] = from_float<A>(fmaf(f, c[i], -g * s[i]));
          x[2 * i + 1] = from_float<A>(fmaf(f, s[i], g * c[i]));
        }
      }
      __stcs(reinterpret_cast<T*>(to[j]), a[j]);
    }
  }
}

template <class A>
void launch_as(const RotaryParams& p, int n, dim3 grid, cudaStream_t stream) {
  if (!p.half) bsa_rotary_kernel<A, false, 8><<<grid, kThreads, 0, stream>>>(p);
  else if (n == 8) bsa_rotary_kernel<A, true, 8><<<grid, kThreads, 0, stream>>>(p);
  else if (n == 4) bsa_rotary_kernel<A, true, 4><<<grid, kThreads, 0, stream>>>(p);
  else if (n == 2) bsa_rotary_kernel<A, true, 2><<<grid, kThreads, 0, stream>>>(p);
  else bsa_rotary_kernel<A, true, 1><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, bool fp16, int sms, cudaStream_t stream) {
  // Numbers of a piece: eight, or (halves) what divides the pairs.
  int n = 8;
  while (p.half && p.pairs % n != 0) n /= 2;
  bool in_place = true;  // then the numbers behind the pairs need no copy
  for (const RotarySide& s : p.side)
    in_place = in_place && (s.heads == 0 || s.in == s.out);
  const int rest = in_place ? 0 : p.d - 2 * p.pairs;
  p.pieces = p.half ? p.pairs / n + rest / n : (2 * p.pairs + rest + 7) / 8;
  // Rows (token, head) of a CTA: a power of two.
  int rows_shift = 0;
  while ((p.pieces << (rows_shift + 1)) <= kThreads) ++rows_shift;
  p.heads = p.side[0].heads + p.side[1].heads;
  // Tokens of a CTA: all its rows, unless that leaves SMs without one; then heads take their place.
  auto tiles = [&](int shift) { return (static_cast<int64_t>(p.L) + (1 << shift) - 1) >> shift; };
  p.token_shift = rows_shift;
  while (p.token_shift > 0 && p.B * tiles(p.token_shift) < sms) --p.token_shift;
  p.tokens = 1 << p.token_shift;
  p.tiles = static_cast<int>(tiles(p.token_shift));
  p.hsubs = 1 << (rows_shift - p.token_shift);
  const int64_t x = static_cast<int64_t>(p.B) * p.tiles;
  if (x > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // Heads split over CTAs until there are about eight for each SM (all that fit).
  const int most = (p.heads + p.hsubs - 1) / p.hsubs;
  int y = 1;
  while (y * 2 <= most && y < 32768 && x * y < 8ll * sms) y *= 2;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  if (fp16) launch_as<__half>(p, n, grid, stream);
  else launch_as<__nv_bfloat16>(p, n, grid, stream);
  return cudaGetLastError();
}

}  // namespace bsa

namespace {

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace

extern "C" {

int bsa_rotary_table(const double* inv_freq, const int32_t* axis, int pairs, bsa_rotary_pair* table) {
  if (inv_freq == nullptr || table == nullptr) return BSA_ERR_NULL;
  if (pairs < 1 || pairs > 128) return BSA_ERR_SHAPE;
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1e6) return BSA_ERR_UNSUPPORTED;
    if (axis != nullptr && (axis[i] < 0 || axis[i] > 7)) return BSA_ERR_SHAPE;
  }
  // 2 pi to 2^-106 of its size, as a sum of two doubles.
  constexpr double kTwoPi = 6.283185307179586, kTwoPiLow = 2.4492935982947064e-16;
  for (int i = 0; i < pairs; ++i) {
    // Turns per position as a 64-bit fraction, which wraps at whole turns.  The quotient comes in two
    // doubles too, the second from the remainder that a fused multiply-add leaves exact (Dekker): one
    // alone is off by 2^-54 of up to 160,000 turns, which 2^31 positions make 0.1 radians.  The first
    // one's part behind whole turns, in [-1/2, 1/2], is exact; 2^64 takes 1/2 no more (-1/2 is the same).
    const double turns = inv_freq[i] / kTwoPi;
    const double more = std::fma(-turns, kTwoPiLow, std::fma(-turns, kTwoPi, inv_freq[i])) / kTwoPi;
    double f = turns - std::nearbyint(turns);
    if (f >= 0.5) f -= 1.0;
    table[i].turns = static_cast<uint64_t>(std::llrint(std::ldexp(f, 64))) +
                     static_cast<uint64_t>(std::llrint(std::ldexp(more, 64)));
    table[i].axis = axis == nullptr ? 0 : axis[i];
    table[i].reserved = 0;
  }
  return BSA_OK;
}

int bsa_rotary(const bsa_rotary_args* a, void* stream) {
  if (a == nullptr) return BSA_ERR_NULL;
  if (a->dtype != BSA_BF16 && a->dtype != BSA_FP16) return BSA_ERR_DTYPE;
  if (a->B < 0 || a->L < 0 || a->L > bsa::kMaxPositions || a->d < 8 || a->d > 256 || a->d % 8 != 0 ||
      a->pairs < 1 || 2 * a->pairs > a->d || a->axes < 1 || a->axes > 8 || a->q.heads < 0 || a->k.heads < 0 ||
      a->q.heads > 65535 || a->k.heads > 65535)
    return BSA_ERR_SHAPE;
  if (a->pairing != BSA_ROTARY_HALF && a->pairing != BSA_ROTARY_ADJACENT) return BSA_ERR_UNSUPPORTED;
  if (a->B == 0 || a->L == 0 || a->q.heads + a->k.heads == 0) return BSA_OK;
  if (a->positions == nullptr || a->table == nullptr) return BSA_ERR_NULL;
  if (!aligned(a->positions, 4) || !aligned(a->table, 16)) return BSA_ERR_ALIGN;
  bsa::RotaryParams p{};
  const bsa_rotary_side* in[2] = {&a->q, &a->k};
  for (int i = 0; i < 2; ++i) {
    const bsa_rotary_side& s = *in[i];
    if (s.heads == 0) continue;
    if (s.in == nullptr || s.out == nullptr) return BSA_ERR_NULL;
    if (!aligned(s.in, 16) || !aligned(s.out, 16)) return BSA_ERR_ALIGN;
    for (int64_t n : {s.in_batch, s.in_head, s.in_token, s.out_batch, s.out_head, s.out_token})
      if (n % 8 != 0) return BSA_ERR_ALIGN;
    // Of the dimensions that have more than one place: in place with other strides, and rows that share a
    // place, which several threads would write.
    const bool many[3] = {a->B > 1, s.heads > 1, a->L > 1};
    const int64_t from[3] = {s.in_batch, s.in_head, s.in_token}, to[3] = {s.out_batch, s.out_head, s.out_token};
    for (int j = 0; j < 3; ++j)
      if (many[j] && (to[j] == 0 || (s.in == s.out && from[j] != to[j]))) return BSA_ERR_UNSUPPORTED;
    p.side[i] = {s.in, s.out, s.heads, s.in_batch, s.in_head, s.in_token, s.out_batch, s.out_head, s.out_token};
  }
  // One side's output over the other side's tensors: turned twice, or read after it was turned.
  if (a->q.heads > 0 && a->k.heads > 0 &&
      (a->q.out == a->k.out || a->q.out == a->k.in || a->k.out == a->q.in))
    return BSA_ERR_UNSUPPORTED;
  p.positions = a->positions;
  p.table = a->table;
  p.pos_axis = a->pos_axis;
  p.pos_batch = a->pos_batch;
  p.B = a->B;
  p.L = a->L;
  p.d = a->d;
  p.pairs = a->pairs;
  p.axes = a->axes;
  p.half = a->pairing == BSA_ROTARY_HALF;
  p.inverse = a->inverse != 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  const int sms = bsa::sm_count(dev);
  if (sms <= 0) return BSA_ERR_CUDA;
  return bsa::launch_rotary(p, a->dtype == BSA_FP16, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BSA_OK
             : BSA_ERR_CUDA;
}

}  // extern "C"
