// bsa_cache.cuh -- element types of the paged 8-bit key/value cache: conversions between
// its stored numbers (e4m3 or int8) and the 16-bit activations (bf16 or fp16).
//
// Every stored number is exact in fp16 (e4m3: 4 significant bits, 2^-9 .. 448; int8:
// integers up to 128), so the products run on fp16 copies of it.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bsa {

// Scales are powers of two in [2^kScaleLogMin, 2^kScaleLogMax].
constexpr int kScaleLogMin = -60;
constexpr int kScaleLogMax = 60;

struct E4M3 {
  static constexpr bool kInt8 = false;
};
struct Int8 {
  static constexpr bool kInt8 = true;
};

// Two stored numbers (the low 16 bits, first one lowest) as an fp16 pair.
template <class C>
__device__ __forceinline__ uint32_t stored_to_half2(uint32_t pair) {
  if constexpr (C::kInt8) {
    // 0x6400 + u is fp16 1024 + u for a byte u; u = x + 128 gives x after subtracting 1152.
    const uint32_t u = __byte_perm((pair ^ 0x8080u) & 0xFFFFu, 0x64006400u, 0x5150);
    const half2 r = __hsub2(*reinterpret_cast<const half2*>(&u), __float2half2_rn(1152.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(pair)));
    return r;
  }
}

// Two fp32 values rounded to stored numbers (nearest, ties to even, saturating); a NaN
// stays a NaN in e4m3 and becomes 0 in int8.
template <class C>
__device__ __forceinline__ uint32_t float2_to_stored(float lo, float hi) {
  if constexpr (C::kInt8) {
    const int a = __float2int_rn(fminf(fmaxf(lo != lo ? 0.f : lo, -127.f), 127.f));
    const int b = __float2int_rn(fminf(fmaxf(hi != hi ? 0.f : hi, -127.f), 127.f));
    return (static_cast<uint32_t>(a) & 0xFFu) | ((static_cast<uint32_t>(b) & 0xFFu) << 8);
  } else {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
}

template <class C>
__device__ __forceinline__ float2 stored_to_float2(uint32_t pair) {
  const uint32_t h = stored_to_half2<C>(pair);
  return __half22float2(*reinterpret_cast<const half2*>(&h));
}

// The smallest power of two s in the scales' range with amax <= qmax * s, qmax the largest
// stored number (448 = 1.75 * 2^8, 127 = 1.984375 * 2^6): with amax = m * 2^e, 1 <= m < 2,
// s = 2^(e - 8) or 2^(e - 7) as m <= 1.75 or not, and likewise for int8.
//
// A power of two makes the division by s exact, so a stored number is the input rounded
// once; and when a page's scale grows by 2^k, an e4m3 number only loses what falls below
// its smallest step, an int8 one at most half a step each time and (1/2 + 1/4 + ...) in
// all, where free scales would round every kept token again at every append.
template <class C>
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);  // amax >= 0 and finite
  const int e = static_cast<int>(u >> 23) - 127;
  const uint32_t frac = u & 0x7FFFFFu;
  constexpr uint32_t kFrac = C::kInt8 ? 0x7E0000u : 0x600000u;  // m - 1 of qmax
  constexpr int kExp = C::kInt8 ? 6 : 8;
  int k = e - kExp + (frac > kFrac ? 1 : 0);
  k = max(kScaleLogMin, min(kScaleLogMax, k));
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Activations.
template <class T>
__device__ __forceinline__ float2 act_to_float2(uint32_t pair);
template <>
__device__ __forceinline__ float2 act_to_float2<__nv_bfloat16>(uint32_t pair) {
  return make_float2(__uint_as_float(pair << 16), __uint_as_float(pair & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 act_to_float2<__half>(uint32_t pair) {
  return __half22float2(*reinterpret_cast<const half2*>(&pair));
}

template <class T>
__device__ __forceinline__ uint32_t float2_to_act(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t float2_to_act<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t float2_to_act<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace bsa
