// Numbers in 8 bits with a scale: signed integers up to 127, or e4m3 (four significant bits, up to 448).
//
// Values x_j of a row share scale = max(max |x_j| / most, 2^-126), a quotient of fp32; the code of x is the number of the
// format that is nearest to x / scale, ties to the even one.  That is the exact quotient's nearest, not a rounded
// quotient's: codes are the same wherever they are computed from the same values.  The quotient is first taken by the
// scale's reciprocal (at most three fp32 roundings, within 2^-22 of itself), and where that leaves the border between two
// codes within reach, which is one value in some 10^4, by fp32's exact remainder or in fp64 (in fp64 throughout: 69 us against
// 63 for 8192 rows of 4096 channels behind the norm).
// A row that holds an infinity or a NaN has codes 0 and a NaN for scale: it reads back as NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/flashbev.h"

namespace fbev {

constexpr float kLeastScale = 0x1p-126f;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

template <int KIND>
struct Codes {
  static constexpr bool kFloat = KIND == FBEV_CODES_E4M3;
  static constexpr float kMost = kFloat ? 448.0f : 127.0f;

  // From the largest abs_bits() of a row (NaN and infinity are the largest of all).  The quotient is the correctly rounded
  // one: a product with the rounded reciprocal, corrected by its exact remainder (Markstein).
  static __device__ __forceinline__ float scale_of(uint32_t top) {
    constexpr float kInverse = 1.0f / kMost;
    const float x = __builtin_bit_cast(float, top), q = x * kInverse;
    const float scale = fmaxf(fmaf(fmaf(-q, kMost, x), kInverse, q), kLeastScale);
    return top >= 0x7f800000u ? __builtin_nanf("") : scale;
  }
  // 1 / scale to a step of fp32: all that pack() asks for.
  static __device__ __forceinline__ float inverse_of(float scale) { return __builtin_amdgcn_rcpf(scale); }

  // A number on the same side of every border as the exact x / scale: the quotient rounded to fp32, moved off itself by one
  // step towards the exact one where it is even (borders are even in fp32, so an odd one lies on none).  Where
  // x is of fp32 its quotient is on a border or at least 2^-33 of itself away: fp64 tells.
  static __device__ __forceinline__ float side_of(double x, double scale) {
    const double exact = x / scale;
    const float q = (float)exact;
    const double rest = exact - (double)q;
    uint32_t b = __builtin_bit_cast(uint32_t, q);
    if (rest != 0.0 && (b & 1) == 0 && (b << 1) != 0) b += ((rest > 0.0) == (q > 0.0f)) ? 1u : ~0u;
    return __builtin_bit_cast(float, b);
  }

  // Four values' codes, one to a byte.  inverse: inverse_of(scale).
  static __device__ __forceinline__ uint32_t pack(const float (&x)[4], float scale, float inverse) {
    return pack(x, scale, inverse, [&](int i) { return x[i]; });
  }
  // The same where x[i], the scale and its inverse are rounded (quotients then are within 2^-21 of themselves): exact(i) and
  // scale are the i-th value and the scale in fp64.
  template <typename F, typename S>
  static __device__ __forceinline__ uint32_t pack(const float (&x)[4], S scale, float inverse, F exact) {
    constexpr bool kWide = sizeof(S) == 8;
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = x[i] * inverse;
    if constexpr (kFloat) {
      // what four significant bits drop lies around the half; under 2^-6 codes are a fixed 2^-9 apart: all of those but 0
      uint32_t half = ~0u, small = ~0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, q[i]);
        half = min(half, (b << 12) + 0x80010000u);
        small = min(small, (b << 1) - 2u);
      }
      if (half <= 0x20000u || small < 0x79000000u - 2u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = side_of(exact(i), scale);
      }
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    } else {
      // 1.5 2^23 + q keeps q's nearest integer in its last byte
      constexpr float kTurn = 12582912.0f;
      uint32_t t[4];
      float off = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float n = q[i] + kTurn;
        off = fmaxf(off, fabsf(q[i] - (n - kTurn)));
        t[i] = __builtin_bit_cast(uint32_t, n);
      }
      if (off > (kWide ? 0.4999f : 0.49996f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kWide) {
            t[i] = __builtin_bit_cast(uint32_t, side_of(exact(i), scale) + kTurn);
          } else {
            // the rest that the nearest integer n leaves of x is exact in fp32, and n off by one at most
            const float n = __builtin_bit_cast(float, t[i]) - kTurn, rest = fmaf(-n, scale, x[i]);
            const float over = fabsf(rest) - 0.5f * scale;
            const bool move = over > 0.0f || (over == 0.0f && (t[i] & 1) != 0);
            t[i] += !move ? 0u : rest > 0.0f ? 1u : ~0u;
          }
        }
      }
      const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(t[3], t[2], 0x0c0c0400u);
      return hi << 16 | lo;
    }
  }

  // The numbers that a word's four codes stand for.
  static __device__ __forceinline__ void unpack(uint32_t w, float (&x)[4]) {
    if constexpr (kFloat) {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
      x[0] = a[0];
      x[1] = a[1];
      x[2] = b[0];
      x[3] = b[1];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    }
  }
};

}  // namespace fbev
