// Numbers in 8 bits with a scale: signed integers up to 127, or e4m3 (four significant bits, up to 448).
//
// Values x_j of a row share scale = max(max |x_j| / most, 2^-126), a quotient of fp32; the code of x is the number of the
// format that is nearest to x / scale, ties to the even one.  That is the exact quotient's nearest, not a rounded
// quotient's: codes are the same wherever they are computed from the same values.  The quotient is first taken by the
// scale's reciprocal (at most three fp32 roundings, within 2^-22 of itself), and where that leaves the border between two
// codes within reach, which is one value in some 10^4, in fp64.
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

  // From the largest abs_bits() of a row (NaN and infinity are the largest of all).
  static __device__ __forceinline__ float scale_of(uint32_t top) {
    if (top >= 0x7f800000u) return __builtin_nanf("");
    return fmaxf(__builtin_bit_cast(float, top) / kMost, kLeastScale);
  }

  // Whether a quotient within 2^-21 of q (relative) might belong to another code than q does.
  static __device__ __forceinline__ bool near_border(float q) {
    if constexpr (!kFloat) return fabsf(q - rintf(q)) > 0.49996f;
    const uint32_t low = __builtin_bit_cast(uint32_t, q) & 0xfffffu;      // what four significant bits drop
    const float t = q * 512.0f;                                           // below 2^-6 the codes are 2^-9 apart
    return low - 0x7fff0u <= 0x20u || (fabsf(q) < 0x1.0002p-6f && fabsf(t - rintf(t)) > 0.4999f);
  }

  // A number on the same side of every border as the exact x / scale: the quotient rounded to fp32, moved off itself by one
  // step towards the exact one where it is even (borders are even in fp32, so an odd one lies on none).  Where
  // x is of fp32 its quotient is on a border or at least 2^-33 of itself away: fp64 tells.
  static __device__ __forceinline__ float side_of(double x, float scale) {
    const double exact = x / (double)scale;
    const float q = (float)exact;
    const double rest = exact - (double)q;
    uint32_t b = __builtin_bit_cast(uint32_t, q);
    if (rest != 0.0 && (b & 1) == 0 && (b << 1) != 0) b += ((rest > 0.0) == (q > 0.0f)) ? 1u : ~0u;
    return __builtin_bit_cast(float, b);
  }

  // Four values' codes, one to a byte.  inverse = 1 / scale.  Values of fp64 are rounded for the quick quotient alone.
  template <typename X>
  static __device__ __forceinline__ uint32_t pack(const X (&x)[4], float scale, float inverse) {
    float q[4];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = (float)x[i] * inverse;
      near |= near_border(q[i]);
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = side_of((double)x[i], scale);
    }
    if constexpr (kFloat) {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)rintf(q[i]) & 0xffu) << (8 * i);
      return w;
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
