// Wave-level pieces of the attention kernels (64-lane waves, 32 x 32 MFMA tiles).
//
// A wave keeps one side of the problem in registers ("own": 32 rows, one per lane pair l, l + 32) and
// walks the other ("moving": tiles of 32 rows in LDS).  The product moving x own^T leaves lane (n, h)
// (n = lane mod 32, h = lane / 32) with own row n and the 16 moving rows 8 (i / 4) + 4 h + (i mod 4) of
// the tile, i < 16: everything a softmax row needs is in two lanes.  Those 16 values are at once the B
// operand of the next product, moving^T x values: its contraction runs over the tile's rows, whose order
// is free as long as the A operand (the transposed tile) uses the same one, so probabilities never leave
// their registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "encoder.h"
#include "wave_ops.h"

namespace fbev {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

// The moving row of accumulator register i (0 .. 15) in half-wave h.
__device__ __forceinline__ int acc_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// Over the two lanes of an own row.
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  const uint32_t a = r[0], b = r[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float pair_sum(float x) { return swap32_add(x, x); }

template <typename T, int DP>
struct Mma;

// bf16: contraction in steps of 16 channels (row products) and 16 rows (transposed products).
template <int DP>
struct Mma<__bf16, DP> {
  using T = __bf16;
  using Frag = bf16x8;
  static constexpr int kFrags = DP / 16;                 // fragments of one row's DP channels
  static constexpr int kPadRow = DP + (DP == 32 ? 8 : 8);  // LDS row stride in elements

  // fragment f of a row: channels 16 f + 8 h ..
  static __device__ __forceinline__ int frag_channel(int f, int h) { return 16 * f + 8 * h; }
  static constexpr int kFragElems = 8;

  static __device__ __forceinline__ f32x16 dot(const Frag& a, const Frag& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }

  // The B operand: values of tile rows 16 c .. 16 c + 15 (accumulator registers 8 c .. 8 c + 7).
  struct Values {
    bf16x8 v[2];
  };
  static __device__ __forceinline__ Values pack(const f32x16& p) {
    Values r;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) r.v[c][j] = (__bf16)p[8 * c + j];
    return r;
  }

  // The A operand: channels 32 blk + n of the rows above, read transposed (four rows by 16 channels for
  // every 16 lanes; lane i of the 16 addresses row i / 4, channels 4 (i mod 4)).
  static __device__ __forceinline__ bf16x8 columns(const T* tile, int c, int blk, int lane) {
    const int h = lane >> 5, i = lane & 15;
    const T* at = tile + (16 * c + 4 * h + (i >> 2)) * kPadRow + 32 * blk + (lane & 16) + 4 * (i & 3);
    auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4*)(uint32_t)(uintptr_t)at);
    auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4*)(uint32_t)(uintptr_t)(at + 8 * kPadRow));
    union {
      i16x4 s[2];
      bf16x8 v;
    } u;
    u.s[0] = lo;
    u.s[1] = hi;
    return u.v;
  }

  template <int NB>
  static __device__ __forceinline__ void accumulate(f32x16 (&acc)[NB], const Values& p, const T* tile, int lane) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(columns(tile, c, blk, lane), p.v[c], acc[blk], 0, 0, 0);
  }

  // Infinities and NaN in a tile of which some (row, own row) pairs are masked: such an element must reach
  // only the own rows that see it.  They are taken out of the product, and whether an own row sees a
  // positive or a negative one (a NaN counts as both) comes from two products with the visibility.
  static __device__ __forceinline__ bool odd(const bf16x8& a) {
    const i32x4 w = __builtin_bit_cast(i32x4, a);
    bool o = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o |= ((w[j] & 0x7F80) == 0x7F80) | ((w[j] & 0x7F800000) == 0x7F800000);
    return o;
  }
  template <int NB>
  static __device__ __forceinline__ void accumulate_masked(f32x16 (&acc)[NB], const Values& p, const Values& seen,
                                                           const T* tile, int lane) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      bf16x8 a[2];
      a[0] = columns(tile, 0, blk, lane);
      a[1] = columns(tile, 1, blk, lane);
      if (__builtin_expect(__any(odd(a[0]) || odd(a[1])), 0)) {
        f32x16 up = {}, down = {};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          bf16x8 u, d;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = (float)a[c][j];
            const bool fin = fabsf(x) < __builtin_huge_valf();
            u[j] = (__bf16)(!fin && !(x < 0.0f) ? 1.0f : 0.0f);
            d[j] = (__bf16)(!fin && !(x > 0.0f) ? 1.0f : 0.0f);
            if (!fin) a[c][j] = (__bf16)0.0f;
          }
          up = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u, seen.v[c], up, 0, 0, 0);
          down = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d, seen.v[c], down, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (up[i] > 0.0f) acc[blk][i] += __builtin_huge_valf();
          if (down[i] > 0.0f) acc[blk][i] += kNegInf;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[c], p.v[c], acc[blk], 0, 0, 0);
    }
  }
};

// fp32: contraction in steps of two; a fragment is four channels (the half-waves' share of eight).
template <int DP>
struct Mma<float, DP> {
  using T = float;
  using Frag = f32x4;
  static constexpr int kFrags = DP / 8;
  static constexpr int kPadRow = DP + 8;
  static __device__ __forceinline__ int frag_channel(int f, int h) { return 8 * f + 4 * h; }
  static constexpr int kFragElems = 4;

  static __device__ __forceinline__ f32x16 dot(const Frag& a, const Frag& b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }

  struct Values {
    f32x16 v;
  };
  static __device__ __forceinline__ Values pack(const f32x16& p) { return Values{p}; }

  static __device__ __forceinline__ float column(const T* tile, int i, int blk, int lane) {
    return tile[acc_row(i, lane >> 5) * kPadRow + 32 * blk + (lane & 31)];
  }

  template <int NB>
  static __device__ __forceinline__ void accumulate(f32x16 (&acc)[NB], const Values& p, const T* tile, int lane) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x2f32(column(tile, i, blk, lane), p.v[i], acc[blk], 0, 0, 0);
  }

  template <int NB>
  static __device__ __forceinline__ void accumulate_masked(f32x16 (&acc)[NB], const Values& p, const Values& seen,
                                                           const T* tile, int lane) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      float a[16];
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        a[i] = column(tile, i, blk, lane);
        odd |= !(fabsf(a[i]) < __builtin_huge_valf());
      }
      if (__builtin_expect(__any(odd), 0)) {
        f32x16 up = {}, down = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool fin = fabsf(a[i]) < __builtin_huge_valf();
          up = __builtin_amdgcn_mfma_f32_32x32x2f32(!fin && !(a[i] < 0.0f) ? 1.0f : 0.0f, seen.v[i], up, 0, 0, 0);
          down = __builtin_amdgcn_mfma_f32_32x32x2f32(!fin && !(a[i] > 0.0f) ? 1.0f : 0.0f, seen.v[i], down, 0, 0, 0);
          if (!fin) a[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (up[i] > 0.0f) acc[blk][i] += __builtin_huge_valf();
          if (down[i] > 0.0f) acc[blk][i] += kNegInf;
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], p.v[i], acc[blk], 0, 0, 0);
    }
  }
};

// One row's fragments from global memory, zero beyond its D channels.
template <typename T, int DP>
__device__ __forceinline__ void load_row(const T* row, bool valid, bool vec, int D, int h,
                                         typename Mma<T, DP>::Frag (&f)[Mma<T, DP>::kFrags]) {
  using M = Mma<T, DP>;
#pragma unroll
  for (int i = 0; i < M::kFrags; ++i) {
    const int c = M::frag_channel(i, h);
    if (valid && vec && c + M::kFragElems <= D) {
      f[i] = *(const typename M::Frag*)(row + c);
    } else {
#pragma unroll
      for (int j = 0; j < M::kFragElems; ++j) f[i][j] = (valid && c + j < D) ? row[c + j] : (T)0.0f;
    }
  }
}

// Rows [r0, r0 + N) of a tensor into LDS rows of stride kPadRow, zero beyond `rows` and beyond D channels.
// row_ptr(r) gives row r's address.  By the whole workgroup.
template <typename T, int DP, int N, int THREADS, typename F>
__device__ __forceinline__ void stage_rows(T* lds, int rows, bool vec, int D, F row_ptr) {
  constexpr int E = 16 / sizeof(T), PIECES = DP / E;
  typedef T Vec __attribute__((ext_vector_type(E)));
#pragma unroll 2
  for (int e = threadIdx.x; e < N * PIECES; e += THREADS) {
    const int r = e / PIECES, c = (e - r * PIECES) * E;
    Vec v;
    if (r < rows && vec && c + E <= D) {
      v = *(const Vec*)(row_ptr(r) + c);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = (T)0.0f;
      if (r < rows && c < D) {
        const T* p = row_ptr(r) + c;
        for (int j = 0; j < E && c + j < D; ++j) v[j] = p[j];
      }
    }
    *(Vec*)(lds + r * Mma<T, DP>::kPadRow + c) = v;
  }
}

// The row fragments of tile row n.
template <typename T, int DP>
__device__ __forceinline__ typename Mma<T, DP>::Frag tile_frag(const T* tile, int f, int lane) {
  using M = Mma<T, DP>;
  return *(const typename M::Frag*)(tile + (lane & 31) * M::kPadRow + M::frag_channel(f, lane >> 5));
}

// tanh(u).  Through e = exp(-2 |u|) as (1 - e) / (1 + e); near zero, where 1 - e cancels, fp32 scores take the odd
// Taylor series instead (|u| < 1/4: the first term left out is below 1e-8 of the value).
template <bool EXACT>
__device__ __forceinline__ float tanh_fast(float u) {
  const float e = __builtin_amdgcn_exp2f(fabsf(u) * (-2.0f * kLog2e));
  float t = copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), u);
  if constexpr (EXACT) {
    const float u2 = u * u;
    float s = fmaf(u2, 0.021869488f, -0.053968254f);
    s = fmaf(u2, s, 0.13333333f);
    s = fmaf(u2, s, -0.33333333f);
    s = fmaf(u2 * u, s, u);
    t = fabsf(u) < 0.25f ? s : t;
  }
  return t;
}

// What an own query row needs to know about itself.
struct Row {
  int r, t, head;       // row, token, query head
  int lim;              // last visible key by order (-1: none)
  int doc;
};

__device__ __forceinline__ int row_limit(const AttnArgs& a, int b, int t) {
  if (!a.causal) return a.Tk - 1;
  const int pre = a.prefix ? a.prefix[b] : 0;
  return min(a.Tk - 1, max(t + a.Tk - a.Tq, pre - 1));
}

__device__ __forceinline__ Row make_row(const AttnArgs& a, int b, int hk, int r) {
  Row w;
  w.r = r;
  w.t = r / a.G;
  w.head = hk * a.G + (r - w.t * a.G);
  w.lim = row_limit(a, b, w.t);
  w.doc = a.doc_q ? a.doc_q[(int64_t)b * a.Tq + w.t] : 0;
  if (w.doc < 0) w.lim = -1;
  return w;
}

// min / max over the wave.
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = min(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = max(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}

// Distances between the lane's own point and the 16 moving points of its accumulator registers
// (pos[axis][tile row] in LDS).
template <int N>
__device__ __forceinline__ void distances(const float (*pos)[N], int at, int dims, const float (&own)[3], int h,
                                          f32x16& d) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = at + 8 * u + 4 * h;
    f32x4 x = *(const f32x4*)&pos[0][r];
    f32x4 y = *(const f32x4*)&pos[1][r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float dx = x[j] - own[0], dy = y[j] - own[1];
      d[4 * u + j] = fmaf(dx, dx, dy * dy);
    }
    if (dims > 2) {
      f32x4 z = *(const f32x4*)&pos[2][r];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float dz = z[j] - own[2];
        d[4 * u + j] = fmaf(dz, dz, d[4 * u + j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i] = __builtin_amdgcn_sqrtf(d[i]);
}

}  // namespace fbev
