// Root-mean-square norm of rows of C channels, with the residual's addition in front of it and, where asked for, an
// output in 8 bits behind it.
//
//   h = x + residual (rounded once to the type: what the backward reads is what was normalised)
//   y = h r w,  r = 1 / sqrt(mean_c h^2 + eps)
//   backward, with u = gy w:   gx = r (u - h r^2 mean_c(u h)) + gh,   gw = sum_rows gy h r
//
// Memory bounds it: each tensor once.  A row belongs to a team of 4 to 1024 lanes that keeps it in registers between the
// reduction and the output, so nothing is read twice.  The team is the narrowest that holds the row in one 16-byte piece a
// lane, up to 1024 pieces (two or four pieces a lane beyond): short rows (heads of 32) fill the wave with rows instead of idle
// lanes, long ones spread over many waves (2000 rows of 8192 channels both directions: 67 us, with four pieces a lane
// 100).  Beyond 8192 channels the backward's 1024 lanes have too few registers for gw as well and keep 10 (bf16) or 65 (fp32) of
// theirs in scratch memory: 2000 rows of 16384 both directions 143 and 246 us, 3.7 and 4.3 TB/s.  Teams of up to 64 lanes reduce by lane exchanges alone, wider ones once through LDS.  Pieces are moved at
// any alignment (the card's global loads and stores take any address), the piece across a row's end element by element.
// The backward's workgroups walk many rows, the next one on its way, and keep their share of gw in registers; partial sums go
// to the workspace once per workgroup and a second launch adds them in a fixed order.
//
// 8192 rows of 4096 bf16 channels with a residual into e4m3, 128 channels to a scale: 56 us, 4.2 of the copy's 5.1 TB/s; 45
// of them issue vector instructions (52 a channel, 7 of them for what the largest product's rounding dropped).  67584 rows
// of 256 both directions: 27 + 29 + 4 us, 4.7 TB/s in the two large launches.  40000 x 8 heads of 32 out of a packed
// projection: 10 us, the launch and 4.1 TB/s.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "codes.h"
#include "decoder.h"
#include "encoder.h"
#include "pieces.h"
#include "wave_ops.h"

namespace fbev {
namespace {

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// Channels c .. c + kVec of a row (`left` of them exist) as fp32, zeros behind the end.
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, int left, float (&v)[kVec<T>]) {
  constexpr int V = kVec<T>;
  T e[V];
  if (left >= V) {
    __builtin_memcpy(e, p, 16);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
  }
}

// The same in two steps, for pieces that are loaded a row ahead.
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, int left, T (&e)[kVec<T>]) {
  constexpr int V = kVec<T>;
  if (left >= V) {
    __builtin_memcpy(e, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = i < left ? p[i] : (T)0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_piece(T* p, int left, const float (&v)[kVec<T>]) {
  constexpr int V = kVec<T>;
  if (left >= V) {
    T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = (T)v[i];
    __builtin_memcpy(p, e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) p[i] = (T)v[i];
  }
}

__device__ __forceinline__ void load_weight(const float* w, int c, int left, float* v, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) v[i] = 1.0f;
  if (w == nullptr || left <= 0) return;
  if (left >= n) {
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      if (j < n) __builtin_memcpy(v + j, w + c + j, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n && i < left) v[i] = w[c + i];
  }
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }

// The largest over aligned groups of n lanes (a power of two up to 64).
template <typename X>
__device__ __forceinline__ X lanes_max(X x, int n) {
  if (n >= 2) x = larger(x, dpp<kQuadSwap1>(x));
  if (n >= 4) x = larger(x, dpp<kQuadSwap2>(x));
  if (n >= 8) x = larger(x, dpp<kHalfMirror>(x));
  if (n >= 16) x = larger(x, dpp<kRowMirror>(x));
  if (n >= 32) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t p = r[0], q = r[1];
    x = larger(__builtin_bit_cast(X, p), __builtin_bit_cast(X, q));
  }
  if (n >= 64) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t p = r[0], q = r[1];
    x = larger(__builtin_bit_cast(X, p), __builtin_bit_cast(X, q));
  }
  return x;
}

// x of the lane that DPP control Ctrl names (32 or 64 bits).
template <int Ctrl, typename X>
__device__ __forceinline__ X dpp_any(X x) {
  if constexpr (sizeof(X) == 4) {
    return dpp<Ctrl>(x);
  } else {
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)dpp<Ctrl>((int)(uint32_t)v), hi = (uint32_t)dpp<Ctrl>((int)(uint32_t)(v >> 32));
    return __builtin_bit_cast(X, (uint64_t)hi << 32 | lo);
  }
}
template <bool HALVES>
__device__ __forceinline__ double swap_add(double x) {
  const uint64_t v = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
  uint32_t a[2], b[2];
  if constexpr (HALVES) {
    const auto p = __builtin_amdgcn_permlane32_swap(lo, lo, false, false), q = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    a[0] = p[0], a[1] = p[1], b[0] = q[0], b[1] = q[1];
  } else {
    const auto p = __builtin_amdgcn_permlane16_swap(lo, lo, false, false), q = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    a[0] = p[0], a[1] = p[1], b[0] = q[0], b[1] = q[1];
  }
  return __builtin_bit_cast(double, (uint64_t)b[0] << 32 | a[0]) + __builtin_bit_cast(double, (uint64_t)b[1] << 32 | a[1]);
}
template <bool HALVES>
__device__ __forceinline__ float swap_add(float x) {
  return HALVES ? swap32_add(x, x) : swap16_add(x, x);
}

template <int L, typename X>
__device__ __forceinline__ X lanes_sum(X x) {
  x += dpp_any<kQuadSwap1>(x);
  x += dpp_any<kQuadSwap2>(x);
  if constexpr (L >= 8) x += dpp_any<kHalfMirror>(x);
  if constexpr (L >= 16) x += dpp_any<kRowMirror>(x);
  if constexpr (L >= 32) x = swap_add<false>(x);
  if constexpr (L >= 64) x = swap_add<true>(x);
  return x;
}

// The team's sum in each of its lanes.  `slots`: LDS for one number of each wave, used by teams of several waves and not
// again before another barrier.
template <int L, typename X>
__device__ __forceinline__ X team_sum(X x, double* slots) {
  if constexpr (L <= 64) return lanes_sum<L>(x);
  x = lanes_sum<64>(x);
  X* mine = (X*)slots;
  if ((threadIdx.x & 63) == 0) mine[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int i = 0; i < L / 64; ++i) x += mine[i];
  return x;
}

template <int L, typename X>
__device__ __forceinline__ X team_max(X x, double* slots) {
  if constexpr (L <= 64) return lanes_max(x, L);
  x = lanes_max(x, 64);
  X* mine = (X*)slots;
  if ((threadIdx.x & 63) == 0) mine[threadIdx.x >> 6] = x;
  __syncthreads();
  x = mine[0];
#pragma unroll
  for (int i = 1; i < L / 64; ++i) x = larger(x, mine[i]);
  return x;
}

constexpr int team_threads(int L) { return L > 64 ? L : 256; }

__device__ __forceinline__ int64_t row_offset(int64_t row, int64_t inner, const int64_t (&s)[2]) {
  if (inner == 1) return row * s[0];
  const uint32_t o = (uint32_t)row / (uint32_t)inner;
  return o * s[0] + (row - (int64_t)o * inner) * s[1];
}

// y = h w r of a row in 8 bits, a scale for each `block` channels.  The codes are those of the exact y over its exact scale,
// where r cancels but for the least one:  r = 2^e m,  p = (2^e h) w,  code = nearest(p m / max(max |p| m / most, 2^-126)).
// p is taken in fp32 and a code near a border again in fp64, where the product is exact; the scale takes what rounding dropped
// of the largest p, and is rounded once.
// Blocks are narrower than the row only where a lane's pieces lie L apart and a block's 4 to 32 lanes side by side.
template <int L>
constexpr int kWaves = team_threads(L) / 64;
template <int KIND, int L, int K, int V>
__device__ __forceinline__ void store_codes(const RmsArgs& a, int64_t row, int lane, bool mine, const float (&h)[K][V], double r,
                                            double* slots) {
#pragma clang fp contract(off)
  using Cd = Codes<KIND>;
  const int nb = a.block < a.C ? a.block / V : 0;       // lanes of a block (0: the row)
  const int blocks = nb ? (a.C + a.block - 1) / a.block : 1;
  uint8_t* out = (uint8_t*)a.y + row * a.C;
  const int e = __builtin_amdgcn_frexp_exp(r) - 1;      // 1 <= m < 2: p is finite where y is
  const double m = 2.0 * __builtin_amdgcn_frexp_mant(r);
  float x[K][V], w[K][V], p[K][V], rest[K];
  uint32_t top[K];
  // the row's largest where a row is a block, else each block's
  const auto widest = [&](auto& t, double* slots) {
    if (nb == 0) {
      auto all = t[0];
#pragma unroll
      for (int k = 1; k < K; ++k) all = larger(all, t[k]);
      all = team_max<L>(all, slots);
#pragma unroll
      for (int k = 0; k < K; ++k) t[k] = all;
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) t[k] = lanes_max(t[k], nb);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + L * k) * V;
    load_weight(a.weight, c, a.C - c, w[k], V);
    top[k] = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[k][i] = __builtin_amdgcn_ldexpf(h[k][i], e);
      p[k][i] = x[k][i] * w[k][i];
      top[k] = larger(top[k], abs_bits(p[k][i]));
    }
  }
  widest(top, slots);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    rest[k] = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t sign = __builtin_bit_cast(uint32_t, p[k][i]) & 0x80000000u;
      const float dropped = fmaf(x[k][i], w[k][i], -p[k][i]);
      const float along = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, dropped) ^ sign);
      rest[k] = abs_bits(p[k][i]) == top[k] ? fmaxf(rest[k], along) : rest[k];
    }
  }
  widest(rest, slots + kWaves<L>);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + L * k) * V, left = a.C - c;
    if (left <= 0 || !mine) continue;
    const double wide = ((double)__builtin_bit_cast(float, top[k]) + (double)rest[k]) * m * (1.0 / Cd::kMost);
    const bool odd = top[k] >= 0x7f800000u || wide != wide;
    const float scale = odd ? __builtin_nanf("") : fmaxf((float)wide, kLeastScale);
    const float inverse = (float)m * Cd::inverse_of(scale);
    uint32_t codes[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = p[k][4 * j + i];
      codes[j] = Cd::pack(y, fmax(wide, (double)kLeastScale), inverse,
                          [&](int i) { return (double)x[k][4 * j + i] * (double)w[k][4 * j + i] * m; });
      if (odd) codes[j] = 0;
    }
    if (left >= V) {
      __builtin_memcpy(out + c, codes, V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) out[c + i] = (uint8_t)(codes[i / 4] >> (8 * (i % 4)));
    }
    if (nb ? (lane & (nb - 1)) == 0 : c == 0) a.scales[row * blocks + (nb ? c / a.block : 0)] = scale;
  }
}

// CODES: the codes have no other rounding than their own.  The sum of squares and 1 / sqrt are fp64.
template <typename T, int L, int K, bool CODES>
__global__ __launch_bounds__(team_threads(L)) void rms_fwd(RmsArgs a) {
  constexpr int V = kVec<T>, kThreads = team_threads(L), kTeams = kThreads / L;
  __shared__ double slots[3 * kWaves<L>];               // one reduction each
  const int lane = threadIdx.x % L;
  const int64_t first = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kTeams + threadIdx.x / L;
  if (L > 64 && first >= a.rows) return;                // the whole workgroup; narrower teams stay for the lane exchanges
  const int64_t row = first < a.rows ? first : a.rows - 1;
  const bool mine = first < a.rows;
  const T* x = (const T*)a.x + row_offset(row, a.inner, a.xs);
  const T* res = a.residual ? (const T*)a.residual + row_offset(row, a.inner, a.rs) : nullptr;
  // (weights in front of the rows: 67584 rows of 256 channels both directions 60 us against 63.5, 10007 of 1001 in fp32 66
  // against 67; not where a row is a wave's smaller part or 1024 threads', whose registers they cost: 40000 x 8 heads of 32
  // 10.7 against 9.9, 2000 rows of 8192 channels 72 against 67)
  constexpr bool kEarly = !CODES && L >= 32 && L <= 512;
  float w[K][V];
  const auto load_weights = [&] {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      load_weight(a.weight, c, a.C - c, w[k], V);
    }
  };
  if (kEarly) load_weights();
  float v[K][V];
  if constexpr (L < 32) {
    float more[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      load_piece(x + c, a.C - c, v[k]);
      if (res) load_piece(res + c, a.C - c, more[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = res ? to_f32((T)(v[k][i] + more[k][i])) : v[k][i];
  } else {
    T xr[K][V], rr[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      load_raw(x + c, a.C - c, xr[k]);
      if (res) load_raw(res + c, a.C - c, rr[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = res ? to_f32((T)(to_f32(xr[k][i]) + to_f32(rr[k][i]))) : to_f32(xr[k][i]);
  }
  if (res && mine) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      store_piece((T*)a.h + row * a.C + c, a.C - c, v[k]);
    }
  }
  if constexpr (CODES) {
    double squares = 0.0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) squares = fma((double)v[k][i], (double)v[k][i], squares);
    // 1 / sqrt from the hardware's, two steps of Newton's method behind it (0, infinity and NaN as they come)
    const double mean = team_sum<L>(squares, slots) * a.part_of_row + (double)a.eps, near = __builtin_amdgcn_rsq(mean);
    double r = near;
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(r, fma(-0.5 * mean * r, r, 0.5), r);
    r = mean > 0.0 && mean < __builtin_huge_val() ? r : near;
    if (a.codes == FBEV_CODES_E4M3)
      store_codes<FBEV_CODES_E4M3, L, K, V>(a, row, lane, mine, v, r, slots + kWaves<L>);
    else
      store_codes<FBEV_CODES_INT8, L, K, V>(a, row, lane, mine, v, r, slots + kWaves<L>);
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(v[k][i], v[k][i], sum);
    sum = team_sum<L>(sum, slots);
    const float r = 1.0f / sqrtf(sum / (float)a.C + a.eps);
    if (a.rstd && lane == 0 && mine) a.rstd[row] = r;
    if (!kEarly) load_weights();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V, left = a.C - c;
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * r * w[k][i];
      if (mine) store_piece((T*)a.y + row * a.C + c, left, v[k]);
    }
  }
}

// gx of the rows, and each workgroup's share of gw in `part` [gridDim.x][C].
template <typename T, int L, int K>
__global__ __launch_bounds__(team_threads(L)) void rms_bwd(RmsArgs a) {
  constexpr int V = kVec<T>, kThreads = team_threads(L), kTeams = kThreads / L;
  __shared__ double slots[2][kWaves<L>];                // of odd and even rounds: the other round's barrier lies between
  const int lane = threadIdx.x % L;
  float w[K][V], gw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (lane + L * k) * V;
    load_weight(a.weight, c, a.C - c, w[k], V);
#pragma unroll
    for (int i = 0; i < V; ++i) gw[k][i] = 0.0f;
  }
  // every team of a workgroup makes the same number of rounds; where a lane has one piece, a row's are on their way while
  // the row before is at work (rows of 1001 fp32 channels, both directions: 82 -> 67 us)
  constexpr bool kAhead = K == 1;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  T hr[K][V], gr[K][V], mr[K][V];
  float rr;
  const auto load_row = [&](int64_t at) {
    const int64_t row = at < a.rows ? at : a.rows - 1;
    const T* x = (const T*)a.x + row_offset(row, a.inner, a.xs);
    const T* gy = (const T*)a.gy + row * a.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      load_raw(x + c, a.C - c, hr[k]);
      load_raw(gy + c, a.C - c, gr[k]);
      if (a.gh) load_raw((const T*)a.gh + row * a.C + c, a.C - c, mr[k]);
    }
    rr = a.rstd[row];
  };
  int64_t at = (int64_t)blockIdx.x * kTeams + threadIdx.x / L;
  if (kAhead) load_row(at);
  int odd = 0;
  for (int64_t base = (int64_t)blockIdx.x * kTeams; base < a.rows; base += step, at += step, odd ^= 1) {
    const bool mine = at < a.rows;
    if (!kAhead) load_row(at);
    float h[K][V], g[K][V], more[K][V], dot = 0.0f;
    const float r = rr;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[k][i] = to_f32(hr[k][i]);
        g[k][i] = to_f32(gr[k][i]);
        more[k][i] = a.gh ? to_f32(mr[k][i]) : 0.0f;
      }
    if (kAhead && base + step < a.rows) load_row(at + step);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) dot = fmaf(g[k][i] * w[k][i], h[k][i], dot);
    dot = team_sum<L>(dot, slots[odd]);
    const float along = dot / (float)a.C * r * r;
    if (!mine) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
      float gx[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        gx[i] = r * (g[k][i] * w[k][i] - h[k][i] * along);
        if (a.gh) gx[i] += more[k][i];
        gw[k][i] = fmaf(g[k][i], h[k][i] * r, gw[k][i]);
      }
      store_piece((T*)a.gx + at * a.C + c, a.C - c, gx);
    }
  }
  if (a.gweight == nullptr) return;
  float* part = a.part + (int64_t)blockIdx.x * a.C;
  if constexpr (L <= 64) {
    // the teams of a wave by lane exchanges, the waves through LDS
    __shared__ float joined[4][L * K * V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s = gw[k][i];
        if constexpr (L <= 4) s += dpp<kRowRor4>(s);
        if constexpr (L <= 8) s += dpp<kRowRor8>(s);
        if constexpr (L <= 16) s = swap16_add(s, s);
        if constexpr (L <= 32) s = swap32_add(s, s);
        if ((threadIdx.x & 63) < L) joined[threadIdx.x >> 6][(k * V + i) * L + lane] = s;
      }
    __syncthreads();
    for (int n = threadIdx.x; n < L * K * V; n += kThreads) {
      const int l = n % L, i = n / L % V, k = n / L / V, c = (l + L * k) * V + i;
      if (c < a.C) part[c] = joined[0][n] + joined[1][n] + joined[2][n] + joined[3][n];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (lane + L * k) * V;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < a.C) part[c + i] = gw[k][i];
    }
  }
}

// gw from the workgroups' shares: 32 channels by 32 runs of shares a workgroup, every run in order.
__global__ __launch_bounds__(1024) void rms_join(const float* part, float* gw, int C, int shares) {
  __shared__ float sums[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int i = run; i < shares; i += 32) s += part[(int64_t)i * C + c];
  }
  sums[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run != 0 || c >= C) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
  gw[c] = s;
}

// The team of a row of `pieces` pieces: f(lanes, pieces a lane).
template <typename F>
auto with_team(int pieces, F f) {
  if (pieces <= 4) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  if (pieces <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (pieces <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (pieces <= 32) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (pieces <= 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (pieces <= 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
  if (pieces <= 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (pieces <= 512) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
  if (pieces <= 1024) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
  if (pieces <= 2048) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

int pieces_of(const RmsArgs& a) { return (int)(((int64_t)a.C * a.elem_bytes + 15) / 16); }

// Workgroups of the backward: 1024 threads a CU (2048: 5000 rows of 2048 channels 48 against 44 us, for the shares), with four
// rounds of rows each where that still leaves a workgroup a CU (eight: 46 us).
int backward_blocks(const RmsArgs& a, int teams, int threads) {
  const int64_t rounds = (a.rows + teams - 1) / teams, most = 256 * (1024 / threads);
  int64_t n = rounds / 4 > 256 ? rounds / 4 : 256;
  if (n > rounds) n = rounds;
  return (int)(n < most ? n : most);
}

}  // namespace

size_t rms_norm_workspace_bytes(const RmsArgs& a) {
  if (a.rows == 0) return 0;
  return with_team(pieces_of(a), [&](auto L, auto) {
    return (size_t)backward_blocks(a, team_threads(L) / L, team_threads(L)) * a.C * sizeof(float);
  });
}

hipError_t launch_rms_norm_forward(const RmsArgs& a, hipStream_t stream) {
  return with_team(pieces_of(a), [&](auto L, auto K) {
    constexpr int kTeams = team_threads(L) / L;
    const dim3 grid = grid_rows((a.rows + kTeams - 1) / kTeams);
    const auto run = [&](auto codes) {
      if (a.elem_bytes == 4)
        rms_fwd<float, L, K, codes><<<grid, team_threads(L), 0, stream>>>(a);
      else if constexpr (!(L == 1024 && K == 4))        // FBEV_MAX_RMS_CHANNELS bf16 are 2048 pieces
        rms_fwd<__bf16, L, K, codes><<<grid, team_threads(L), 0, stream>>>(a);
    };
    if (a.codes < 0)
      run(std::false_type{});
    else
      run(std::true_type{});
    return hipGetLastError();
  });
}

hipError_t launch_rms_norm_backward(const RmsArgs& a, hipStream_t stream) {
  if (a.rows == 0) {      // no rows: gw is zero
    rms_join<<<(a.C + 31) / 32, 1024, 0, stream>>>(a.part, a.gweight, a.C, 0);
    return hipGetLastError();
  }
  return with_team(pieces_of(a), [&](auto L, auto K) {
    const int blocks = backward_blocks(a, team_threads(L) / L, team_threads(L));
    if (a.elem_bytes == 4)
      rms_bwd<float, L, K><<<blocks, team_threads(L), 0, stream>>>(a);
    else if constexpr (!(L == 1024 && K == 4))
      rms_bwd<__bf16, L, K><<<blocks, team_threads(L), 0, stream>>>(a);
    if (a.gweight) rms_join<<<(a.C + 31) / 32, 1024, 0, stream>>>(a.part, a.gweight, a.C, blocks);
    return hipGetLastError();
  });
}

}  // namespace fbev
