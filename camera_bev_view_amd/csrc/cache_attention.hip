// Attention of query tokens, a tree of drafted ones among others, over the token cache.
//
//   s_ij = scale q_i . (kc_j ks_j),  s = cap tanh(s / cap),  o_i = sum_j softmax_j(s) (vc_j vs_j)
//
// kc, vc: codes in 8 bits; ks, vs: a token's scales.  Codes of either format are bf16 numbers without rounding, so the
// matrix products run on bf16 codes while the scales join in fp32: ks multiplies the score, vs the weight.  What is not
// exact in bf16 goes in as parts: fp32 queries and weights as three (24 bits), the weights of bf16 tensors as two (16 bits:
// one would add as much error as the result's own rounding), bf16 queries as they are.
//
// Memory bounds the calls of serving (few rows over a long cache): the cache's codes are read once and straight into the
// registers that feed the matrix instructions, with no turn through LDS.  A wave takes a page of 64 tokens at a time, both
// products with the tokens (or channels) as the instruction's rows and 16 queries as its columns:
//   S^T = K Q^T:  lane (r, g) of r = lane mod 16, g = lane / 16 loads 16 bytes (channels 16 g ..) of token 16 (r / 4) + 4 u + r mod 4,
//                 u = 0 .. 3, so that the result leaves it the scores of tokens 16 g .. 16 g + 15 of query r;
//   O^T = V^T P^T: those 16 weights are its operand as they stand, and the values, kept with their tokens side by side, are
//                 16 bytes (tokens 16 g ..) of channel r.
// A page's keys are loaded while the one before is in its softmax and second product, its values under the first one.
// The waves of a workgroup share the rows and take pages in turn; where rows are few, the pages are split over workgroups
// as well and a second launch joins them.  Row tiles (16 queries times heads of a key head) are held RT at a time: each
// code is read and converted once for all of them.
#include <hip/hip_runtime.h>

#include "attention_core.h"
#include "codes.h"
#include "decoder.h"
#include "encoder.h"
#include "wave_ops.h"

namespace fbev {
namespace {

constexpr int kWaves = 4;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

union Frag {
  uint32_t w[4];
  bf16x8 v;
};

// The high halves of two fp32 (bf16 numbers already).
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  const bf16x2 p = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, p);
}

// Eight codes as bf16.
template <int KIND>
__device__ __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
  Frag f;
  const uint32_t in[2] = {a, b};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (KIND == FBEV_CODES_E4M3) {
      f.w[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(in[j], 1.0f, false));
      f.w[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(in[j], 1.0f, true));
    } else {
      float x[4];
      Codes<KIND>::unpack(in[j], x);
      f.w[2 * j] = high_halves(x[0], x[1]);
      f.w[2 * j + 1] = high_halves(x[2], x[3]);
    }
  }
  return f.v;
}

// x[0 .. 7] as PARTS bf16 each that add up to it.
template <int PARTS>
__device__ __forceinline__ void split(const float (&x)[8], bf16x8 (&out)[PARTS]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = x[i];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.w[i] = to_bf16x2(rest[2 * i], rest[2 * i + 1]);
    out[p] = f.v;
    if (p + 1 < PARTS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rest[2 * i] -= __builtin_bit_cast(float, f.w[i] << 16);
        rest[2 * i + 1] -= __builtin_bit_cast(float, f.w[i] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Over the four lanes of a query.
__device__ __forceinline__ float query_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  const uint32_t a = r[0], b = r[1];
  return pair_max(fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
}
__device__ __forceinline__ float query_sum(float x) {
  x = swap16_add(x, x);
  return swap32_add(x, x);
}

// Tokens of the cache and of the call that somebody in rows up to `last_t` sees.
__device__ __forceinline__ int64_t visible_end(const CacheAttnArgs& a, int start, int rows, int last_t) {
  int64_t n = start;
  if (a.mode == FBEV_DRAFT_CHAIN) n += min(rows, last_t + 1);
  if (a.mode == FBEV_DRAFT_TREE) n += rows;
  return min(n, (int64_t)a.c.W * kPage);
}

// Bits of the 16 tokens from `pos` on that query t sees (pos: in the sequence).
__device__ __forceinline__ uint32_t seen_bits(const CacheAttnArgs& a, int b, int t, int start, int rows, int pos) {
  int n = start;                                        // every token below is seen
  if (a.mode == FBEV_DRAFT_CHAIN) n += t + 1;
  const int k = min(max(n - pos, 0), 16);
  uint32_t bits = (1u << k) - 1u;
  if (a.mode == FBEV_DRAFT_TREE && k < 16) {
    const uint64_t* words = a.ancestors + ((int64_t)b * a.c.T + t) * a.words;
    const int j = pos - start;                          // -15 .. : the first token's place among the drafted ones
    const int w = j >> 6, s = j & 63;                   // (a negative one lies in word -1, which has no bits)
    const int used = (a.c.T + 63) >> 6;
    uint64_t x = w >= 0 && w < used ? words[w] >> s : 0;
    if (s > 48 && w + 1 < used) x |= words[w + 1] << (64 - s);
    const int left = min(max(rows - j, 0), 16);         // what lies behind the last row does not exist
    bits |= (uint32_t)x & ((1u << left) - 1u) & 0xffffu;
  }
  return bits;
}

// What sums kept against the maximum m count for against `top`.  Without a maximum there is nothing to count, or nothing
// but NaN, which stays.
__device__ __forceinline__ float share(float m, float l, float top) {
  if (m == kNegInf) return l == 0.0f ? 0.0f : 1.0f;
  return __builtin_amdgcn_exp2f(m - top);
}

// DC: channels held, 32, 64 or 128.
template <typename T, int KIND, int DC, int RT>
struct Shape {
  static constexpr int kQ = sizeof(T) == 4 ? 3 : 1;     // parts of a query
  static constexpr int kP = sizeof(T) == 4 ? 3 : 2;     // parts of a weight
  static constexpr int kSteps = DC / 32;                // of the first product
  static constexpr int kChunk = DC >= 64 ? 16 : 8;      // bytes a lane loads of a key
  static constexpr int kChunks = DC >= 64 ? DC / 64 : 1;
  static constexpr int kTiles = DC / 16;                // of the second product's rows
  static constexpr int kQBytes = RT * kSteps * kQ * 64 * 16;
  static constexpr int kRow = DC + 4;                   // floats of a row in the join
  static constexpr int kJoinBytes = kWaves * 16 * kRow * 4;
  static constexpr int kLds = kQBytes > kJoinBytes ? kQBytes : kJoinBytes;
};

template <typename T, int KIND, int DC, int RT>
__global__ __launch_bounds__(64 * kWaves) void cache_attn(CacheAttnArgs a) {
  using Sh = Shape<T, KIND, DC, RT>;
  __shared__ alignas(16) char lds[Sh::kLds];
  __shared__ float2 joined[kWaves][16 * RT];
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int heads = c.B * c.Hk;
  int id = xcd_block(blockIdx.x, gridDim.x);
  const int rb = id % a.row_blocks;
  id /= a.row_blocks;
  const int part = id % a.splits, bh = id / a.splits;
  const int b = bh / c.Hk, hk = bh % c.Hk;
  const int row0 = rb * 16 * RT;

  // queries as the first product's columns: channel 64 c + 16 g + 8 h + j of step 2 c + h (8 g + j where one step is all)
#pragma unroll
  for (int i = 0; i < RT * Sh::kSteps / kWaves + (RT * Sh::kSteps % kWaves ? 1 : 0); ++i) {
    const int item = i * kWaves + wave;
    if (item < RT * Sh::kSteps) {
      const int rt = item / Sh::kSteps, step = item % Sh::kSteps;
      const int row = row0 + rt * 16 + r16, t = row / a.G, h = row - t * a.G;
      const int ch = Sh::kChunk == 16 ? (step >> 1) * 64 + g * 16 + (step & 1) * 8 : g * 8;
      const int left = row < a.R ? c.D - ch : 0;
      const T* q = (const T*)a.q + b * a.qs[0] + (int64_t)t * a.qs[1] + (int64_t)(hk * a.G + h) * a.qs[2] + ch;
      float x[8];
      if (left >= 8) {
        T e[8];
        __builtin_memcpy(e, q, sizeof e);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)e[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < left ? (float)q[j] : 0.0f;
      }
      bf16x8 parts[Sh::kQ];
      split<Sh::kQ>(x, parts);
#pragma unroll
      for (int p = 0; p < Sh::kQ; ++p) ((bf16x8*)lds)[(item * Sh::kQ + p) * 64 + lane] = parts[p];
    }
  }
  __syncthreads();

  const int start = min(c.start[b], c.W * kPage);       // (what lies beyond the table does not exist)
  const int rows = start < 0 ? 0 : min(c.count ? max(c.count[b], 0) : c.T, c.T);
  const int last_t = (min(row0 + 16 * RT, a.R) - 1) / a.G;
  const int end = rows > 0 ? (int)visible_end(a, start, rows, last_t) : 0;
  const int pages = (end + kPage - 1) / kPage;
  const int p0 = (int)((int64_t)pages * part / a.splits), p1 = (int)((int64_t)pages * (part + 1) / a.splits);
  const int32_t* table = c.table + (int64_t)b * c.W;

  f32x4 o[RT][Sh::kTiles];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = kNegInf;
    l[rt] = 0.0f;
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i) o[rt][i] = f32x4{0, 0, 0, 0};
  }

  // a page's codes and scales of this lane
  uint32_t kw[4][Sh::kChunks * Sh::kChunk / 4], vw[Sh::kTiles][4];
  f32x4 ks[4], vs[4];
  const int key = 16 * (r16 >> 2) + (r16 & 3);
  const auto load_keys = [&](int page) {
    const int64_t at = (int64_t)page * c.Hk + hk;
    const uint8_t* p = (const uint8_t*)c.k + at * kPage * c.Dp + key * c.Dp + Sh::kChunk * g;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < Sh::kChunks; ++i) {
        constexpr int kWordsOf = Sh::kChunk / 4;
        const bool there = 64 * i + Sh::kChunk * g < c.Dp;
#pragma unroll
        for (int j = 0; j < kWordsOf; ++j) kw[u][i * kWordsOf + j] = 0;
        if (there)
          __builtin_memcpy(&kw[u][i * kWordsOf], __builtin_assume_aligned(p + 4 * u * c.Dp + 64 * i, Sh::kChunk),
                           Sh::kChunk);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u) ks[u] = *(const f32x4*)(c.k_scale + at * kPage + 16 * g + 4 * u);
  };
  const auto load_values = [&](int page) {
    const int64_t at = (int64_t)page * c.Hk + hk;
    const uint8_t* p = (const uint8_t*)c.v + at * kPage * c.Dp + r16 * kPage + 16 * g;
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i) {
      const bool there = 16 * i < c.Dp;
      u32x4 x = {0, 0, 0, 0};
      if (there) x = *(const u32x4*)(p + 16 * kPage * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) vw[i][j] = x[j];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) vs[u] = *(const f32x4*)(c.v_scale + at * kPage + 16 * g + 4 * u);
  };
  // the wave's next page that exists, from `at` on (p1: none); its number in `page`
  int page = -1;
  const auto next_page = [&](int at) {
    for (; at < p1; at += kWaves) {
      page = uniform(table[at]);
      if (page >= 0 && page < c.pages) return at;
    }
    return p1;
  };

  const float unit = a.cap > 0 ? a.scale / a.cap : a.scale * kLog2e;
  int at = next_page(p0 + wave);
  if (at < p1) {
    load_keys(page);
    load_values(page);
  }
  while (at < p1) {
    f32x4 s[RT][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      bf16x8 kf[Sh::kSteps];
#pragma unroll
      for (int i = 0; i < Sh::kSteps; ++i) kf[i] = widen<KIND>(kw[u][2 * i], kw[u][2 * i + 1]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Sh::kSteps; ++i)
#pragma unroll
          for (int p = Sh::kQ - 1; p >= 0; --p)
            acc = mfma(kf[i], ((const bf16x8*)lds)[((rt * Sh::kSteps + i) * Sh::kQ + p) * 64 + lane], acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[rt][u][i] = acc[i] * unit * ks[u][i];
      }
    }
    const int pos = at * kPage;
    at = next_page(at + kWaves);
    if (at < p1) load_keys(page);

    if (a.cap > 0) {
      const float top = a.cap * kLog2e;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[rt][u][i] = top * tanh_fast<true>(s[rt][u][i]);
    }
    // a page that holds a token which some query does not see
    const bool masked = pos + kPage > (a.mode == FBEV_DRAFT_NONE ? end : min(start, end));
    uint32_t bits[RT];
    if (masked) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int row = row0 + rt * 16 + r16, t = row / a.G;
        bits[rt] = t < rows ? seen_bits(a, b, t, start, rows, pos + 16 * g) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(bits[rt] >> (4 * u + i) & 1)) s[rt][u][i] = kNegInf;
      }
      if constexpr (KIND == FBEV_CODES_E4M3) {          // what was never written may be the code of a NaN
        const int left = end - pos - 16 * g;
#pragma unroll
        for (int i = 0; i < Sh::kTiles; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = min(max(left - 4 * j, 0), 4);
            vw[i][j] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
          }
      }
    }
    bf16x8 pf[RT][2][Sh::kP];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float top = s[rt][0][0];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[rt][u][i]);
      top = query_max(top);
      // the maximum moves where it grows by 2^8 or more: weights stay below that, and sums in fp32 do not mind
      if (__any(top > m[rt] + 8.0f)) {
        const float to = top > m[rt] + 8.0f ? top : m[rt];
        const float less = to == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - to);
        m[rt] = to;
        l[rt] *= less;
#pragma unroll
        for (int i = 0; i < Sh::kTiles; ++i) o[rt][i] *= less;
      }
      const float base = m[rt] == kNegInf ? 0.0f : m[rt];
      float w[16], sum = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(s[rt][u][i] - base);
          sum += p;
          w[4 * u + i] = p * vs[u][i];
        }
      l[rt] += sum;
      if (masked) {                                     // an unseen token's scale may be anything
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(bits[rt] >> i & 1)) w[i] = 0.0f;
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = w[8 * kk + i];
        split<Sh::kP>(x, pf[rt][kk]);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const bf16x8 vf = widen<KIND>(vw[i][2 * kk], vw[i][2 * kk + 1]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int p = Sh::kP - 1; p >= 0; --p) o[rt][i] = mfma(vf, pf[rt][kk][p], o[rt][i]);
      }
    if (at < p1) load_values(page);
  }

  // the waves' sums, row tile by row tile
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = query_sum(l[rt]);
    if (g == 0) joined[wave][rt * 16 + r16] = float2{m[rt], l[rt]};
  }
  float* sums = (float*)lds;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    __syncthreads();                                    // the queries, or the last tile, have been read
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i)
      *(f32x4*)(sums + (wave * 16 + r16) * Sh::kRow + 16 * i + 4 * g) = o[rt][i];
    __syncthreads();
    const int mine = threadIdx.x >> 4, row = row0 + rt * 16 + mine;
    if (row < a.R) {
      const int t = row / a.G, h = row - t * a.G;
      float2 ml[kWaves];
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        ml[w] = t < rows ? joined[w][rt * 16 + mine] : float2{kNegInf, 0.0f};     // padding sees nothing
        top = fmaxf(top, ml[w].x);
      }
      float total = 0.0f, f[kWaves];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = share(ml[w].x, ml[w].y, top);
        total += f[w] * ml[w].y;
      }
      const bool last = a.splits == 1;
      const float inv = last ? (total == 0.0f ? 0.0f : 1.0f / total) : 1.0f;
      T* out = (T*)a.out + (((int64_t)b * c.T + t) * a.Hq + hk * a.G + h) * c.D;
      float* keep = a.part + (((int64_t)part * heads + bh) * a.R + row) * (c.D + 2);
      for (int ch = (int)threadIdx.x & 15; ch < c.D; ch += 16) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) x += f[w] == 0.0f ? 0.0f : f[w] * sums[(w * 16 + mine) * Sh::kRow + ch];
        if (last)
          out[ch] = (T)(x * inv);
        else
          keep[ch] = x;
      }
      if (!last && (threadIdx.x & 15) == 0) {
        keep[c.D] = top;
        keep[c.D + 1] = total;
      }
    }
  }
}

// Rows split over the pages, a wave a row.
template <typename T>
__global__ __launch_bounds__(256) void cache_attn_join(CacheAttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)a.c.B * a.c.Hk * a.R, at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (at >= n) return;
  const int D = a.c.D, stride = D + 2;
  const float* p = a.part + at * stride;
  const int64_t step = n * stride;
  float top = kNegInf;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, p[s * step + D]);
  for (int i = 32; i > 0; i /= 2) top = fmaxf(top, __shfl_xor(top, i));
  float x[2] = {0, 0}, total = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float l = p[s * step + D + 1], f = share(p[s * step + D], l, top);
    total += f * l;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64 * i < D && f != 0.0f) x[i] += f * p[s * step + lane + 64 * i];
  }
  const int64_t bh = at / a.R;
  const int row = (int)(at - bh * a.R), t = row / a.G, h = row - t * a.G;
  const int64_t b = bh / a.c.Hk, hk = bh - b * a.c.Hk;
  T* out = (T*)a.out + ((b * a.c.T + t) * a.Hq + hk * a.G + h) * D;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < D) out[lane + 64 * i] = (T)(x[i] * inv);
}

// Row tiles a workgroup holds.
int row_tiles(const CacheAttnArgs& a) {
  if (a.R <= 16) return 1;
  // fp32 (three parts a weight) and wide heads leave registers for two
  if (a.R <= 32 || a.elem_bytes == 4 || a.c.D > 64) return 2;
  return 4;
}

void set_splits(CacheAttnArgs& a) {
  a.row_blocks = (a.R + 16 * row_tiles(a) - 1) / (16 * row_tiles(a));
  const int64_t blocks = (int64_t)a.c.B * a.c.Hk * a.row_blocks;
  // two workgroups a CU, where every wave of each still has a page
  const int64_t want = blocks > 0 ? (512 + blocks - 1) / blocks : 1, most = (a.c.W + kWaves - 1) / kWaves;
  a.splits = (int)(want < most ? want : most);
  if (a.splits < 1) a.splits = 1;
}

template <typename T, int KIND, int DC>
void launch_rows(const CacheAttnArgs& a, unsigned blocks, hipStream_t stream) {
  switch (row_tiles(a)) {
    case 1: cache_attn<T, KIND, DC, 1><<<blocks, 64 * kWaves, 0, stream>>>(a); break;
    case 2: cache_attn<T, KIND, DC, 2><<<blocks, 64 * kWaves, 0, stream>>>(a); break;
    default:
      if constexpr (sizeof(T) == 2 && DC <= 64) cache_attn<T, KIND, DC, 4><<<blocks, 64 * kWaves, 0, stream>>>(a);
  }
}

template <typename T, int KIND>
void launch_width(const CacheAttnArgs& a, unsigned blocks, hipStream_t stream) {
  if (a.c.D <= 32)
    launch_rows<T, KIND, 32>(a, blocks, stream);
  else if (a.c.D <= 64)
    launch_rows<T, KIND, 64>(a, blocks, stream);
  else
    launch_rows<T, KIND, 128>(a, blocks, stream);
}

template <typename T>
hipError_t launch_type(const CacheAttnArgs& a, hipStream_t stream) {
  const unsigned blocks = (unsigned)((int64_t)a.c.B * a.c.Hk * a.row_blocks * a.splits);
  if (a.c.codes == FBEV_CODES_E4M3)
    launch_width<T, FBEV_CODES_E4M3>(a, blocks, stream);
  else
    launch_width<T, FBEV_CODES_INT8>(a, blocks, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.c.B * a.c.Hk * a.R;
  cache_attn_join<T><<<(unsigned)((rows + 3) / 4), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t cache_attention_workspace_bytes(const CacheAttnArgs& args) {
  CacheAttnArgs a = args;
  set_splits(a);
  if (a.splits == 1) return 0;
  return (size_t)a.splits * a.c.B * a.c.Hk * a.R * (a.c.D + 2) * sizeof(float);
}

hipError_t launch_cache_attention(CacheAttnArgs a, hipStream_t stream) {
  set_splits(a);
  return a.elem_bytes == 4 ? launch_type<float>(a, stream) : launch_type<__bf16>(a, stream);
}

}  // namespace fbev
