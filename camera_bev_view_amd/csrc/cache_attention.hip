// Attention of query tokens, a tree of drafted ones among others, over the token cache.
//
//   s_ij = scale q_i . (kc_j ks_j),  s = cap tanh(s / cap),  o_i = sum_j softmax_j(s) (vc_j vs_j)
//
// kc, vc: codes in 8 bits; ks, vs: a token's scales.  Codes of either format are bf16 numbers without rounding, so the
// matrix products run on bf16 codes while the scales join in fp32: ks multiplies the score, vs the weight.  What is not
// exact in bf16 goes in as parts: fp32 queries and weights as three (24 bits), the weights of bf16 tensors as two (16 bits:
// one would add as much error as the result's own rounding), bf16 queries as they are.
//
// Both products have the tokens (or channels) as the matrix instruction's rows and 16 queries (times heads of a key head, a
// row tile) as its columns, a page of 64 tokens at a time:
//   S^T = K Q^T:  lane (r, g) of r = lane mod 16, g = lane / 16 takes 16 codes (channels 16 g ..) of token 16 (r / 4) + 4 u + r mod 4,
//                 u = 0 .. 3, so that the result leaves it the scores of tokens 16 g .. 16 g + 15 of query r;
//   O^T = V^T P^T: those 16 weights are its operand as they stand, and the values, kept with their tokens side by side, are
//                 16 codes (tokens 16 g ..) of channel r.
//
// Two forms.  Up to one row tile (serving) memory bounds the call: every wave takes pages of its own, straight into the
// registers that feed the matrix instructions, a page's keys while the one before is in its softmax and second product,
// its values under the first one.  With more row tiles the arithmetic does: the waves of a workgroup hold row tiles of their
// own and share every page, which they widen to bf16 once, a part each, into LDS, one page ahead.  Few rows over many pages
// are split over workgroups as well, and a second launch joins them.
//
// One token of each of 32 sequences (8192 to 4096 tokens, 32 heads over 8 of 128, e4m3): 83 us, 420 MB at 5.1 TB/s, the copy's
// rate.  60 rows over 200000 tokens of 2 heads of 64 (int8, 51 MB): 27 us and 5 for the join of 128 splits; fetching one hot
// page instead changes nothing.  2 x 4000 rows behind 6000 and 4500 tokens, 4 heads of
// 128: 177 us, of which the matrix units are busy 57 and vector instructions issue 84 (a quarter more with the exponentials); LDS
// reads take 58.  They hide each other little: all of a workgroup's waves come to the same stage together.  fp32 (three parts for
// queries and weights) does the 64 tokens of 16 scenes at 128 us against 73 in bf16.
#include <hip/hip_runtime.h>

#include "attention_core.h"
#include "codes.h"
#include "decoder.h"
#include "encoder.h"
#include "wave_ops.h"

namespace fbev {
namespace {

constexpr int kMostSplits = 512;

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
template <typename T, int DC>
struct Shape {
  static constexpr int kQ = sizeof(T) == 4 ? 3 : 1;     // parts of a query
  static constexpr int kP = sizeof(T) == 4 ? 3 : 2;     // parts of a weight
  static constexpr int kSteps = DC / 32;                // of the first product
  static constexpr int kChunk = DC >= 64 ? 16 : 8;      // bytes a lane takes of a key at a time
  static constexpr int kChunks = DC >= 64 ? DC / 64 : 1;
  static constexpr int kTiles = DC / 16;                // of the second product's rows
  static constexpr int kRow = DC + 4;                   // floats of a row in the join
};

// A call's rows of one sequence and key head, as a workgroup sees them.
struct Part {
  int b, hk, bh, split;
  int row0;               // first row
  int start, rows;        // tokens in the cache; rows that are no padding
  int end;                // tokens that any of the workgroup's rows sees
  int p0, p1;             // its pages
};

// APART: what follows on an XCD lies eight apart.  Sequences differ in length, and all heads of a long one on one XCD would
// outlast the others (8 x 4000 rows behind 3000 to 1500 tokens: 316 us against 360).  Not where every workgroup has a CU
// and pages of its own (32 sequences of 8192 to 4096 tokens: 89 us against 87).
template <bool APART>
__device__ __forceinline__ Part find_part(const CacheAttnArgs& a, int rows_held) {
  const CacheArgs& c = a.c;
  Part p;
  int id = xcd_block(blockIdx.x, gridDim.x);
  const int rb = id % a.row_blocks;
  id /= a.row_blocks;
  if constexpr (APART) {
    const int n = c.B * c.Hk * a.splits, q = n / 8, r = n % 8, more = r * (q + 1);
    const int x = id < more ? id / (q + 1) : r + (id - more) / max(q, 1);
    id = 8 * (id < more ? id - x * (q + 1) : id - more - (x - r) * q) + x;
  }
  p.split = id % a.splits;
  p.bh = id / a.splits;
  p.b = p.bh / c.Hk;
  p.hk = p.bh % c.Hk;
  p.row0 = (a.row_blocks - 1 - rb) * rows_held;         // the last rows see most: they begin first
  p.start = min(c.start[p.b], c.W * kPage);             // (what lies beyond the table does not exist)
  p.rows = p.start < 0 ? 0 : min(c.count ? max(c.count[p.b], 0) : c.T, c.T);
  const int last_t = (min(p.row0 + rows_held, a.R) - 1) / a.G;
  p.end = p.rows > 0 ? (int)visible_end(a, p.start, p.rows, last_t) : 0;
  const int pages = (p.end + kPage - 1) / kPage;
  const int each = pages / a.splits, rest = pages % a.splits;
  p.p0 = each * p.split + rest * p.split / a.splits;
  p.p1 = each * (p.split + 1) + rest * (p.split + 1) / a.splits;
  return p;
}

// Walks the pages p0, p0 + STEP, .. of a part that exist.  A wave reads 64 of the table's entries at a time: one entry a page
// would put a whole memory latency in front of each page's loads.
template <int STEP>
struct Walk {
  const int32_t* table;
  int end, pages;
  int at, page = 0;       // the current page's place in the sequence (end: none) and its number
  int first, ids;         // lane i: table[first + STEP i]

  __device__ __forceinline__ Walk(const CacheArgs& c, const Part& p, int from)
      : table(c.table + (int64_t)p.b * c.W), end(p.p1), pages(c.pages), at(from - STEP), first(from) {
    fetch();
    next();
  }
  __device__ __forceinline__ void fetch() {
    const int i = first + STEP * ((int)threadIdx.x & 63);
    ids = i < end ? table[i] : -1;
  }
  __device__ __forceinline__ void next() {
    for (at += STEP; at < end; at += STEP) {
      if (at >= first + 64 * STEP) {
        first = at;
        fetch();
      }
      page = __builtin_amdgcn_readlane(ids, (at - first) / STEP);
      if (page >= 0 && page < pages) return;
    }
    at = end;
  }
  __device__ __forceinline__ bool there() const { return at < end; }
};

// A row tile's queries as the first product's columns: step 2 c + h of lane group g has channels 64 c + 16 g + 8 h ..
// (8 g .. where one step is all).
template <typename T, int DC>
__device__ __forceinline__ void load_queries(const CacheAttnArgs& a, const Part& p, int row, int step, int g,
                                             bf16x8 (&parts)[Shape<T, DC>::kQ]) {
  using Sh = Shape<T, DC>;
  const int t = row / a.G, h = row - t * a.G;
  const int ch = Sh::kChunk == 16 ? (step >> 1) * 64 + g * 16 + (step & 1) * 8 : g * 8;
  const int left = row < a.R ? a.c.D - ch : 0;
  const T* q = (const T*)a.q + p.b * a.qs[0] + (int64_t)t * a.qs[1] + (int64_t)(p.hk * a.G + h) * a.qs[2] + ch;
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
  split<Sh::kQ>(x, parts);
}

// A page's codes and scales of one key head, as buffers: what lies outside reads as zero, all of it where there is no
// page.  So loads need no branches, whose joins would make the compiler wait for them on the spot.
struct Page {
  __amdgpu_buffer_rsrc_t k, v, ks, vs;
};

constexpr int kNowhere = 0x7fffff00;                    // an offset outside every page

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

__device__ __forceinline__ Page find_page(const CacheArgs& c, int hk, int page, bool there) {
  const int64_t at = there ? (int64_t)page * c.Hk + hk : 0;
  const int codes = there ? kPage * c.Dp : 0, scales = there ? kPage * 4 : 0;
  Page p;
  p.k = buffer_of((const uint8_t*)c.k + at * kPage * c.Dp, codes);
  p.v = buffer_of((const uint8_t*)c.v + at * kPage * c.Dp, codes);
  p.ks = buffer_of(c.k_scale + at * kPage, scales);
  p.vs = buffer_of(c.v_scale + at * kPage, scales);
  return p;
}

// Key codes of the token 16 (r / 4) + 4 u + r mod 4 of a page, channels 64 i + 16 g .. (8 g .. where eight are a lane's).
template <typename Sh>
__device__ __forceinline__ void load_key(const CacheArgs& c, const Page& p, int r16, int g, int u, int i,
                                         uint32_t (&kw)[4]) {
  const int ch = 64 * i + Sh::kChunk * g;
  const int at = ch < c.Dp && u < 4 ? (16 * (r16 >> 2) + (r16 & 3) + 4 * u) * c.Dp + ch : kNowhere;
  if constexpr (Sh::kChunk == 16) {
    const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(p.k, at, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) kw[j] = x[j];
  } else {
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(p.k, at, 0, 0);
    kw[0] = x[0];
    kw[1] = x[1];
  }
}

// Value codes of channel 16 i + r, tokens 16 g .. 16 g + 15.
__device__ __forceinline__ void load_value(const Page& p, int r16, int g, int i, uint32_t (&vw)[4]) {
  const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(p.v, (16 * i + r16) * kPage + 16 * g, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) vw[j] = x[j];
}

// Scales of the tokens 16 g .. 16 g + 15.
__device__ __forceinline__ void load_scales(__amdgpu_buffer_rsrc_t p, int g, float (&x)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(p, 64 * g + 16 * u, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * u + j] = __builtin_bit_cast(float, (uint32_t)w[j]);
  }
}

// Clears the codes behind the first `left` of 16: what was never written may be the code of a NaN.
template <int KIND>
__device__ __forceinline__ void keep_codes(uint32_t (&w)[4], int left) {
  if constexpr (KIND != FBEV_CODES_E4M3) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = min(max(left - 4 * j, 0), 4);
    w[j] &= n == 4 ? ~0u : (1u << (8 * n)) - 1u;
  }
}

// What a row's scores are taken against: its running maximum, once there is one.
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.0f : m; }

// A score from a product and its token's scale: against the base in base-2 units, or, with a cap, divided by the cap (the base
// comes off behind the tanh).
__device__ __forceinline__ float score(float acc, float scale, bool capped, float base) {
  return fmaf(acc, scale, capped ? 0.0f : -base);
}

// Scores to weights, in parts, for one row tile and page; m, l, o: the row's running maximum, this lane's share of the sum of
// weights, and the sums.  `s`: of score(); vs(kk, x): scales of the lane's tokens 8 kk .. 8 kk + 7.
template <int KP, int TILES, typename F>
__device__ __forceinline__ void weigh(float (&s)[16], F vs, bool masked, uint32_t bits, float cap, float& m, float& l,
                                      f32x4 (&o)[TILES], bf16x8 (&pf)[2][KP]) {
  const float base = base_of(m);
  if (cap > 0) {
    const float top = cap * kLog2e;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = fmaf(top, tanh_fast<true>(s[i]), -base);
  }
  if (masked) {
    const uint32_t seen = opaque(bits);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(seen >> i & 1)) s[i] = kNegInf;
  }
  float x[2][8];
  vs(0, x[0]);
  float top = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
  top = query_max(top);
  // the maximum moves where it grows by 2^8 or more: weights stay below that, for which room_for() leaves room
  const bool moves = top > (m == kNegInf ? kNegInf : 8.0f);
  if (__any(moves)) {
    const float to = moves ? base + top : m, by = moves ? to - base : 0.0f;
    const float less = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(-by);
    m = to;
    l *= less;
#pragma unroll
    for (int i = 0; i < TILES; ++i) o[i] *= less;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] -= by;
  }
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    if (kk == 0) vs(1, x[1]);                           // under the first half's work
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __builtin_amdgcn_exp2f(s[8 * kk + i]);
      sum[i & 1] += p;
      x[kk][i] *= p;
    }
    l += sum[0] + sum[1];
    if (masked) {                                       // an unseen token's scale may be anything
      const uint32_t seen = opaque(bits >> (8 * kk));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(seen >> i & 1)) x[kk][i] = 0.0f;
    }
    split<KP>(x[kk], pf[kk]);
  }
}

// Eight neighbouring channels (from 8 `lane` on, 16 lanes a row) of a row's results from what N sums hold of it: sums[w] + 8
// lane, their maxima and sums of weights in ml.
template <typename T, int N>
__device__ __forceinline__ void finish_row(const CacheAttnArgs& a, const Part& p, int row, const float2 (&ml)[N],
                                           const float* const (&sums)[N], int lane) {
  const CacheArgs& c = a.c;
  const int t = row / a.G, h = row - t * a.G;
  const bool seen = t < p.rows;                         // padding sees nothing
  float top = kNegInf;
#pragma unroll
  for (int w = 0; w < N; ++w) top = fmaxf(top, seen ? ml[w].x : kNegInf);
  float total = 0.0f, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int ch = 8 * lane, left = c.D - ch;
  if (left <= 0) return;
#pragma unroll
  for (int w = 0; w < N; ++w) {
    const float f = seen ? share(ml[w].x, ml[w].y, top) : 0.0f;
    if (f == 0.0f) continue;
    total += f * ml[w].y;
    const f32x4 lo = *(const f32x4*)(sums[w] + ch), hi = *(const f32x4*)(sums[w] + ch + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += f * (i < 4 ? lo[i] : hi[i - 4]);
  }
  if (a.splits == 1) {
    const float inv = total == 0.0f ? 0.0f : 1.0f / (total * a.down);
    T* out = (T*)a.out + (((int64_t)p.b * c.T + t) * a.Hq + p.hk * a.G + h) * c.D + ch;
    T y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (T)(x[i] * inv);
    if (left >= 8) {
      __builtin_memcpy(out, y, sizeof y);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) out[i] = y[i];
    }
  } else {
    float* keep = a.part + (((int64_t)p.split * c.B * c.Hk + p.bh) * a.R + row) * (c.D + 2);
    if (left >= 8) {
      __builtin_memcpy(keep + ch, x, sizeof x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) keep[ch + i] = x[i];
    }
    if (lane == 0) {
      keep[c.D] = top;
      keep[c.D + 1] = total;
    }
  }
}

// What values are scaled by until a row is finished, a power of two: sums of the table's tokens at weights of up to 2^8 (what
// weigh() lets them grow to) stay below 2^127 for values of any size.
float room_for(int W) {
  int tokens = 6;                                       // log2 of them, rounded up
  while (((int64_t)1 << tokens) < (int64_t)W * kPage) ++tokens;
  return ldexpf(1.0f, -(9 + tokens));
}

// Up to 16 rows: every wave has pages of its own.
template <typename T, int KIND, int DC, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void cache_attn_few(CacheAttnArgs a) {
  using Sh = Shape<T, DC>;
  constexpr int kQBytes = Sh::kSteps * Sh::kQ * 64 * 16, kSumBytes = WAVES * 16 * Sh::kRow * 4;
  __shared__ alignas(16) char lds[kQBytes > kSumBytes ? kQBytes : kSumBytes];
  __shared__ float2 joined[WAVES][16];
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Part p = find_part<WAVES == 4>(a, 16);
  if (wave < Sh::kSteps) {
    bf16x8 parts[Sh::kQ];
    load_queries<T, DC>(a, p, p.row0 + r16, wave, g, parts);
#pragma unroll
    for (int i = 0; i < Sh::kQ; ++i) ((bf16x8*)lds)[(wave * Sh::kQ + i) * 64 + lane] = parts[i];
  }
  __syncthreads();

  f32x4 o[Sh::kTiles];
  float m = kNegInf, l = 0.0f;
#pragma unroll
  for (int i = 0; i < Sh::kTiles; ++i) o[i] = f32x4{0, 0, 0, 0};
  uint32_t kw[4][Sh::kChunks][4], vw[Sh::kTiles][4];
  float ks[16], vs[16];
  const auto load_keys = [&](const Page& page) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < Sh::kChunks; ++i) load_key<Sh>(c, page, r16, g, u, i, kw[u][i]);
    load_scales(page.ks, g, ks);
  };
  const auto load_values = [&](const Page& page) {
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i) load_value(page, r16, g, i, vw[i]);
    load_scales(page.vs, g, vs);
  };
  const float unit = a.cap > 0 ? a.scale / a.cap : a.scale * kLog2e;
  const int whole = a.mode == FBEV_DRAFT_NONE ? p.end : min(p.start, p.end);      // tokens below are seen by all
  const int t = (p.row0 + r16) / a.G;
  Walk<WAVES> walk(c, p, p.p0 + wave);
  Page page = find_page(c, p.hk, walk.page, walk.there());
  load_keys(page);
  load_values(page);
  while (walk.there()) {
    const float base = base_of(m);
    float s[16];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < Sh::kSteps; ++i) {
        const bf16x8 kf = widen<KIND>(kw[u][i / 2][2 * (i % 2)], kw[u][i / 2][2 * (i % 2) + 1]);
#pragma unroll
        for (int q = Sh::kQ - 1; q >= 0; --q) acc = mfma(kf, ((const bf16x8*)lds)[(i * Sh::kQ + q) * 64 + lane], acc);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[4 * u + i] = score(acc[i], unit * ks[4 * u + i], a.cap > 0, base);
    }
    const int pos = walk.at * kPage;
    walk.next();
    page = find_page(c, p.hk, walk.page, walk.there());
    load_keys(page);
    const bool masked = pos + kPage > whole;
    uint32_t bits = 0;
    if (masked) {
      bits = t < p.rows ? seen_bits(a, p.b, t, p.start, p.rows, pos + 16 * g) : 0;
#pragma unroll
      for (int i = 0; i < Sh::kTiles; ++i) keep_codes<KIND>(vw[i], p.end - pos - 16 * g);
    }
    bf16x8 pf[2][Sh::kP];
    weigh<Sh::kP, Sh::kTiles>(
        s,
        [&](int kk, float(&x)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = vs[8 * kk + i] * a.down;
        },
        masked, bits, a.cap, m, l, o, pf);
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const bf16x8 vf = widen<KIND>(vw[i][2 * kk], vw[i][2 * kk + 1]);
#pragma unroll
        for (int q = Sh::kP - 1; q >= 0; --q) o[i] = mfma(vf, pf[kk][q], o[i]);
      }
    load_values(page);
  }

  l = query_sum(l);
  if (g == 0) joined[wave][r16] = float2{m, l};
  float* sums = (float*)lds;
  __syncthreads();                                      // the queries have been read
#pragma unroll
  for (int i = 0; i < Sh::kTiles; ++i) *(f32x4*)(sums + (wave * 16 + r16) * Sh::kRow + 16 * i + 4 * g) = o[i];
  __syncthreads();
  const int mine = threadIdx.x >> 4, row = p.row0 + mine;
  if (mine >= 16 || row >= a.R) return;
  float2 ml[WAVES];
  const float* of[WAVES];
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    ml[w] = joined[w][mine];
    of[w] = sums + (w * 16 + mine) * Sh::kRow;
  }
  finish_row<T>(a, p, row, ml, of, r16);
}

// More rows: every wave has a row tile of its own, the pages are shared.  GROUPS of waves have the same row tiles and take turns
// at the pages.  SIMD_WAVES: waves a SIMD that the registers are meant for.
template <typename T, int KIND, int DC, int WAVES, int GROUPS, int SIMD_WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(SIMD_WAVES, SIMD_WAVES))) void cache_attn_many(CacheAttnArgs a) {
  using Sh = Shape<T, DC>;
  constexpr int kKeys = 4 * Sh::kSteps, kFrags = kKeys + 2 * Sh::kTiles;          // of a widened page
  constexpr int kPageBytes = kFrags * 64 * 16, kSumBytes = WAVES * 16 * Sh::kRow * 4;
  constexpr int kHeldBytes = GROUPS * 2 * kPageBytes;
  __shared__ alignas(16) char lds[kHeldBytes > kSumBytes ? kHeldBytes : kSumBytes];
  __shared__ alignas(16) float all_scales[GROUPS][2][2][kPage];
  __shared__ float2 joined[GROUPS == 1 ? 1 : WAVES][16];
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  constexpr int kTileWaves = WAVES / GROUPS;
  const int group = GROUPS == 1 ? 0 : wave / kTileWaves, tile = wave - group * kTileWaves;
  const Part p = find_part<true>(a, 16 * kTileWaves);
  const int row0 = p.row0 + tile * 16;
  char* const pages = lds + group * 2 * kPageBytes;
  float(&scales)[2][2][kPage] = all_scales[group];
  const bool idle = row0 >= a.R;                        // it moves pages for the others
  bf16x8 qf[Sh::kSteps][Sh::kQ];
  f32x4 o[Sh::kTiles];
  float m = kNegInf, l = 0.0f;
#pragma unroll
  for (int i = 0; i < Sh::kSteps; ++i) load_queries<T, DC>(a, p, row0 + r16, i, g, qf[i]);
#pragma unroll
  for (int i = 0; i < Sh::kTiles; ++i) o[i] = f32x4{0, 0, 0, 0};

  // a wave's part of a page: pieces of 16 codes a lane, keys (u and chunk) from the first wave on, value tiles from the last
  constexpr int kKeyPieces = 4 * Sh::kChunks, kKeyMine = (kKeyPieces + kTileWaves - 1) / kTileWaves;
  constexpr int kValueMine = (Sh::kTiles + kTileWaves - 1) / kTileWaves;
  uint32_t kw[kKeyMine][4], vw[kValueMine][4];
  float scale = 0.0f;
  const int back = kTileWaves - 1 - tile;
  const auto load_page = [&](int number, bool there) {
    const Page page = find_page(c, p.hk, number, there);
#pragma unroll
    for (int j = 0; j < kKeyMine; ++j) {
      const int piece = tile + kTileWaves * j;          // (one behind the last is outside the page)
      load_key<Sh>(c, page, r16, g, piece / Sh::kChunks, piece % Sh::kChunks, kw[j]);
    }
#pragma unroll
    for (int j = 0; j < kValueMine; ++j) load_value(page, r16, g, back + kTileWaves * j, vw[j]);
    scale = __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(tile & 1 ? page.vs : page.ks, 4 * lane, 0, 0));
  };
  const float unit = a.cap > 0 ? a.scale / a.cap : a.scale * kLog2e;
  const auto put_page = [&](int buf, int pos) {
    bf16x8* to = (bf16x8*)(pages + buf * kPageBytes) + lane;
#pragma unroll
    for (int j = 0; j < kKeyMine; ++j) {
      const int piece = tile + kTileWaves * j;
      if (kKeyPieces % kTileWaves == 0 || piece < kKeyPieces) {
        const int u = piece / Sh::kChunks, i = piece % Sh::kChunks;
        to[(u * Sh::kSteps + 2 * i) * 64] = widen<KIND>(kw[j][0], kw[j][1]);
        if constexpr (Sh::kChunk == 16) to[(u * Sh::kSteps + 2 * i + 1) * 64] = widen<KIND>(kw[j][2], kw[j][3]);
      }
    }
#pragma unroll
    for (int j = 0; j < kValueMine; ++j) {
      const int rows = back + kTileWaves * j;
      if (Sh::kTiles % kTileWaves == 0 || rows < Sh::kTiles) {
        if (pos + kPage > p.end) keep_codes<KIND>(vw[j], p.end - pos - 16 * g);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) to[(kKeys + 2 * rows + kk) * 64] = widen<KIND>(vw[j][2 * kk], vw[j][2 * kk + 1]);
      }
    }
    if (tile < 2) scales[buf][tile][lane] = scale * (tile ? a.down : unit);
  };

  const int whole = a.mode == FBEV_DRAFT_NONE ? p.end : min(p.start, p.end);      // tokens below are seen by all
  Walk<GROUPS> walk(c, p, p.p0 + group);                // the page ahead of the one at work
  int at = walk.at, buf = 0;
  load_page(walk.page, walk.there());
  put_page(0, at * kPage);
  walk.next();
  load_page(walk.page, walk.there());
  // (groups may find different numbers of pages that exist: all go round as often as one could have to)
  const int rounds = (p.p1 - p.p0 + GROUPS - 1) / GROUPS;
  for (int round = 0; GROUPS == 1 ? at < p.p1 : round < rounds; ++round) {
    const int pos = at * kPage;
    const bool here = GROUPS == 1 || at < p.p1;
    __syncthreads();                                    // this page is in; the other buffer has been read
    const bf16x8* from = (const bf16x8*)(pages + buf * kPageBytes) + lane;
    const float(&sc)[2][kPage] = scales[buf];
    at = walk.at;
    buf ^= 1;
    put_page(buf, at * kPage);                          // (behind the last one: zeros that nobody reads)
    walk.next();
    load_page(walk.page, walk.there());
    if (idle || !here) continue;
    const bool masked = pos + kPage > whole;
    uint32_t bits = 0;
    if (masked) {
      const int t = (int)(opaque(row0 + r16) / (uint32_t)a.G);
      if (t < p.rows) bits = seen_bits(a, p.b, t, p.start, p.rows, pos + 16 * g);
    }
    const float base = base_of(m);
    float s[16];
    {
      float ks[16];
      __builtin_memcpy(ks, __builtin_assume_aligned(&sc[0][16 * g], 16), 64);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Sh::kSteps; ++i) {
          const bf16x8 kf = from[(u * Sh::kSteps + i) * 64];
#pragma unroll
          for (int q = Sh::kQ - 1; q >= 0; --q) acc = mfma(kf, qf[i][q], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * u + i] = score(acc[i], ks[4 * u + i], a.cap > 0, base);
      }
    }
    bf16x8 pf[2][Sh::kP];
    weigh<Sh::kP, Sh::kTiles>(
        s, [&](int kk, float(&x)[8]) { __builtin_memcpy(x, __builtin_assume_aligned(&sc[1][16 * g + 8 * kk], 16), 32); },
        masked, bits, a.cap, m, l, o, pf);
#pragma unroll
    for (int i = 0; i < Sh::kTiles; ++i)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const bf16x8 vf = from[(kKeys + 2 * i + kk) * 64];
#pragma unroll
        for (int q = Sh::kP - 1; q >= 0; --q) o[i] = mfma(vf, pf[kk][q], o[i]);
      }
  }

  // a row's channels side by side again, by way of the pages' LDS
  float* sums = (float*)lds + wave * 16 * Sh::kRow;
  l = query_sum(l);
  if (GROUPS > 1 && g == 0) joined[wave][r16] = float2{m, l};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < Sh::kTiles; ++i) *(f32x4*)(sums + r16 * Sh::kRow + 16 * i + 4 * g) = o[i];
  if constexpr (GROUPS == 1) {
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float2 ml[1] = {float2{__shfl(m, i + g), __shfl(l, i + g)}};
      const float* const of[1] = {sums + (i + g) * Sh::kRow};
      const int row = row0 + i + g;
      if (row < a.R) finish_row<T>(a, p, row, ml, of, r16);
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16 / GROUPS; i += 4) {
      const int mine = wave * (16 / GROUPS) + i + g, from = mine / 16, r = mine % 16, row = p.row0 + mine;
      float2 ml[GROUPS];
      const float* of[GROUPS];
#pragma unroll
      for (int n = 0; n < GROUPS; ++n) {
        ml[n] = joined[from + n * kTileWaves][r];
        of[n] = (const float*)lds + ((from + n * kTileWaves) * 16 + r) * Sh::kRow;
      }
      if (row < a.R) finish_row<T>(a, p, row, ml, of, r16);
    }
  }
}

// Rows split into up to N parts: 32 lanes a row, four channels each, all parts' loads in flight.
template <typename T, int N>
__global__ __launch_bounds__(256) void cache_attn_join_few(CacheAttnArgs a) {
  const int64_t n = (int64_t)a.c.B * a.c.Hk * a.R, at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int D = a.c.D, ch = 4 * ((int)threadIdx.x & 31), left = D - ch;
  if (at >= n || left <= 0) return;
  const float* p = a.part + at * (D + 2);
  const int64_t step = n * (D + 2);
  float2 ml[N];
  float x[N][4];
  float top = kNegInf;
#pragma unroll
  for (int s = 0; s < N; ++s) {
    ml[s] = float2{kNegInf, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[s][i] = 0.0f;
    if (s < a.splits) {
      ml[s] = float2{p[s * step + D], p[s * step + D + 1]};
      if (left >= 4) {
        __builtin_memcpy(x[s], p + s * step + ch, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) x[s][i] = p[s * step + ch + i];
      }
    }
    top = fmaxf(top, ml[s].x);
  }
  float total = 0.0f, y[4] = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < N; ++s) {
    const float f = share(ml[s].x, ml[s].y, top);
    if (f == 0.0f) continue;
    total += f * ml[s].y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += f * x[s][i];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / (total * a.down);
  const int64_t bh = at / a.R;
  const int row = (int)(at - bh * a.R), t = row / a.G, h = row - t * a.G;
  const int64_t b = bh / a.c.Hk, hk = bh - b * a.c.Hk;
  T* out = (T*)a.out + ((b * a.c.T + t) * a.Hq + hk * a.G + h) * D + ch;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) out[i] = (T)(y[i] * inv);
}

// Rows split into many, a workgroup a row.  A wave takes every waves-th split, kHeld at a time; the first are on their way
// before anything of the shares is known, so a call of up to 256 splits waits for memory once.
template <typename T>
__global__ __launch_bounds__(1024) void cache_attn_join(CacheAttnArgs a) {
  constexpr int kHeld = 16;
  __shared__ float2 shares[kMostSplits];                // maximum and sum, then the share
  __shared__ float sums[16][128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t n = (int64_t)a.c.B * a.c.Hk * a.R, at = blockIdx.x;
  const int D = a.c.D, stride = D + 2;
  const float* p = a.part + at * stride;
  const int64_t step = n * stride;
  float held[kHeld][2];
  const auto load = [&](int s0) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int s = s0 + j * waves;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        held[j][i] = s < a.splits && lane + 64 * i < D ? p[s * step + lane + 64 * i] : 0.0f;
    }
  };
  load(wave);
  for (int s = threadIdx.x; s < a.splits; s += blockDim.x) shares[s] = float2{p[s * step + D], p[s * step + D + 1]};
  __syncthreads();
  // every wave finds the maximum and the total for itself
  float top = kNegInf;
  for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, shares[s].x);
#pragma unroll
  for (int i = 32; i > 0; i /= 2) top = fmaxf(top, __shfl_xor(top, i));
  float total = 0.0f;
  for (int s = lane; s < a.splits; s += 64) total += share(shares[s].x, shares[s].y, top) * shares[s].y;
  total = wave_sum(total);
  float x[2] = {0, 0};
  for (int s0 = wave; s0 < a.splits; s0 += kHeld * waves) {
    if (s0 != wave) load(s0);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int s = s0 + j * waves;
      const float2 ml = shares[s < a.splits ? s : 0];
      const float f = s < a.splits ? share(ml.x, ml.y, top) : 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] += f == 0.0f ? 0.0f : f * held[j][i];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) sums[wave][lane + 64 * i] = x[i];
  __syncthreads();
  const int ch = threadIdx.x;
  if (ch >= D) return;
  float y = 0.0f;
  for (int w = 0; w < waves; ++w) y += sums[w][ch];
  const int64_t bh = at / a.R;
  const int row = (int)(at - bh * a.R), t = row / a.G, h = row - t * a.G;
  const int64_t b = bh / a.c.Hk, hk = bh - b * a.c.Hk;
  ((T*)a.out)[((b * a.c.T + t) * a.Hq + hk * a.G + h) * D + ch] = (T)(total == 0.0f ? 0.0f : y / (total * a.down));
}

// How a call's rows lie on workgroups.
struct Plan {
  bool few;               // up to one row tile: waves with pages of their own
  int waves;              // that hold different rows (few: all)
  int groups;             // of waves with the same rows
  int row_blocks, splits;
};

// Few rows: eight waves where that alone gives most CUs a workgroup (192 of 256; no split, no join: 32 sequences of 4000 tokens, 8
// key heads of 128, 46 us against 52 with four waves and two splits; 28 x 8 heads 42 against 47, 20 x 8 heads 37 either way), else
// four and splits (one sequence of 4000 tokens, 8 heads of 64: 10 us against 21).  More rows: up to 64 in four waves' tiles, two
// groups of those to a workgroup, which halves what a join reads (15 drafted tokens over 200000: 34 us against 38 with a
// group and twice the splits), four in long caches where their registers and LDS let 16 waves in (32 us; 40 sequences of 32
// rows over 1000 tokens 28 against 23).  Heads of 128 in two groups hold 134 KB of LDS: a workgroup a CU, two waves a SIMD (16
// scenes of 16 drafted tokens x 16 over 4 heads behind 4096 to 2176 tokens 33 us, where bytes would take 11).  Beyond, eight tiles
// share the widening of a page (64 rows of 16 scenes x 4 heads of 128: 73 us against 116).
//
// Splits make up 512 workgroups of few rows, 256 of more (900 rows of 8 heads of 32 over 3600 tokens: 28 us against 37 with
// 512, in fp32 32 against 41), or 512 where a CU holds two (bf16) and either a wave's work on a page is long (heads of 128: 1000
// rows of 16 heads behind 9000 tokens 153 us against 164) or each has a dozen pages and there are half a workgroup a CU
// without a split (4 x 900 rows of 8 heads of 32 over 3600 tokens 59 us against 72, 16 x 32 rows of 8 heads of 64 over 4000 28 against
// 33, 20 x 32 rows over 6000 45 against 51; 12 x 32 would win too, 36 against 39; 32 rows of 8 heads over 1000 28 against 23).  Calls that come near those numbers unsplit
// are not split in two, where that would leave CUs with one and two parts: from 384 workgroups of 512 on (448 of 128 rows over 2000
// tokens 106 us against 122 split, over 8000 330 against 324; 320 of them 102 against 100 unsplit and 248 against 287), from 192 of
// 256 where waves share pages (fp32: 224 over 2000 tokens 100 against 103, over 6000 251 against 214; 160 of them 95 against 103
// unsplit and 187 against 250), always below 256 where groups take turns (240 over 2000 tokens 46 against 40 unsplit, over
// 6000 97 against 104).  Every workgroup still has four pages.
//
// All of that goes by the table's width, which the host knows, and not by what the sequences hold: a table far wider than
// they need costs splits without a page and a join of them (8 tokens over 500 tokens each, 4 heads: 9.5 us behind a table of 8
// pages, 11.5 behind one of 1024).
Plan plan_of(const CacheAttnArgs& a) {
  Plan p;
  const int64_t heads = (int64_t)a.c.B * a.c.Hk;
  p.few = a.R <= 16;
  p.waves = (p.few ? heads >= 192 : a.R > 64) ? 8 : 4;
  const int held = p.few ? 16 : 16 * p.waves;
  p.row_blocks = (a.R + held - 1) / held;
  const bool half = a.elem_bytes == 2, wide = a.c.D > 64;
  const int64_t blocks = heads * p.row_blocks, most = (a.c.W + 3) / 4, twice = (512 + blocks - 1) / (blocks > 0 ? blocks : 1);
  const bool two = p.few || (half && (wide ? p.waves == 8 : blocks >= 128 && a.c.W >= 12 * twice));
  int64_t want = 1;
  if (p.few ? p.waves == 4 : blocks < (two ? 384 : p.waves == 4 ? 256 : 192)) want = two ? twice : (256 + blocks - 1) / blocks;
  if (want > most) want = most;
  p.splits = (int)(want < 1 ? 1 : want > kMostSplits ? kMostSplits : want);
  p.groups = p.few || p.waves == 8 ? 1 : half && a.c.D <= 64 && blocks <= 64 && a.c.W >= 20 * p.splits ? 4 : 2;
  return p;
}

template <typename T, int KIND, int DC>
void launch_rows(const CacheAttnArgs& a, const Plan& plan, unsigned blocks, hipStream_t stream) {
  if (plan.few) {
    if (plan.waves == 8)
      cache_attn_few<T, KIND, DC, 8><<<blocks, 512, 0, stream>>>(a);
    else
      cache_attn_few<T, KIND, DC, 4><<<blocks, 256, 0, stream>>>(a);
  } else if (plan.groups == 4) {
    if constexpr (sizeof(T) == 2 && DC < 128) cache_attn_many<T, KIND, DC, 16, 4, 4><<<blocks, 1024, 0, stream>>>(a);
  } else if (plan.groups == 2) {
    cache_attn_many<T, KIND, DC, 8, 2, sizeof(T) == 2 && DC < 128 ? 4 : 2><<<blocks, 512, 0, stream>>>(a);
  } else {
    // bf16 takes tighter code that leaves four waves a SIMD (8 x 4000 rows of 128 channels: 371 us against 450; 25 x 256 rows:
    // 89 against 102; 2 x 1200 rows, a workgroup on every third CU: 25.0 against 24.3); fp32's parts of queries do not fit
    cache_attn_many<T, KIND, DC, 8, 1, sizeof(T) == 2 ? 4 : 2><<<blocks, 512, 0, stream>>>(a);
  }
}

template <typename T, int KIND>
void launch_width(const CacheAttnArgs& a, const Plan& plan, unsigned blocks, hipStream_t stream) {
  if (a.c.D <= 32)
    launch_rows<T, KIND, 32>(a, plan, blocks, stream);
  else if (a.c.D <= 64)
    launch_rows<T, KIND, 64>(a, plan, blocks, stream);
  else
    launch_rows<T, KIND, 128>(a, plan, blocks, stream);
}

template <typename T>
hipError_t launch_type(const CacheAttnArgs& a, const Plan& plan, hipStream_t stream) {
  const unsigned blocks = (unsigned)((int64_t)a.c.B * a.c.Hk * a.row_blocks * a.splits);
  if (a.c.codes == FBEV_CODES_E4M3)
    launch_width<T, FBEV_CODES_E4M3>(a, plan, blocks, stream);
  else
    launch_width<T, FBEV_CODES_INT8>(a, plan, blocks, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.c.B * a.c.Hk * a.R;
  if (a.splits <= 16) {   // (8 splits of 4096 rows, both launches: 33 us against 39 with a workgroup a row)
    const unsigned n = (unsigned)((rows + 7) / 8);
    if (a.splits <= 4)
      cache_attn_join_few<T, 4><<<n, 256, 0, stream>>>(a);
    else if (a.splits <= 8)
      cache_attn_join_few<T, 8><<<n, 256, 0, stream>>>(a);
    else
      cache_attn_join_few<T, 16><<<n, 256, 0, stream>>>(a);
    return hipGetLastError();
  }
  // a wave for every eight splits: three at least, which have a thread for each channel
  const int waves = a.splits >= 128 ? 16 : (a.splits + 7) / 8;
  cache_attn_join<T><<<(unsigned)rows, 64 * waves, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t cache_attention_workspace_bytes(const CacheAttnArgs& a) {
  const int splits = plan_of(a).splits;
  return splits == 1 ? 0 : (size_t)splits * a.c.B * a.c.Hk * a.R * (a.c.D + 2) * sizeof(float);
}

hipError_t launch_cache_attention(CacheAttnArgs a, hipStream_t stream) {
  const Plan plan = plan_of(a);
  a.row_blocks = plan.row_blocks;
  a.down = room_for(a.c.W);
  a.splits = plan.splits;
  return a.elem_bytes == 4 ? launch_type<float>(a, plan, stream) : launch_type<__bf16>(a, plan, stream);
}

}  // namespace fbev
