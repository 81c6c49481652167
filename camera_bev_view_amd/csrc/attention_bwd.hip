// Attention between queries, cells and tokens, backward.
//
//   p_ij = 2^(s_ij - m_i) / l_i,  delta_i = go_i . o_i,  ds_ij = p_ij (go_i . v_j - delta_i),
//   gslope_i = - sum_j ds_ij |pos_i - pos_j|,   ds'_ij = ds_ij (1 - tanh^2)   (with a cap),
//   gq_i = scale sum_j ds'_ij k_j,   gk_j = scale sum_i ds'_ij q_i,   gv_j = sum_i p_ij go_i.
//
// Each launch recomputes the scores tile by tile: one owns query rows and walks the keys (delta, gq, gslope; for bf16 delta
// comes from a launch before it), one owns keys and walks the rows of all query heads that share them (gk, gv).  Every sum
// stays in registers and is written once (as an fp32 part where the walk is split over workgroups, which a launch behind
// joins in order), so nothing is added by atomics and results are the same from run to run; the price is seven matrix
// products a tile where five would do with atomics.  Distances are not differentiated: positions are given.
//
// What bounds it.  bf16, D = 32, distances, 10000 x 10000 cells of 8 heads: 1550 us, a trace 377 (delta), 545 (rows) and
// 811 us (keys), of which vector instructions, with the quarter rate of exponentials and roots, issue for 227, 340 and 426
// us and matrix ones for 82, 123 and 184; the rest is stages that are waited for in full, 1252 workgroups on 768 places, and
// in the keys' launch a few spilled registers.  fp32, 2 x 2048 packed rows of 8 heads over 4, D = 64, a cap: rows 109 us,
// keys 176 us, of which matrix and vector instructions issue for 27 + 25 and 35 + 38 us: the tiles' LDS leaves one or two
// workgroups a CU, whose work is unequal, and nothing hides their waits.
//
// Roundings of bf16 tensors: probabilities and score gradients go into their products as two bf16 each (16 bits).  With
// one each, gk and gv were 0.0024 off where their own rounding leaves 0.0017; the second part took the cells' backward from
// 1111 to 1280 us and that of 4 x 900 queries from 77 to 87 us.
#include "attention_core.h"

namespace fbev {
namespace {

constexpr int kThreads = 256;

// HB heads of a wave (two with a distance bias, whose distances they share), KW waves over the moving rows.
template <typename T, int DP, int KW, int HB>
struct Bwd {
  static constexpr int kWaves = KW == 8 ? 8 : 4, kThreads = 64 * kWaves;
  static constexpr int RW = kWaves / KW;
  static constexpr int MT = KW == 1 ? shared_rows<T>(DP) : 32 * KW;   // moving rows staged at a time
  static constexpr size_t kTile = (size_t)MT * Tile<T, DP>::kRowBytes;
  static constexpr size_t kTiles = 2 * HB * kTile;
  static constexpr size_t kMerge = (size_t)KW * 32 * (DP + 4) * 4;
  // two heads a wave: their own rows' fragments are read from LDS, which leaves registers for a third wave a SIMD
  static constexpr bool kOwnLds = HB == 2;
  static constexpr int kOwn = Mma<T, DP>::kFrags * 64 * 16;        // bytes of a tensor's fragments
  static constexpr size_t kBytes = KW == 1 || kTiles > kMerge ? kTiles : kMerge;
};

// Waves a SIMD, from the registers of two tensors' own rows and one or two of sums.
template <typename T, int DP>
constexpr int min_waves(int hb) {
  if (sizeof(T) == 4) return DP <= 64 && hb == 1 ? 2 : 1;
  return DP == 128 ? 1 : DP == 64 ? 2 : 3;
}

// Writes own rows' sums (scaled), or adds the waves' sums over LDS first.  dst(n) is own row n's
// address or NULL.
template <typename T, int DP, int KW, typename F>
__device__ __forceinline__ void write_own(f32x16 (&acc)[DP / 32], float scale, float* mo, int D, bool vec_out, int kw,
                                          int lane, F dst) {
  constexpr int NB = DP / 32, kThreads = KW == 8 ? 512 : 256;
  const int n = lane & 31, h = lane >> 5;
  if constexpr (KW == 1) {
    T* out = dst(n);
    if (out == nullptr) return;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = 32 * blk + 8 * u + 4 * h;
        if (vec_out) {
          if (c < D) {
            typedef T V4 __attribute__((ext_vector_type(4)));
            V4 o;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = (T)(acc[blk][4 * u + j] * scale);
            *(V4*)(out + c) = o;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < D) out[c + j] = (T)(acc[blk][4 * u + j] * scale);
        }
      }
  } else {
    __syncthreads();
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = acc[blk][4 * u + j];
        *(f32x4*)(mo + (kw * 32 + n) * (DP + 4) + 32 * blk + 8 * u + 4 * h) = o;
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * DP; e += kThreads) {
      const int r = e / DP, c = e - r * DP;
      T* out = dst(r);
      if (c >= D || out == nullptr) continue;
      float o = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) o += mo[(k * 32 + r) * (DP + 4) + c];
      out[c] = (T)(o * scale);
    }
  }
}

// A (sample, key head)'s rows in the workspace, for the keys' launch: delta, the exponents' offset (fp32: the maximum m;
// bf16: m + log2 l, in score units unless a cap comes between) and 1 / l, with a bias slope and position.
struct RowStats {
  float *delta, *off, *inv, *slope, *pos;
};

__host__ __device__ __forceinline__ int64_t stat_floats(const AttnArgs& a) { return a.dims ? 4 + a.dims : 3; }

__device__ __forceinline__ RowStats row_stats(const AttnArgs& a, int64_t bh) {
  float* p = a.delta + bh * a.R * stat_floats(a);
  const int64_t R = a.R;
  return RowStats{p, p + R, p + 2 * R, p + 3 * R, p + 4 * R};
}

// Where few own tiles stand against a long other side, its rows are split over `splits` workgroups, `per` (a multiple of
// every stage) each; their fp32 sums are joined in split order (bf16, D = 64: one token of 8 heads over 40000 keys of 2
// heads 587 -> 84 us; D = 32, distances: 40000 tokens of 8 heads over 900 keys of one head 4157 -> 838 us).
struct Split {
  int splits, per;
  float* part;
};

// Floats of a partial row: gq with the sums of ds, ds d and p d (or the sum of ds alone); gk or gv.
__host__ __device__ __forceinline__ int row_floats(bool grads, int D) { return grads ? (D + 6) / 4 * 4 : 1; }
__host__ __device__ __forceinline__ int key_floats(int D) { return (D + 3) / 4 * 4; }

// ---- query rows: delta, gq, gslope

// Delta is the mean of go . v over a row's weights, go . o with the output before its rounding.  Taken from the rounded
// output it is off by up to half a step of that, which in a row that looks at one key is many times the differences
// go . v - delta that make its gradients (bf16, 400 points of a 100 m square, slope 2: one row in twenty of gq off by more
// than itself, with the exact delta by 0.002).  fp32 outputs are exact enough for gq (half a step is 2^-24, what the products
// are off by too), and the sum of the row's ds corrects what the keys' launch and the slopes get.  For bf16 a launch of its
// own (kDelta: the scores once more, no gradients) sums up ds first: 290 us of the 100 x 100 cells' 1550, 19 us of the 106 of
// 4 x 900 queries.
enum Pass { kDelta, kGradients };

// Delta and its error.  Without a sum of ds (NaN: a key of the row is infinite) it stays as it came from the output, which
// knows what weight such a key has.
__device__ __forceinline__ float corrected(float delta, float sd) { return sd == sd ? delta + sd : delta; }

template <typename T>
constexpr bool kOwnDelta = sizeof(T) == 4;                // the gradients' launch forms delta itself

template <typename T, int DP, int KW, int HB, bool BIAS, bool CAP, Pass PASS>
__global__ __launch_bounds__((Bwd<T, DP, KW, HB>::kThreads), (min_waves<T, DP>(HB))) void attn_bwd_rows(AttnArgs a, int tiles, int blocks, Split sp) {
  using C = Bwd<T, DP, KW, HB>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, MT = C::MT, RW = C::RW;
  constexpr bool SUM = PASS == kDelta || kOwnDelta<T>, GRADS = PASS == kGradients;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[BIAS ? 3 * MT : 1];   // [key][axis]
  __shared__ alignas(16) int docs[MT];
  __shared__ int doc_range[C::kWaves][2];
  __shared__ uint32_t stage_bits;
  __shared__ float slopes[KW][3][32];
  char* Ks = smem;                                        // HB tiles each
  char* Vs = smem + HB * C::kTile;

  const int block = blockIdx.z * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const int bid = xcd_block(block, blocks);
  const int bh = bid / tiles, order = bid - bh * tiles;
  const int tile = a.causal ? tiles - 1 - order : order;  // causal rows: those with the most keys first
  const int b = bh / (a.Hk / HB), hk = (bh - b * (a.Hk / HB)) * HB;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int first = tile * 32 * RW + rw * 32;
  const Row w = make_row(a, b, hk, min(first + n, a.R - 1));
  const Unit un = make_unit(a);
  const Stager st = make_stager<T, DP>(a.D);
  __shared__ alignas(16) char own_frags[C::kOwnLds ? RW * HB * 2 * C::kOwn : 16];   // [row tile][head][q, go]
  char* own_at = own_frags + rw * HB * 2 * C::kOwn;
  typename M::Frag q[C::kOwnLds ? 1 : HB][M::kFrags], go[C::kOwnLds ? 1 : HB][M::kFrags];
  float delta[HB], neg_m[HB], inv_l[HB], slope[HB] = {};
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    const int64_t row_at = (((int64_t)b * a.Tq + w.t) * a.Hq + w.head + i) * a.D;
    constexpr bool L = C::kOwnLds;
    auto& qi = q[L ? 0 : i];
    auto& gi = go[L ? 0 : i];
    load_row<T, DP>((const T*)a.q + b * a.qs[0] + w.t * a.qs[1] + (w.head + i) * a.qs[2], a.vec, a.D, h, qi);
    sign_row<T, DP>(a, qi);
    load_row<T, DP>((const T*)a.gout + row_at, a.vec, a.D, h, gi);
    if (L && kw == 0) {
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) {
        *(typename M::Frag*)(own_at + 2 * i * C::kOwn + (f * 64 + lane) * 16) = qi[f];
        *(typename M::Frag*)(own_at + (2 * i + 1) * C::kOwn + (f * 64 + lane) * 16) = gi[f];
      }
    }
    const RowStats rs = row_stats(a, (int64_t)b * a.Hk + hk + i);
    if constexpr (SUM) {
      typename M::Frag o[M::kFrags];
      load_row<T, DP>((const T*)a.out + row_at, a.vec, a.D, h, o);
      float sum = 0.0f;
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f)
#pragma unroll
        for (int j = 0; j < M::kFragElems; ++j) sum = fmaf((float)gi[f][j], (float)o[f][j], sum);
      delta[i] = pair_sum(sum);
    } else {
      delta[i] = rs.delta[w.r];
    }
    // exponentials are taken around the forward's maximum and divided by its sum at the end: a logarithm of the sum
    // would be off by its own size times 2^-24.  A row without weights: all p are 0.
    const float2 ml = a.stats[((int64_t)b * a.Hq + w.head + i) * a.Tq + w.t];
    neg_m[i] = ml.y == 0.0f ? kNegInf : -ml.x;
    inv_l[i] = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
    if constexpr (BIAS) slope[i] = a.slope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head + i] / un.raw;
    if (SUM && kw == 0 && h == 0 && first + n < a.R && blockIdx.y == 0) {
      const float lse2 = ml.y == 0.0f ? -kNegInf : ml.x + __builtin_amdgcn_logf(ml.y);
      rs.off[w.r] = sizeof(T) == 4 ? -neg_m[i] : CAP ? lse2 : lse2 / un.unit;
      rs.inv[w.r] = inv_l[i];
      if constexpr (BIAS) {
        rs.slope[w.r] = slope[i];
        for (int ax = 0; ax < a.dims; ++ax)
          rs.pos[(int64_t)w.r * a.dims + ax] = a.pos_q[((int64_t)b * a.Tq + w.t) * a.dims + ax];
      }
    }
  }
  float own[3] = {0.0f, 0.0f, 0.0f};
  if constexpr (BIAS) {
    own_point(a.pos_q + ((int64_t)b * a.Tq + w.t) * a.dims, a.dims, h, own);
  }
  for (int e = threadIdx.x; e < MT; e += C::kThreads) docs[e] = 0;
  const int lim_lo = row_limit(a, b, min(first, a.R - 1) / a.G);
  const int lim_hi = row_limit(a, b, min(first + 31, a.R - 1) / a.G);
  const int blk_lo = row_limit(a, b, min(tile * 32 * RW, a.R - 1) / a.G);
  const int blk_hi = row_limit(a, b, min(tile * 32 * RW + 32 * RW - 1, a.R - 1) / a.G);
  int dmin = 0, dmax = 0, bmin = 0, bmax = 0;
  if (a.doc_q) {
    dmin = wave_min(w.doc < 0 ? INT32_MAX : w.doc);
    dmax = wave_max(w.doc);
    if (lane == 0) doc_range[wave][0] = dmin, doc_range[wave][1] = dmax;
    __syncthreads();
    bmin = doc_range[0][0], bmax = doc_range[0][1];
#pragma unroll
    for (int i = 1; i < C::kWaves; ++i) bmin = min(bmin, doc_range[i][0]), bmax = max(bmax, doc_range[i][1]);
  }
  const bool one_doc = dmin == dmax && wave_min(w.doc) == dmin;

  f32x16 acc[HB][NB] = {};
  bool odd[HB] = {};                                      // the row sees a key with an infinite or NaN element
  float sum_ds[HB] = {}, sum_dsd[HB] = {}, sum_pd[HB] = {};
  const int k_begin = (int)blockIdx.y * sp.per;
  const int k_end = min(min(a.Tk, blk_hi + 1), k_begin + sp.per);
  uint32_t stages = 0;
  for (int s0 = k_begin; s0 < k_end; s0 += MT) {
    const int nk = min(MT, a.Tk - s0);
    int my_doc = -1;
    if (a.doc_q) {
      const int stage = (s0 - k_begin) / MT & 31;
      if (stage == 0)
        stages = stages_with<MT, C::kThreads>(&stage_bits, s0, k_end, bmin, bmax, [&](int j) { return a.doc_k[(int64_t)b * a.Tk + j]; });
      if (!((stages >> stage) & 1)) continue;
      if ((int)threadIdx.x < nk) my_doc = a.doc_k[(int64_t)b * a.Tk + s0 + threadIdx.x];
    }
    __syncthreads();
    const bool mixed = a.doc_q != nullptr || (a.causal && s0 + MT - 1 > blk_lo);
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      stage_rows<T, DP, MT, C::kThreads>(Ks + i * C::kTile, (const T*)a.k + b * a.ks[0] + s0 * a.ks[1] + (hk + i) * a.ks[2], a.ks[1],
                            nk, a.vec, a.D, st);
      stage_rows<T, DP, MT, C::kThreads>(Vs + i * C::kTile, (const T*)a.v + b * a.vs[0] + s0 * a.vs[1] + (hk + i) * a.vs[2], a.vs[1],
                            nk, a.vec, a.D, st);
    }
    if (a.doc_q && (int)threadIdx.x < MT) docs[threadIdx.x] = my_doc;
    if constexpr (BIAS) stage_floats<C::kThreads>(pos, a.pos_k + ((int64_t)b * a.Tk + s0) * a.dims, nk * a.dims, MT * a.dims);
    auto visible = [&](int at) {
      uint32_t vis = 0;
      const int hh = (int)opaque(h);
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        const int kr = at + acc_row(i, hh);
        vis = 2 * vis + (s0 + kr <= w.lim && docs[kr] == w.doc ? 1u : 0u);
      }
      return vis;
    };
    wait_staged();
    __syncthreads();
    if (GRADS && mixed && __builtin_expect(__syncthreads_or(holds_odd<T, DP, HB * MT, C::kThreads>(Ks)), 0)) {
#pragma unroll 1
      for (int at = 32 * kw; at < MT; at += 32 * KW) {
        const uint32_t vis = visible(at);
#pragma unroll
        for (int hd = 0; hd < HB; ++hd) odd[hd] |= sees_odd<T, DP>(Ks + hd * C::kTile, at, vis, lane);
      }
      __syncthreads();
      clean_rows<T, DP, HB * MT, C::kThreads>(Ks);
      __syncthreads();
    }
#pragma unroll 1
    for (int sub = 0; sub < MT / (32 * KW); ++sub) {
      const int at = 32 * (sub * KW + kw), key0 = s0 + at;
      if (key0 > lim_hi || key0 >= a.Tk) continue;
      bool whole = key0 + 31 <= lim_lo;
      if (a.doc_q) {
        const int d = docs[at + n];
        if (!__any(d >= dmin && d <= dmax)) continue;
        whole = whole && one_doc && __all(d == dmin);
      }
      const uint32_t seen = whole ? 0xFFFFu : visible(at);
      f32x16 d;
      if constexpr (BIAS) distances(pos, at, a.dims, own, lane, d);
      if constexpr (BIAS) {
        if (!whole) {
          const uint32_t vis = opaque(seen);
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = (vis >> i) & 1 ? d[i] : 0.0f;
        }
      }
#pragma unroll
      for (int hd = 0; hd < HB; ++hd) {
        __builtin_amdgcn_sched_barrier(0);                // one head's registers at a time
        const char* kt = Ks + hd * C::kTile;
        f32x16 s;
        if constexpr (C::kOwnLds)
          s = tile_dot<T, DP>(kt, at, own_at + 2 * hd * C::kOwn, lane);
        else
          s = tile_dot<T, DP>(kt, at, q[hd], lane);
        // dp - delta: the sum starts from -delta
        f32x16 dp = outer_sum(h == 0 ? 1.0f : 0.0f, h == 0 ? -delta[hd] : 0.0f);
        if constexpr (C::kOwnLds)
          dp = tile_dot<T, DP>(Vs + hd * C::kTile, at, own_at + (2 * hd + 1) * C::kOwn, lane, dp);
        else
          dp = tile_dot<T, DP>(Vs + hd * C::kTile, at, go[hd], lane, dp);
        f32x16 th;
        if constexpr (CAP) {
          cap_scores<T>(s, un);
          th = s;
        }
        if constexpr (BIAS) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = fmaf(-slope[hd], d[i], s[i]);
        }
        if (!whole) {
          const uint32_t vis = opaque(seen);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[i] = (vis >> i) & 1 ? s[i] : kNegInf;
            dp[i] = (vis >> i) & 1 ? dp[i] : 0.0f;
          }
        }
        float t_ds = 0.0f, t_dsd = 0.0f, t_pd = 0.0f;     // a tile's sums first: thousands of keys in one chain add up errors
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(fmaf(s[i], un.unit, neg_m[hd]));
          s[i] = p * dp[i];
          if constexpr (SUM) t_ds += s[i];
          if constexpr (BIAS && GRADS) t_dsd = fmaf(s[i], d[i], t_dsd);
          if constexpr (BIAS && GRADS && SUM) t_pd = fmaf(p, d[i], t_pd);
        }
        if constexpr (SUM) pin(sum_ds[hd] += t_ds);
        if constexpr (BIAS && GRADS) pin(sum_dsd[hd] += t_dsd);
        if constexpr (BIAS && GRADS && SUM) pin(sum_pd[hd] += t_pd);
        if constexpr (GRADS) {
          if constexpr (CAP) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = whole || (seen >> i) & 1 ? s[i] * fmaf(-th[i], th[i], 1.0f) : 0.0f;
          }
          __builtin_amdgcn_sched_barrier(0);
          M::template accumulate<NB>(acc[hd], s, kt, at, lane);
        }
      }
    }
  }
#pragma unroll
  for (int hd = 0; hd < HB; ++hd) {
    const bool split = KW > 1 && HB == 1 && sp.splits > 1;
    const RowStats rs = row_stats(a, (int64_t)b * a.Hk + hk + hd);
    // partial rows of a split, from the tile's first row on
    float* part = nullptr;
    if (split) part = sp.part + (((int64_t)blockIdx.y * a.B * a.Hk + bh) * a.R + first) * row_floats(GRADS, a.D);
    if constexpr (GRADS) {
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[hd][blk][i] *= inv_l[hd];
      make_nan<NB>(acc[hd], odd[hd]);
      // the queries' sign is in s, not in k: a zero scale gives zeros
      if (split)
        write_own<float, DP, KW>(acc[hd], a.scale, (float*)smem, a.D, false, kw, lane, [&](int r) -> float* {
          return first + r < a.R ? part + (int64_t)r * row_floats(GRADS, a.D) : nullptr;
        });
      else
        write_own<T, DP, KW>(acc[hd], a.scale, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) -> T* {
          if (first + r >= a.R) return nullptr;
          const int t = (first + r) / a.G, head = hk * a.G + (first + r - t * a.G) + hd;
          return (T*)a.gq + (((int64_t)b * a.Tq + t) * a.Hq + head) * a.D;
        });
    }
    // ds sums to the error of delta (sum_j p_ij = 1): the keys' launch (and bf16 gradients) get delta without it, and the
    // distances' mean takes it out of an fp32 slope's gradient
    // (a row that sees an infinite or NaN key gets NaN: its scores here are those of the cleaned key)
    float sd = odd[hd] ? __builtin_nanf("") : pair_sum(sum_ds[hd]) * inv_l[hd], sdd = 0.0f, pd = 0.0f;
    if constexpr (BIAS && GRADS) {
      sdd = pair_sum(sum_dsd[hd]) * inv_l[hd];
      pd = pair_sum(sum_pd[hd]) * inv_l[hd];
    }
    if constexpr (KW > 1) {
      __syncthreads();
      if (h == 0) slopes[kw][0][n] = sd, slopes[kw][1][n] = sdd, slopes[kw][2][n] = pd;
      __syncthreads();
      sd = sdd = pd = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) sd += slopes[k][0][n], sdd += slopes[k][1][n], pd += slopes[k][2][n];
    }
    if (kw != 0 || h != 0 || first + n >= a.R) continue;
    if (split) {
      float* sums = part + (int64_t)n * row_floats(GRADS, a.D) + (GRADS ? a.D : 0);
      sums[0] = sd;
      if constexpr (GRADS) sums[1] = sdd, sums[2] = pd;
      if (SUM && blockIdx.y == 0) rs.delta[w.r] = delta[hd];
    } else {
      if constexpr (SUM) rs.delta[w.r] = corrected(delta[hd], sd);
      if (GRADS && BIAS && a.gslope)
        a.gslope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head + hd] = fmaf(sd, pd, -sdd);
    }
  }
}

// ---- keys: gk, gv

template <typename T, int DP, int KW, int HB, bool BIAS, bool CAP>
__global__ __launch_bounds__((Bwd<T, DP, KW, HB>::kThreads), (min_waves<T, DP>(HB))) void attn_bwd_keys(AttnArgs a, int tiles, int blocks, Split sp) {
  using C = Bwd<T, DP, KW, HB>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, MT = C::MT, RW = C::RW;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[BIAS ? 3 * MT : 1];   // [row][axis]
  constexpr bool EXACT = sizeof(T) == 4;                  // p from the maximum and 1 / l, not from their logarithm
  __shared__ alignas(16) float offs[HB][MT], invs[EXACT ? HB : 1][EXACT ? MT : 4], deltas[HB][MT];
  __shared__ alignas(16) float slopes[HB][BIAS ? MT : 4];
  __shared__ alignas(16) int docs[MT], lims[MT];
  __shared__ int doc_range[C::kWaves][2];
  __shared__ uint32_t stage_bits;
  char* Qs = smem;                                        // HB tiles each
  char* Gs = smem + HB * C::kTile;

  const int block = blockIdx.z * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const int bid = xcd_block(block, blocks);
  const int tile = bid % tiles, bh = bid / tiles;
  const int b = bh / (a.Hk / HB), hk = (bh - b * (a.Hk / HB)) * HB;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int key0 = tile * 32 * RW + rw * 32;              // the wave's keys
  const int key = min(key0 + n, a.Tk - 1);
  const Unit un = make_unit(a);
  const Stager st = make_stager<T, DP>(a.D);
  __shared__ alignas(16) char own_frags[C::kOwnLds ? RW * HB * 2 * C::kOwn : 16];   // [key tile][head][k, v]
  char* own_at = own_frags + rw * HB * 2 * C::kOwn;
  typename M::Frag k[C::kOwnLds ? 1 : HB][M::kFrags], v[C::kOwnLds ? 1 : HB][M::kFrags];
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    constexpr bool L = C::kOwnLds;
    auto& ki = k[L ? 0 : i];
    auto& vi = v[L ? 0 : i];
    load_row<T, DP>((const T*)a.k + b * a.ks[0] + key * a.ks[1] + (hk + i) * a.ks[2], a.vec, a.D, h, ki);
    sign_row<T, DP>(a, ki);                               // the sign of the scale, on the side that only scores read
    load_row<T, DP>((const T*)a.v + b * a.vs[0] + key * a.vs[1] + (hk + i) * a.vs[2], a.vec, a.D, h, vi);
    if (L && kw == 0) {
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) {
        *(typename M::Frag*)(own_at + 2 * i * C::kOwn + (f * 64 + lane) * 16) = ki[f];
        *(typename M::Frag*)(own_at + (2 * i + 1) * C::kOwn + (f * 64 + lane) * 16) = vi[f];
      }
    }
  }
  float own[3] = {0.0f, 0.0f, 0.0f};
  if constexpr (BIAS) {
    own_point(a.pos_k + ((int64_t)b * a.Tk + key) * a.dims, a.dims, h, own);
  }
  const int doc = a.doc_k ? a.doc_k[(int64_t)b * a.Tk + key] : 0;
  int dmin = 0, dmax = 0, bmin = 0, bmax = 0;
  if (a.doc_q) {
    dmin = wave_min(doc < 0 ? INT32_MAX : doc);
    dmax = wave_max(doc);
    if (lane == 0) doc_range[wave][0] = dmin, doc_range[wave][1] = dmax;
    __syncthreads();
    bmin = doc_range[0][0], bmax = doc_range[0][1];
#pragma unroll
    for (int i = 1; i < C::kWaves; ++i) bmin = min(bmin, doc_range[i][0]), bmax = max(bmax, doc_range[i][1]);
  }
  const bool one_doc = dmin == dmax && wave_min(doc) == dmin;

  f32x16 gk[HB][NB] = {}, gv[HB][NB] = {};
  uint32_t odd[HB][NB] = {};                              // infinite or NaN output gradients the key is seen with
  bool odd_key[HB] = {};                                  // seen by a query with an infinite or NaN element
  // rows from the first whose order lets it see the workgroup's first key
  const int blk_key = tile * 32 * RW;
  int r_begin = 0;
  if (a.causal && !(a.prefix && a.prefix[b] > blk_key)) {
    const int64_t t0 = (int64_t)blk_key - a.Tk + a.Tq;
    if (t0 > 0) r_begin = (int)((t0 < a.Tq ? t0 : a.Tq) * a.G) / MT * MT;
  }
  r_begin = max(r_begin, (int)blockIdx.y * sp.per);
  const int r_end = min(a.R, (int)blockIdx.y * sp.per + sp.per);
  uint32_t stages = 0;
  for (int s0 = r_begin; s0 < r_end; s0 += MT) {
    const int nr = min(MT, a.R - s0);
    Row w;
    w.doc = -1, w.lim = -1;
    if (a.doc_q) {
      const int stage = (s0 - r_begin) / MT & 31;
      if (stage == 0)
        stages = stages_with<MT, C::kThreads>(&stage_bits, s0, a.R, bmin, bmax,
                                 [&](int r) { return a.doc_q[(int64_t)b * a.Tq + r / a.G]; });
      if (!((stages >> stage) & 1)) continue;
    }
    if (a.causal || a.doc_q) {
      if ((int)threadIdx.x < nr) w = make_row(a, b, hk, s0 + threadIdx.x);
    }
    __syncthreads();
    // some row of the tile may not see some key of the workgroup
    const bool mixed = a.doc_q != nullptr ||
                       (a.causal && row_limit(a, b, s0 / a.G) < min(blk_key + 32 * RW, a.Tk) - 1);
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      if (a.G == 1) {
        stage_rows<T, DP, MT, C::kThreads>(Qs + i * C::kTile, (const T*)a.q + b * a.qs[0] + s0 * a.qs[1] + (hk + i) * a.qs[2],
                              a.qs[1], nr, a.vec, a.D, st);
        stage_rows<T, DP, MT, C::kThreads>(Gs + i * C::kTile, (const T*)a.gout + (((int64_t)b * a.Tq + s0) * a.Hq + hk + i) * a.D,
                              (int64_t)a.Hq * a.D, nr, a.vec, a.D, st);
      } else {
        stage_group<T, DP, MT, C::kThreads>(Qs, (const T*)a.q + b * a.qs[0] + hk * a.G * a.qs[2], a.qs[1], a.qs[2], s0, a.G, nr, a.vec,
                               a.D);
        stage_group<T, DP, MT, C::kThreads>(Gs, (const T*)a.gout + ((int64_t)b * a.Tq * a.Hq + hk * a.G) * a.D, (int64_t)a.Hq * a.D,
                               a.D, s0, a.G, nr, a.vec, a.D);
      }
    }
    if ((a.causal || a.doc_q) && (int)threadIdx.x < MT) {
      docs[threadIdx.x] = w.doc;
      lims[threadIdx.x] = w.lim;
    }
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      const RowStats rs = row_stats(a, (int64_t)b * a.Hk + hk + i);
      stage_floats<C::kThreads>(offs[i], rs.off + s0, nr, MT);
      if constexpr (EXACT) stage_floats<C::kThreads>(invs[i], rs.inv + s0, nr, MT);
      stage_floats<C::kThreads>(deltas[i], rs.delta + s0, nr, MT);
      if constexpr (BIAS) {
        stage_floats<C::kThreads>(slopes[i], rs.slope + s0, nr, MT);
        if (i == 0) stage_floats<C::kThreads>(pos, rs.pos + (int64_t)s0 * a.dims, nr * a.dims, MT * a.dims);
      }
    }
    auto visible = [&](int at) {
      uint32_t vis = 0;
      const int hh = (int)opaque(h);
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        const int r = at + acc_row(i, hh);
        vis = 2 * vis + (key0 + n <= lims[r] && docs[r] == doc ? 1u : 0u);
      }
      return vis;
    };
    wait_staged();
    __syncthreads();
    if (mixed && __builtin_expect(__syncthreads_or(holds_odd<T, DP, 2 * HB * MT, C::kThreads>(Qs)), 0)) {
#pragma unroll 1
      for (int at = 32 * kw; at < MT; at += 32 * KW) {
        const uint32_t vis = visible(at);
#pragma unroll
        for (int hd = 0; hd < HB; ++hd) {
          const char* gt = Gs + hd * C::kTile;
          odd_key[hd] |= sees_odd<T, DP>(Qs + hd * C::kTile, at, vis, lane);
          odd_key[hd] |= sees_odd<T, DP>(gt, at, vis, lane);
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) odd[hd][blk] |= find_odd<T, DP>(gt, at, blk, vis, lane);
        }
      }
      __syncthreads();
      clean_rows<T, DP, 2 * HB * MT, C::kThreads>(Qs);
      __syncthreads();
    }
#pragma unroll 1
    for (int sub = 0; sub < MT / (32 * KW); ++sub) {
      const int at = 32 * (sub * KW + kw);
      if (s0 + at >= a.R) continue;
      bool whole = true;
      if (a.causal || a.doc_q) {
        const int lim = s0 + at + n < a.R ? lims[at + n] : INT32_MAX;
        if (!__any(lim != INT32_MAX && lim >= key0)) continue;
        whole = __all(lim >= min(key0 + 31, a.Tk - 1));
      }
      if (a.doc_q) {
        const int d = docs[at + n];
        if (!__any(d >= dmin && d <= dmax)) continue;
        whole = whole && one_doc && __all(d == dmin);
      }
      const uint32_t seen = whole ? 0xFFFFu : visible(at);
      f32x16 d;
      if constexpr (BIAS) distances(pos, at, a.dims, own, lane, d);
#pragma unroll
      for (int hd = 0; hd < HB; ++hd) {
        __builtin_amdgcn_sched_barrier(0);                // one head's registers at a time
        const char* qt = Qs + hd * C::kTile;
        const char* gt = Gs + hd * C::kTile;
        // the sums start from the exponents' offset (bf16 without a cap) and -delta of the moving row
        constexpr bool FOLD = !CAP && !EXACT;
        const float one = h == 0 ? 1.0f : 0.0f;
        const float l2 = !FOLD || h != 0 ? 0.0f : -offs[hd][at + n];
        f32x16 s = {}, dp = outer_sum(h == 0 ? -deltas[hd][at + n] : 0.0f, one);
        if constexpr (FOLD) s = outer_sum(l2, one);
        if constexpr (C::kOwnLds) {
          s = tile_dot<T, DP>(qt, at, own_at + 2 * hd * C::kOwn, lane, s);
          dp = tile_dot<T, DP>(gt, at, own_at + (2 * hd + 1) * C::kOwn, lane, dp);
        } else {
          s = tile_dot<T, DP>(qt, at, k[hd], lane, s);
          dp = tile_dot<T, DP>(gt, at, v[hd], lane, dp);
        }
        f32x16 th;
        if constexpr (CAP) {
          cap_scores<T>(s, un);
          th = s;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = at + 8 * u + 4 * h;
          f32x4 sl = {}, l2 = {}, inv = {};
          if constexpr (!FOLD) l2 = *(const f32x4*)&offs[hd][r];
          if constexpr (EXACT) inv = *(const f32x4*)&invs[hd][r];
          if constexpr (BIAS) sl = *(const f32x4*)&slopes[hd][r];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 4 * u + j;
            if constexpr (BIAS) s[i] = fmaf(-sl[j], d[i], s[i]);
            s[i] = __builtin_amdgcn_exp2f(FOLD ? s[i] * un.unit : fmaf(s[i], un.unit, -l2[j]));
            if constexpr (EXACT) s[i] *= inv[j];
            dp[i] *= s[i];
            if constexpr (CAP) dp[i] *= fmaf(-th[i], th[i], 1.0f);
          }
        }
        if (!whole) {
          const uint32_t vis = opaque(seen);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[i] = (vis >> i) & 1 ? s[i] : 0.0f;
            dp[i] = (vis >> i) & 1 ? dp[i] : 0.0f;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        M::template accumulate<NB>(gv[hd], s, gt, at, lane);
        M::template accumulate<NB>(gk[hd], dp, qt, at, lane);
      }
    }
  }
#pragma unroll
  for (int hd = 0; hd < HB; ++hd) {
    auto at_key = [&](void* base, int r) -> T* {
      if (key0 + r >= a.Tk) return nullptr;
      return (T*)base + (((int64_t)b * a.Tk + key0 + r) * a.Hk + hk + hd) * a.D;
    };
    add_odd<NB>(gv[hd], odd[hd]);
    make_nan<NB>(gk[hd], odd_key[hd]);
    if constexpr (KW > 1 && HB == 1) {
      if (sp.splits > 1) {
        const int pf = key_floats(a.D);
        float* part = sp.part + (((int64_t)blockIdx.y * a.B * a.Hk + bh) * a.Tk + key0) * 2 * pf;
        auto row = [&](int r, int which) { return key0 + r < a.Tk ? part + ((int64_t)r * 2 + which) * pf : nullptr; };
        write_own<float, DP, KW>(gv[hd], 1.0f, (float*)smem, a.D, false, kw, lane, [&](int r) { return row(r, 1); });
        write_own<float, DP, KW>(gk[hd], a.scale, (float*)smem, a.D, false, kw, lane, [&](int r) { return row(r, 0); });
        return;
      }
    }
    write_own<T, DP, KW>(gv[hd], 1.0f, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) { return at_key(a.gv, r); });
    write_own<T, DP, KW>(gk[hd], a.scale, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) { return at_key(a.gk, r); });
  }
}

// ---- joins of the splits: a wave a row

// Sum of element lane + 64 j of a row over the splits, eight of them in flight at once.
template <int N>
__device__ __forceinline__ void sum_splits(const float* row, int64_t stride, int splits, int floats, int lane,
                                           float (&o)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = 0.0f;
  for (int s0 = 0; s0 < splits; s0 += 8) {
    float v[8][N];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = row[min(s0 + i, splits - 1) * stride + min(lane + 64 * j, floats - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] += s0 + i < splits ? v[i][j] : 0.0f;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void attn_bwd_join_rows(AttnArgs a, Split sp) {
  const int64_t rows = (int64_t)a.B * a.Hk * a.R, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int lane = threadIdx.x & 63, pf = row_floats(true, a.D);
  float o[3];
  sum_splits<3>(sp.part + row * pf, rows * pf, sp.splits, a.D + 3, lane, o);
  const int64_t bh = row / a.R;
  const int r = (int)(row - bh * a.R), t = r / a.G, b = (int)(bh / a.Hk);
  const int head = (int)(bh - (int64_t)b * a.Hk) * a.G + (r - t * a.G);
  T* gq = (T*)a.gq + (((int64_t)b * a.Tq + t) * a.Hq + head) * a.D;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 64 * j < a.D) gq[lane + 64 * j] = (T)o[j];
  auto at = [&](int i) { return __shfl(i < 64 ? o[0] : i < 128 ? o[1] : o[2], i & 63); };
  const float sd = at(a.D), sdd = at(a.D + 1), pd = at(a.D + 2);
  if (lane == 0) {
    float& delta = row_stats(a, bh).delta[r];
    if (kOwnDelta<T>) delta = corrected(delta, sd);
    if (a.dims && a.gslope) a.gslope[((int64_t)b * a.Tq + t) * a.Hq + head] = fmaf(sd, pd, -sdd);
  }
}

// The sums of ds alone: a lane a row.
__global__ __launch_bounds__(kThreads) void attn_bwd_join_delta(AttnArgs a, Split sp) {
  const int64_t rows = (int64_t)a.B * a.Hk * a.R, row = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (row >= rows) return;
  float o[1];
  sum_splits<1>(sp.part + row, rows, sp.splits, 1, 0, o);
  const int64_t bh = row / a.R;
  float& delta = row_stats(a, bh).delta[row - bh * a.R];
  delta = corrected(delta, o[0]);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void attn_bwd_join_keys(AttnArgs a, Split sp) {
  const int64_t rows = (int64_t)a.B * a.Hk * a.Tk * 2, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int lane = threadIdx.x & 63, pf = key_floats(a.D);
  float o[2];
  sum_splits<2>(sp.part + row * pf, rows * pf, sp.splits, a.D, lane, o);
  const int64_t bh = row / 2 / a.Tk;
  const int key = (int)(row / 2 - bh * a.Tk), b = (int)(bh / a.Hk), hk = (int)(bh - (int64_t)b * a.Hk);
  T* out = (T*)(row & 1 ? a.gv : a.gk) + (((int64_t)b * a.Tk + key) * a.Hk + hk) * a.D;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 64 * j < a.D) out[lane + 64 * j] = (T)o[j];
}

// `own` rows a head against `len` others: split under 128 tiles of 32, as the forward's keys are.
Split make_split(const AttnArgs& a, int own, int len) {
  const int64_t tiles = (int64_t)a.B * a.Hk * ((own + 31) / 32);
  Split sp{1, INT32_MAX / 256 * 256, nullptr};
  if (tiles == 0 || tiles >= 128 || len <= 256) return sp;
  const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  const int64_t want = least((1024 + tiles - 1) / tiles, ((int64_t)len + 511) / 512);
  const int64_t fill = least((256 + tiles - 1) / tiles, ((int64_t)len + 255) / 256);
  const int64_t n = want > fill ? want : fill;
  sp.per = (int)((((int64_t)len + n - 1) / n + 255) / 256 * 256);
  sp.splits = (int)(((int64_t)len + sp.per - 1) / sp.per);
  return sp;
}

// Waves that split the moving rows of a tile of own rows.
template <typename T, int DP, int HB>
int pick_waves(const AttnArgs& a, int64_t heads, int rows) {
  // 128 own rows a workgroup, which share staged tiles, when there are enough to fill the card several times over
  if (heads * ((rows + 127) / 128) >= (a.D <= 64 ? 2048 : 512)) return 1;
  // too few workgroups to keep every SIMD busy and to even out masked ones: eight (512 workgroups of packed fp32 keys:
  // the pass takes 266 us against 299 us; with 1024 of them eight waves lose what they gain)
  if (HB == 1 && eight_waves<T>(DP) && heads * ((rows + 31) / 32) < 768) return 8;
  return 4;
}

// Workgroups by splits, rows of workgroups in the third dimension.
dim3 split_grid(int blocks, const Split& sp) {
  const dim3 rows = grid_rows(blocks);
  return dim3(rows.x, (unsigned)sp.splits, rows.y);
}

// The rows' figures, then the splits' partial rows (of one launch at a time).
int64_t stats_size(const AttnArgs& a) { return ((int64_t)a.B * a.Hk * a.R * stat_floats(a) + 3) / 4 * 4; }
float* split_part(const AttnArgs& a) { return a.delta == nullptr ? nullptr : a.delta + stats_size(a); }

template <typename T, int DP, int HB, bool BIAS, bool CAP, Pass PASS>
void launch_rows(const AttnArgs& a, int kw, dim3 grid, int tiles, int blocks, const Split& sp, hipStream_t stream) {
  if (kw == 1)
    attn_bwd_rows<T, DP, 1, HB, BIAS, CAP, PASS><<<grid, 256, 0, stream>>>(a, tiles, blocks, sp);
  else if (kw == 4)
    attn_bwd_rows<T, DP, 4, HB, BIAS, CAP, PASS><<<grid, 256, 0, stream>>>(a, tiles, blocks, sp);
  else if constexpr (HB == 1 && eight_waves<T>(DP))
    attn_bwd_rows<T, DP, 8, HB, BIAS, CAP, PASS><<<grid, 512, 0, stream>>>(a, tiles, blocks, sp);
}

template <typename T, int DP, int HB, bool BIAS, bool CAP>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const int64_t heads = (int64_t)a.B * a.Hk / HB;
  if (a.R > 0) {
    const int kw = pick_waves<T, DP, HB>(a, heads, a.R), rows = kw == 1 ? 128 : 32;
    const int tiles = (a.R + rows - 1) / rows;
    Split sp = make_split(a, a.R, a.Tk);
    sp.part = split_part(a);
    const int blocks = (int)(heads * tiles);
    const dim3 grid = split_grid(blocks, sp);
    if constexpr (!kOwnDelta<T>) {
      launch_rows<T, DP, HB, BIAS, CAP, kDelta>(a, kw, grid, tiles, blocks, sp, stream);
      if (sp.splits > 1)
        attn_bwd_join_delta<<<dim3((unsigned)(((int64_t)a.B * a.Hk * a.R + kThreads - 1) / kThreads)), kThreads, 0, stream>>>(a, sp);
    }
    launch_rows<T, DP, HB, BIAS, CAP, kGradients>(a, kw, grid, tiles, blocks, sp, stream);
    if (sp.splits > 1)
      attn_bwd_join_rows<T><<<dim3((unsigned)(((int64_t)a.B * a.Hk * a.R + 3) / 4)), kThreads, 0, stream>>>(a, sp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.Tk > 0) {
    const int kw = pick_waves<T, DP, HB>(a, heads, a.Tk), rows = kw == 1 ? 128 : 32;
    const int tiles = (a.Tk + rows - 1) / rows;
    Split sp = make_split(a, a.Tk, a.R);
    sp.part = split_part(a);
    const int blocks = (int)(heads * tiles);
    const dim3 grid = split_grid(blocks, sp);
    if (kw == 1)
      attn_bwd_keys<T, DP, 1, HB, BIAS, CAP><<<grid, 256, 0, stream>>>(a, tiles, blocks, sp);
    else if (kw == 4)
      attn_bwd_keys<T, DP, 4, HB, BIAS, CAP><<<grid, 256, 0, stream>>>(a, tiles, blocks, sp);
    else if constexpr (HB == 1 && eight_waves<T>(DP))
      attn_bwd_keys<T, DP, 8, HB, BIAS, CAP><<<grid, 512, 0, stream>>>(a, tiles, blocks, sp);
    if (sp.splits > 1)
      attn_bwd_join_keys<T><<<dim3((unsigned)(((int64_t)a.B * a.Hk * a.Tk * 2 + 3) / 4)), kThreads, 0, stream>>>(a, sp);
  }
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t run(const AttnArgs& a, hipStream_t stream) {
  if (a.cap > 0.0f)
    return a.dims ? launch<T, DP, 1, true, true>(a, stream) : launch<T, DP, 1, false, true>(a, stream);
  if (a.dims == 0) return launch<T, DP, 1, false, false>(a, stream);
  // two heads a wave where they share the distances and there are enough of them to fill the card
  if constexpr (DP == 32) {
    const int64_t shorter = a.R < a.Tk ? a.R : a.Tk;
    if (a.G == 1 && a.Hk % 2 == 0 && (int64_t)a.B * a.Hk * ((shorter + 31) / 32) >= 512)
      return launch<T, DP, 2, true, false>(a, stream);
  }
  return launch<T, DP, 1, true, false>(a, stream);
}

template <typename T>
hipError_t by_width(const AttnArgs& a, hipStream_t stream) {
  if (a.D <= 32) return run<T, 32>(a, stream);
  if (a.D <= 64) return run<T, 64>(a, stream);
  return run<T, 128>(a, stream);
}

}  // namespace

size_t attention_backward_workspace_bytes(const AttnArgs& a) {
  const int64_t heads = (int64_t)a.B * a.Hk;
  const Split r = make_split(a, a.R, a.Tk), k = make_split(a, a.Tk, a.R);
  const int64_t rows = r.splits > 1 ? heads * a.R * row_floats(true, a.D) * r.splits : 0;
  const int64_t keys = k.splits > 1 ? heads * a.Tk * 2 * key_floats(a.D) * k.splits : 0;
  return (size_t)(stats_size(a) + (rows > keys ? rows : keys)) * sizeof(float);
}

hipError_t launch_attention_backward(AttnArgs a, hipStream_t stream) {
  return a.elem_bytes == 4 ? by_width<float>(a, stream) : by_width<__bf16>(a, stream);
}

}  // namespace fbev
