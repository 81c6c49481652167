// Attention between queries, cells and tokens, backward.
//
//   p_ij = exp(s_ij - lse_i),  delta_i = go_i . o_i,  ds_ij = p_ij (go_i . v_j - delta_i),
//   gslope_i = - sum_j ds_ij |pos_i - pos_j|,   ds'_ij = ds_ij (1 - tanh^2)   (with a cap),
//   gq_i = scale sum_j ds'_ij k_j,   gk_j = scale sum_i ds'_ij q_i,   gv_j = sum_i p_ij go_i.
//
// Two launches, each recomputing the scores tile by tile: one owns query rows and walks the keys (delta,
// gq, gslope), one owns keys and walks the rows of all query heads that share them (gk, gv).  Every sum
// stays in registers and is written once, so nothing is added by atomics and results are the same from
// run to run; the price is seven matrix products a tile where five would do with atomics.  Distances
// are not differentiated: positions are given.
#include "attention_core.h"

namespace fbev {
namespace {

constexpr int kThreads = 256;

template <typename T, int DP, int KW>
struct Bwd {
  static constexpr int RW = 4 / KW;
  static constexpr int MT = KW == 1 ? 64 : 32 * KW;       // moving rows staged at a time
  static constexpr int kPad = Mma<T, DP>::kPadRow;
  static constexpr size_t kTiles = (size_t)2 * MT * kPad * sizeof(T);
  static constexpr size_t kMerge = (size_t)4 * 32 * (DP + 4) * 4;
  static constexpr size_t kBytes = KW == 1 || kTiles > kMerge ? kTiles : kMerge;
};

// Writes own rows' sums (scaled), or adds the four waves' sums over LDS first.  dst(n) is own row n's
// address or NULL.
template <typename T, int DP, int KW, typename F>
__device__ __forceinline__ void write_own(f32x16 (&acc)[DP / 32], float scale, float* mo, int D, bool vec_out, int kw,
                                          int lane, F dst) {
  constexpr int NB = DP / 32;
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
      for (int k = 0; k < 4; ++k) o += mo[(k * 32 + r) * (DP + 4) + c];
      out[c] = (T)(o * scale);
    }
  }
}

// ---- query rows: delta, gq, gslope

template <typename T, int DP, int KW>
__global__ __launch_bounds__(kThreads) void attn_bwd_rows(AttnArgs a, int tiles) {
  using C = Bwd<T, DP, KW>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, MT = C::MT, RW = C::RW;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[3][MT];
  __shared__ alignas(16) int docs[MT];
  __shared__ int doc_range[4][2];
  __shared__ float slopes[4][3][32];
  T* Ks = (T*)smem;
  T* Vs = Ks + MT * C::kPad;

  const int bid = xcd_block(blockIdx.x, gridDim.x);
  const int tile = bid % tiles, bh = bid / tiles;
  const int b = bh / a.Hk, hk = bh - b * a.Hk;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int first = tile * 32 * RW + rw * 32;
  const Row w = make_row(a, b, hk, min(first + n, a.R - 1));
  const int64_t row_at = (((int64_t)b * a.Tq + w.t) * a.Hq + w.head) * a.D;
  typename M::Frag q[M::kFrags], go[M::kFrags];
  load_row<T, DP>((const T*)a.q + b * a.qs[0] + w.t * a.qs[1] + w.head * a.qs[2], true, a.vec, a.D, h, q);
  load_row<T, DP>((const T*)a.gout + row_at, true, a.vec, a.D, h, go);
  float delta = 0.0f;
  {
    typename M::Frag o[M::kFrags];
    load_row<T, DP>((const T*)a.out + row_at, true, a.vec, a.D, h, o);
#pragma unroll
    for (int f = 0; f < M::kFrags; ++f)
#pragma unroll
      for (int j = 0; j < M::kFragElems; ++j) delta = fmaf((float)go[f][j], (float)o[f][j], delta);
    delta = pair_sum(delta);
  }
  const int64_t stat_at = ((int64_t)b * a.Hq + w.head) * a.Tq + w.t;
  if (kw == 0 && h == 0 && first + n < a.R) a.delta[stat_at] = delta;
  float lse2 = a.lse[stat_at] * kLog2e;
  if (lse2 == kNegInf) lse2 = -kNegInf;                   // a row without weights: all p are 0

  float own[3] = {0.0f, 0.0f, 0.0f}, slope2 = 0.0f;
  if (a.dims) {
    for (int ax = 0; ax < a.dims; ++ax) own[ax] = a.pos_q[((int64_t)b * a.Tq + w.t) * a.dims + ax];
    slope2 = a.slope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head] * kLog2e;
  }
  for (int e = threadIdx.x; e < MT; e += kThreads) pos[0][e] = pos[1][e] = pos[2][e] = 0.0f, docs[e] = 0;
  const int lim_lo = row_limit(a, b, min(first, a.R - 1) / a.G);
  const int lim_hi = row_limit(a, b, min(first + 31, a.R - 1) / a.G);
  const int blk_hi = row_limit(a, b, min(tile * 32 * RW + 32 * RW - 1, a.R - 1) / a.G);
  int dmin = 0, dmax = 0, bmin = 0, bmax = 0;
  if (a.doc_q) {
    dmin = wave_min(w.doc < 0 ? INT32_MAX : w.doc);
    dmax = wave_max(w.doc);
    if (lane == 0) doc_range[wave][0] = dmin, doc_range[wave][1] = dmax;
    __syncthreads();
    bmin = min(min(doc_range[0][0], doc_range[1][0]), min(doc_range[2][0], doc_range[3][0]));
    bmax = max(max(doc_range[0][1], doc_range[1][1]), max(doc_range[2][1], doc_range[3][1]));
  }
  const bool one_doc = dmin == dmax && wave_min(w.doc) == dmin;

  f32x16 acc[NB] = {};
  float sum_ds = 0.0f, sum_dsd = 0.0f, sum_pd = 0.0f;
  const float c1 = a.scale * kLog2e, inv_cap = a.cap > 0.0f ? a.scale / a.cap : 0.0f, c0 = a.cap * kLog2e;
  const int k_end = min(a.Tk, blk_hi + 1);
  for (int s0 = 0; s0 < k_end; s0 += MT) {
    const int nk = min(MT, a.Tk - s0);
    int my_doc = -1;
    if (a.doc_q) {
      if ((int)threadIdx.x < nk) my_doc = a.doc_k[(int64_t)b * a.Tk + s0 + threadIdx.x];
      if (!__syncthreads_or(my_doc >= bmin && my_doc <= bmax)) continue;
    } else {
      __syncthreads();
    }
    stage_rows<T, DP, MT, kThreads>(Ks, nk, a.vec, a.D, [&](int r) {
      return (const T*)a.k + b * a.ks[0] + (int64_t)(s0 + r) * a.ks[1] + hk * a.ks[2];
    });
    stage_rows<T, DP, MT, kThreads>(Vs, nk, a.vec, a.D, [&](int r) {
      return (const T*)a.v + b * a.vs[0] + (int64_t)(s0 + r) * a.vs[1] + hk * a.vs[2];
    });
    if ((int)threadIdx.x < MT) {
      if (a.doc_q) docs[threadIdx.x] = my_doc;
      if (a.dims && (int)threadIdx.x < nk)
        for (int ax = 0; ax < a.dims; ++ax)
          pos[ax][threadIdx.x] = a.pos_k[((int64_t)b * a.Tk + s0 + threadIdx.x) * a.dims + ax];
    }
    __syncthreads();
#pragma unroll 1
    for (int at = 32 * kw; at < MT; at += 32 * KW) {
      const int key0 = s0 + at;
      if (key0 > lim_hi || key0 >= a.Tk) continue;
      bool whole = key0 + 31 <= lim_lo;
      if (a.doc_q) {
        const int d = docs[at + n];
        if (!__any(d >= dmin && d <= dmax)) continue;
        whole = whole && one_doc && __all(d == dmin);
      }
      const T* kt = Ks + at * C::kPad;
      const T* vt = Vs + at * C::kPad;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) s = M::dot(tile_frag<T, DP>(kt, f, lane), q[f], s);
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) dp = M::dot(tile_frag<T, DP>(vt, f, lane), go[f], dp);
      f32x16 th;
      if (a.cap > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          th[i] = tanh_fast<sizeof(T) == 4>(s[i] * inv_cap);
          s[i] = c0 * th[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= c1;
      }
      f32x16 seen;
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int kr = acc_row(i, h);
          seen[i] = key0 + kr <= w.lim && docs[at + kr] == w.doc ? 1.0f : 0.0f;
        }
      }
      f32x16 d;
      if (a.dims) {
        distances<MT>(pos, at, a.dims, own, h, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fmaf(-slope2, d[i], s[i]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(s[i] - lse2);
        s[i] = p * (dp[i] - delta);
        dp[i] = p;
      }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = seen[i] > 0.0f ? s[i] : 0.0f;
      }
      if (a.dims) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool vis = whole || seen[i] > 0.0f;
          sum_ds += s[i];
          sum_dsd = fmaf(s[i], vis ? d[i] : 0.0f, sum_dsd);
          sum_pd += vis ? dp[i] * d[i] : 0.0f;
        }
      }
      if (a.cap > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float g = s[i] * fmaf(-th[i], th[i], 1.0f);
          s[i] = whole || seen[i] > 0.0f ? g : 0.0f;
        }
      }
      if (whole)
        M::template accumulate<NB>(acc, M::pack(s), kt, lane);
      else
        M::template accumulate_masked<NB>(acc, M::pack(s), M::pack(seen), kt, lane);
    }
  }
  write_own<T, DP, KW>(acc, a.scale, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) -> T* {
    if (first + r >= a.R) return nullptr;
    const int t = (first + r) / a.G, head = hk * a.G + (first + r - t * a.G);
    return (T*)a.gq + (((int64_t)b * a.Tq + t) * a.Hq + head) * a.D;
  });
  if (a.gslope) {
    // delta came from the rounded output; ds sums to the error it made (sum_j p_ij = 1), which the distances'
    // mean takes back out: the slope's gradient is fp32 whatever the tensors' type
    sum_ds = pair_sum(sum_ds);
    sum_dsd = pair_sum(sum_dsd);
    sum_pd = pair_sum(sum_pd);
    if constexpr (KW > 1) {
      if (h == 0) slopes[kw][0][n] = sum_ds, slopes[kw][1][n] = sum_dsd, slopes[kw][2][n] = sum_pd;
      __syncthreads();
      sum_ds = (slopes[0][0][n] + slopes[1][0][n]) + (slopes[2][0][n] + slopes[3][0][n]);
      sum_dsd = (slopes[0][1][n] + slopes[1][1][n]) + (slopes[2][1][n] + slopes[3][1][n]);
      sum_pd = (slopes[0][2][n] + slopes[1][2][n]) + (slopes[2][2][n] + slopes[3][2][n]);
    }
    if (kw == 0 && h == 0 && first + n < a.R)
      a.gslope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head] = fmaf(sum_ds, sum_pd, -sum_dsd);
  }
}

// ---- keys: gk, gv

template <typename T, int DP, int KW>
__global__ __launch_bounds__(kThreads) void attn_bwd_keys(AttnArgs a, int tiles) {
  using C = Bwd<T, DP, KW>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, MT = C::MT, RW = C::RW;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[3][MT];
  __shared__ alignas(16) float lse2s[MT], deltas[MT], slope2s[MT];
  __shared__ alignas(16) int docs[MT], lims[MT];
  __shared__ int doc_range[4][2];
  T* Qs = (T*)smem;
  T* Gs = Qs + MT * C::kPad;

  const int bid = xcd_block(blockIdx.x, gridDim.x);
  const int tile = bid % tiles, bh = bid / tiles;
  const int b = bh / a.Hk, hk = bh - b * a.Hk;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int key0 = tile * 32 * RW + rw * 32;              // the wave's keys
  const int key = min(key0 + n, a.Tk - 1);
  typename M::Frag k[M::kFrags], v[M::kFrags];
  load_row<T, DP>((const T*)a.k + b * a.ks[0] + key * a.ks[1] + hk * a.ks[2], true, a.vec, a.D, h, k);
  load_row<T, DP>((const T*)a.v + b * a.vs[0] + key * a.vs[1] + hk * a.vs[2], true, a.vec, a.D, h, v);
  float own[3] = {0.0f, 0.0f, 0.0f};
  for (int ax = 0; ax < a.dims; ++ax) own[ax] = a.pos_k[((int64_t)b * a.Tk + key) * a.dims + ax];
  const int doc = a.doc_k ? a.doc_k[(int64_t)b * a.Tk + key] : 0;
  for (int e = threadIdx.x; e < MT; e += kThreads) {
    pos[0][e] = pos[1][e] = pos[2][e] = 0.0f;
    slope2s[e] = 0.0f;
  }
  int dmin = 0, dmax = 0, bmin = 0, bmax = 0;
  if (a.doc_q) {
    dmin = wave_min(doc < 0 ? INT32_MAX : doc);
    dmax = wave_max(doc);
    if (lane == 0) doc_range[wave][0] = dmin, doc_range[wave][1] = dmax;
    __syncthreads();
    bmin = min(min(doc_range[0][0], doc_range[1][0]), min(doc_range[2][0], doc_range[3][0]));
    bmax = max(max(doc_range[0][1], doc_range[1][1]), max(doc_range[2][1], doc_range[3][1]));
  }
  const bool one_doc = dmin == dmax && wave_min(doc) == dmin;

  f32x16 gk[NB] = {}, gv[NB] = {};
  const float c1 = a.scale * kLog2e, inv_cap = a.cap > 0.0f ? a.scale / a.cap : 0.0f, c0 = a.cap * kLog2e;
  // rows from the first whose order lets it see the workgroup's first key
  const int blk_key = tile * 32 * RW;
  int r_begin = 0;
  if (a.causal && !(a.prefix && a.prefix[b] > blk_key)) {
    const int64_t t0 = (int64_t)blk_key - a.Tk + a.Tq;
    if (t0 > 0) r_begin = (int)((t0 < a.Tq ? t0 : a.Tq) * a.G) / MT * MT;
  }
  for (int s0 = r_begin; s0 < a.R; s0 += MT) {
    const int nr = min(MT, a.R - s0);
    Row w;
    w.doc = -1, w.lim = -1, w.t = 0, w.head = 0;
    if ((int)threadIdx.x < nr) w = make_row(a, b, hk, s0 + threadIdx.x);
    if (a.doc_q) {
      if (!__syncthreads_or(w.doc >= bmin && w.doc <= bmax)) continue;
    } else {
      __syncthreads();
    }
    stage_rows<T, DP, MT, kThreads>(Qs, nr, a.vec, a.D, [&](int r) {
      const int t = (s0 + r) / a.G, head = hk * a.G + (s0 + r - t * a.G);
      return (const T*)a.q + b * a.qs[0] + t * a.qs[1] + head * a.qs[2];
    });
    stage_rows<T, DP, MT, kThreads>(Gs, nr, a.vec, a.D, [&](int r) {
      const int t = (s0 + r) / a.G, head = hk * a.G + (s0 + r - t * a.G);
      return (const T*)a.gout + (((int64_t)b * a.Tq + t) * a.Hq + head) * a.D;
    });
    if ((int)threadIdx.x < MT) {
      docs[threadIdx.x] = w.doc;
      lims[threadIdx.x] = w.lim;
      float l2 = -kNegInf, dl = 0.0f;
      if ((int)threadIdx.x < nr) {
        const int64_t at = ((int64_t)b * a.Hq + w.head) * a.Tq + w.t;
        const float x = a.lse[at] * kLog2e;
        l2 = x == kNegInf ? -kNegInf : x;
        dl = a.delta[at];
        if (a.dims) {
          for (int ax = 0; ax < a.dims; ++ax) pos[ax][threadIdx.x] = a.pos_q[((int64_t)b * a.Tq + w.t) * a.dims + ax];
          slope2s[threadIdx.x] = a.slope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head] * kLog2e;
        }
      }
      lse2s[threadIdx.x] = l2;
      deltas[threadIdx.x] = dl;
    }
    __syncthreads();
#pragma unroll 1
    for (int at = 32 * kw; at < MT; at += 32 * KW) {
      if (s0 + at >= a.R) continue;
      const int lim = s0 + at + n < a.R ? lims[at + n] : INT32_MAX;
      if (!__any(lim != INT32_MAX && lim >= key0)) continue;
      bool whole = __all(lim >= min(key0 + 31, a.Tk - 1));
      if (a.doc_q) {
        const int d = docs[at + n];
        if (!__any(d >= dmin && d <= dmax)) continue;
        whole = whole && one_doc && __all(d == dmin);
      }
      const T* qt = Qs + at * C::kPad;
      const T* gt = Gs + at * C::kPad;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) s = M::dot(tile_frag<T, DP>(qt, f, lane), k[f], s);
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) dp = M::dot(tile_frag<T, DP>(gt, f, lane), v[f], dp);
      f32x16 th;
      if (a.cap > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          th[i] = tanh_fast<sizeof(T) == 4>(s[i] * inv_cap);
          s[i] = c0 * th[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= c1;
      }
      if (a.dims) {
        f32x16 d;
        distances<MT>(pos, at, a.dims, own, h, d);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const f32x4 sl = *(const f32x4*)&slope2s[at + 8 * u + 4 * h];
#pragma unroll
          for (int j = 0; j < 4; ++j) s[4 * u + j] = fmaf(-sl[j], d[4 * u + j], s[4 * u + j]);
        }
      }
      f32x16 seen;
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = at + acc_row(i, h);
          seen[i] = key0 + n <= lims[r] && docs[r] == doc ? 1.0f : 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const f32x4 l2 = *(const f32x4*)&lse2s[at + 8 * u + 4 * h];
        const f32x4 dl = *(const f32x4*)&deltas[at + 8 * u + 4 * h];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * u + j;
          s[i] = __builtin_amdgcn_exp2f(s[i] - l2[j]);
          dp[i] = s[i] * (dp[i] - dl[j]);
          if (a.cap > 0.0f) dp[i] *= fmaf(-th[i], th[i], 1.0f);
        }
      }
      if (whole) {
        M::template accumulate<NB>(gv, M::pack(s), gt, lane);
        M::template accumulate<NB>(gk, M::pack(dp), qt, lane);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = seen[i] > 0.0f ? s[i] : 0.0f;
          dp[i] = seen[i] > 0.0f ? dp[i] : 0.0f;
        }
        const typename M::Values sv = M::pack(seen);
        M::template accumulate_masked<NB>(gv, M::pack(s), sv, gt, lane);
        M::template accumulate_masked<NB>(gk, M::pack(dp), sv, qt, lane);
      }
    }
  }
  auto at_key = [&](void* base, int r) -> T* {
    if (key0 + r >= a.Tk) return nullptr;
    return (T*)base + (((int64_t)b * a.Tk + key0 + r) * a.Hk + hk) * a.D;
  };
  write_own<T, DP, KW>(gv, 1.0f, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) { return at_key(a.gv, r); });
  write_own<T, DP, KW>(gk, a.scale, (float*)smem, a.D, a.vec_out, kw, lane, [&](int r) { return at_key(a.gk, r); });
}

template <typename T, int DP>
hipError_t run(const AttnArgs& a, hipStream_t stream) {
  const int64_t bh = (int64_t)a.B * a.Hk;
  if (a.R > 0) {
    const bool wide = bh * ((a.R + 127) / 128) >= 512;
    const int tiles = (a.R + (wide ? 127 : 31)) / (wide ? 128 : 32);
    if (wide)
      attn_bwd_rows<T, DP, 1><<<dim3((unsigned)(bh * tiles)), kThreads, 0, stream>>>(a, tiles);
    else
      attn_bwd_rows<T, DP, 4><<<dim3((unsigned)(bh * tiles)), kThreads, 0, stream>>>(a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.Tk > 0) {
    const bool wide = bh * ((a.Tk + 127) / 128) >= 512;
    const int tiles = (a.Tk + (wide ? 127 : 31)) / (wide ? 128 : 32);
    if (wide)
      attn_bwd_keys<T, DP, 1><<<dim3((unsigned)(bh * tiles)), kThreads, 0, stream>>>(a, tiles);
    else
      attn_bwd_keys<T, DP, 4><<<dim3((unsigned)(bh * tiles)), kThreads, 0, stream>>>(a, tiles);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t by_width(const AttnArgs& a, hipStream_t stream) {
  if (a.D <= 32) return run<T, 32>(a, stream);
  if (a.D <= 64) return run<T, 64>(a, stream);
  return run<T, 128>(a, stream);
}

}  // namespace

size_t attention_backward_workspace_bytes(const AttnArgs& a) { return (size_t)a.B * a.Hq * a.Tq * sizeof(float); }

hipError_t launch_attention_backward(AttnArgs a, hipStream_t stream) {
  return a.elem_bytes == 4 ? by_width<float>(a, stream) : by_width<__bf16>(a, stream);
}

}  // namespace fbev
