// Attention between queries, cells and tokens, forward.
//
//   s_ij = cap tanh(scale q_i . k_j / cap) - slope_i |pos_i - pos_j|     (cap and bias optional)
//   o_i  = sum_j p_ij v_j,  p = softmax of s over the keys row i sees
//
// One pass over the keys with a running maximum and sum per row (in fp32, base-2 exponentials).  A key
// head's G query heads are rows of one problem (row = token G + head), so single tokens with grouped heads
// still fill a tile and keys are read once for the group.
//
// What bounds it.  bf16, D = 128, 16 heads over 4, 2 x 3100 tokens with a prefix of 2816: 254 us; the counters see matrix
// instructions issue for 86 us and vector ones for 79 us, which alternate within a wave, and every stage waits for its tile
// in full, with two workgroups a CU to fill the waits.  D = 32 with distances (10000 x 10000 cells of 8 heads): 466 us, of
// which vector instructions issue for 256 us (12.6 a score: half a distance and its root, as two heads a wave share them,
// bias, maximum, exponential, sum, two roundings), the quarter rate of exponentials and roots for 90 and matrix ones for 82.
//
// Probabilities of bf16 tensors go into the second product as the sum of two bf16 (16 bits of each): one, rounded by up to
// 2^-8, left outputs 0.0022 off where their own rounding leaves 0.0017.  The second part costs a product and three vector
// instructions a score (the prefix case took 193 us without, the cells 395 us).
#include "attention_core.h"

namespace fbev {
namespace {

constexpr int kThreads = 256;
constexpr int kFewSplits = 8;

// HB heads of a wave (two with a distance bias, whose distances they share), KW waves over the keys of a
// row tile (their sums are joined at the end), 4 / KW row tiles.
template <typename T, int DP, int KW, int HB>
struct Fwd {
  static constexpr int kWaves = KW == 8 ? 8 : 4, kThreads = 64 * kWaves;
  static constexpr int RW = kWaves / KW;                       // row tiles of a workgroup
  static constexpr int KT = KW == 1 ? shared_rows<T>(DP) : 32 * KW;   // keys staged at a time
  static constexpr size_t kTile = (size_t)KT * Tile<T, DP>::kRowBytes;
  static constexpr size_t kTiles = 2 * HB * kTile;
  static constexpr size_t kMerge = (size_t)KW * 32 * (DP + 4) * 4 + KW * 32 * 8;
  static constexpr size_t kBytes = KW == 1 || kTiles > kMerge ? kTiles : kMerge;
};

// Waves a SIMD that the registers allow: the sums take DP / 2 of them for each head, the own rows' fragments DP / 4 (bf16).
template <typename T, int DP>
constexpr int min_waves(int hb) {
  if (sizeof(T) == 4) return DP <= 64 && hb == 1 ? 2 : 1;
  return DP == 128 || hb == 2 ? 2 : DP == 64 ? 3 : 4;
}

// Writes a head's rows (or their split's partial rows); the KW waves of a tile add up their parts first.
template <typename T, int DP, int KW, int HB>
__device__ __forceinline__ void finish(const AttnArgs& a, const Row& w, int first, int split, int64_t bh, int hd, int kw,
                                       int lane, f32x16 (&acc)[DP / 32], float m, float l, char* smem) {
  using C = Fwd<T, DP, KW, HB>;
  constexpr int NB = DP / 32;
  const int n = lane & 31, h = lane >> 5, head = w.head + hd;
  const int b = (int)(bh / a.Hk), hk = (int)(bh - (int64_t)b * a.Hk);
  if constexpr (KW == 1) {                          // 128 rows a workgroup: so many of them that no keys are split
    if (first + n < a.R) {
      T* out = (T*)a.out + (((int64_t)b * a.Tq + w.t) * a.Hq + head) * a.D;
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = 32 * blk + 8 * u + 4 * h;
          if (a.vec_out) {
            if (c < a.D) {
              typedef T V4 __attribute__((ext_vector_type(4)));
              V4 o;
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = (T)(acc[blk][4 * u + j] * inv);
              *(V4*)(out + c) = o;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (c + j < a.D) out[c + j] = (T)(acc[blk][4 * u + j] * inv);
          }
        }
      if (h == 0) a.stats[((int64_t)b * a.Hq + head) * a.Tq + w.t] = make_float2(m, l);
    }
  } else {
    // the waves' sums over their keys, added in wave order
    const bool part = a.splits > 1;
    float* mo = (float*)smem;                       // [KW][32][DP + 4]
    float* ml = mo + KW * 32 * (DP + 4);            // [KW][32][2]
    __syncthreads();
    if (h == 0) ml[(kw * 32 + n) * 2] = m, ml[(kw * 32 + n) * 2 + 1] = l;
    __syncthreads();
    float top = kNegInf;
#pragma unroll
    for (int k = 0; k < KW; ++k) top = fmaxf(top, ml[(k * 32 + n) * 2]);
    float tot = 0.0f;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const float mk = ml[(k * 32 + n) * 2];
      tot += ml[(k * 32 + n) * 2 + 1] * (mk == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(mk - top));
    }
    const float f = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = acc[blk][4 * u + j] * f;
        *(f32x4*)(mo + (kw * 32 + n) * (DP + 4) + 32 * blk + 8 * u + 4 * h) = o;
      }
    if (kw == 0 && h == 0 && first + n < a.R) {
      if (part) {
        float* po = a.part + (((int64_t)split * a.B * a.Hk + bh) * a.R + w.r) * (a.D + 2);
        po[a.D] = top, po[a.D + 1] = tot;
      } else {
        a.stats[((int64_t)b * a.Hq + head) * a.Tq + w.t] = make_float2(top, tot);
      }
    }
    __syncthreads();
    if (kw == 0 && h == 0) ml[n * 2] = part ? 1.0f : (tot > 0.0f || tot != tot ? 1.0f / tot : 0.0f);
    __syncthreads();
    const int rows = min(32, a.R - first);
    for (int e = threadIdx.x; e < rows * DP; e += C::kThreads) {
      const int r = e / DP, c = e - r * DP;
      if (c >= a.D) continue;
      float o = 0.0f;
#pragma unroll
      for (int k = 0; k < KW; ++k) o += mo[(k * 32 + r) * (DP + 4) + c];
      const int row = first + r, t = row / a.G, hh = hk * a.G + (row - t * a.G);
      if (part)
        a.part[(((int64_t)split * a.B * a.Hk + bh) * a.R + row) * (a.D + 2) + c] = o;
      else
        ((T*)a.out)[(((int64_t)b * a.Tq + t) * a.Hq + hh) * a.D + c] = (T)(o * ml[r * 2]);
    }
  }
}

template <typename T, int DP, int KW, int HB, bool BIAS>
__global__ __launch_bounds__((Fwd<T, DP, KW, HB>::kThreads), (min_waves<T, DP>(HB))) void attn_fwd(AttnArgs a, int tiles,
                                                                                                   int blocks) {
  using C = Fwd<T, DP, KW, HB>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, KT = C::KT, RW = C::RW;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[BIAS ? 3 * KT : 1];   // [key][axis]
  __shared__ alignas(16) int docs[KT];
  __shared__ int doc_range[C::kWaves][2];
  __shared__ uint32_t stage_bits;
  char* Ks = smem;                                        // HB tiles each
  char* Vs = smem + HB * C::kTile;

  const int block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const int bid = xcd_block(block, blocks);
  const int split = bid % a.splits, bh = bid / a.splits / tiles;
  const int order = bid / a.splits - bh * tiles;
  const int tile = a.causal ? tiles - 1 - order : order;  // causal rows: those with the most keys first
  const int b = bh / (a.Hk / HB), hk = (bh - b * (a.Hk / HB)) * HB;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int first = tile * 32 * RW + rw * 32;            // the wave's rows
  const Row w = make_row(a, b, hk, min(first + n, a.R - 1));
  const Unit un = make_unit(a);
  const Stager st = make_stager<T, DP>(a.D);
  typename M::Frag q[HB][M::kFrags];
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    load_row<T, DP>((const T*)a.q + b * a.qs[0] + w.t * a.qs[1] + (w.head + i) * a.qs[2], a.vec, a.D, h, q[i]);
    sign_row<T, DP>(a, q[i]);
  }

  float own[3] = {0.0f, 0.0f, 0.0f}, slope[HB] = {};
  if constexpr (BIAS) {
    own_point(a.pos_q + ((int64_t)b * a.Tq + w.t) * a.dims, a.dims, h, own);
#pragma unroll
    for (int i = 0; i < HB; ++i) slope[i] = a.slope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head + i] / un.raw;
  }
  for (int e = threadIdx.x; e < KT; e += C::kThreads) docs[e] = 0;
  // the keys the workgroup's and the wave's rows can see by order
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
  const bool one_doc = dmin == dmax && wave_min(w.doc) == dmin;   // every row of the wave in one document

  f32x16 acc[HB][NB] = {};
  uint32_t odd[HB][NB] = {};
  float m[HB], l[HB];
#pragma unroll
  for (int i = 0; i < HB; ++i) m[i] = kNegInf, l[i] = 0.0f;
  const int k_begin = split * a.split_keys;
  const int k_end = min(min(a.Tk, blk_hi + 1), (split + 1) * a.split_keys);
  uint32_t stages = 0;
  for (int s0 = k_begin; s0 < k_end; s0 += KT) {
    const int nk = min(KT, a.Tk - s0);
    int my_doc = -1;
    if (a.doc_q) {
      const int stage = (s0 - k_begin) / KT & 31;
      if (stage == 0)
        stages = stages_with<KT, C::kThreads>(&stage_bits, s0, k_end, bmin, bmax, [&](int k) { return a.doc_k[(int64_t)b * a.Tk + k]; });
      if (!((stages >> stage) & 1)) continue;
      if ((int)threadIdx.x < nk) my_doc = a.doc_k[(int64_t)b * a.Tk + s0 + threadIdx.x];
    }
    __syncthreads();
    // some row of the workgroup may not see some key
    const bool mixed = a.doc_q != nullptr || (a.causal && s0 + KT - 1 > blk_lo);
#pragma unroll
    for (int i = 0; i < HB; ++i) {
      stage_rows<T, DP, KT, C::kThreads>(Ks + i * C::kTile, (const T*)a.k + b * a.ks[0] + s0 * a.ks[1] + (hk + i) * a.ks[2], a.ks[1],
                            nk, a.vec, a.D, st);
      stage_rows<T, DP, KT, C::kThreads>(Vs + i * C::kTile, (const T*)a.v + b * a.vs[0] + s0 * a.vs[1] + (hk + i) * a.vs[2], a.vs[1],
                            nk, a.vec, a.D, st);
    }
    if (a.doc_q && (int)threadIdx.x < KT) docs[threadIdx.x] = my_doc;
    if constexpr (BIAS) stage_floats<C::kThreads>(pos, a.pos_k + ((int64_t)b * a.Tk + s0) * a.dims, nk * a.dims, KT * a.dims);
    // which of the tile's keys (16 of the lane's half) the lane's row sees
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
    if (mixed && __builtin_expect(__syncthreads_or(holds_odd<T, DP, HB * KT, C::kThreads>(Vs)), 0)) {
#pragma unroll 1
      for (int at = 32 * kw; at < KT; at += 32 * KW) {
        const uint32_t vis = visible(at);
#pragma unroll
        for (int hd = 0; hd < HB; ++hd)
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) odd[hd][blk] |= find_odd<T, DP>(Vs + hd * C::kTile, at, blk, vis, lane);
      }
      __syncthreads();
      clean_rows<T, DP, HB * KT, C::kThreads>(Vs);
      __syncthreads();
    }
#pragma unroll 1
    for (int sub = 0; sub < KT / (32 * KW); ++sub) {
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
#pragma unroll
      for (int hd = 0; hd < HB; ++hd) {
        if constexpr (HB > 1) __builtin_amdgcn_sched_barrier(0);      // one head's registers at a time
        f32x16 s = tile_dot<T, DP>(Ks + hd * C::kTile, at, q[hd], lane);
        if (a.cap > 0.0f) cap_scores<T>(s, un);
        if constexpr (BIAS) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = fmaf(-slope[hd], d[i], s[i]);
        }
        if (!whole) {
          const uint32_t vis = opaque(seen);
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = (vis >> i) & 1 ? s[i] : kNegInf;
        }
        if constexpr (HB > 1) __builtin_amdgcn_sched_barrier(0);
        float top = fmaxf(s[0], s[1]);
#pragma unroll
        for (int i = 2; i < 16; i += 2) top = fmaxf(fmaxf(top, s[i]), s[i + 1]);
        top = pair_max(top) * un.unit;
        // the maximum is only moved when some row's grew by more than 2^8: sums and products stay in range, and after
        // a few tiles hardly any wave scales its sums again
        if (__any(top > m[hd] + 8.0f)) {
          const float m2 = fmaxf(m[hd], top);
          const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[hd] - m2);
          m[hd] = m2;
          l[hd] *= f;
#pragma unroll
          for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[hd][blk][i] *= f;
        }
        const float base = m[hd] == kNegInf ? 0.0f : -m[hd];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], un.unit, base));
          sum += s[i];
        }
        l[hd] += sum;
        pin(l[hd]);
        if constexpr (HB > 1) __builtin_amdgcn_sched_barrier(0);
        M::template accumulate<NB>(acc[hd], s, Vs + hd * C::kTile, at, lane);
      }
    }
  }

#pragma unroll
  for (int hd = 0; hd < HB; ++hd) {
    add_odd<NB>(acc[hd], odd[hd]);
    finish<T, DP, KW, HB>(a, w, first, split, (int64_t)b * a.Hk + hk + hd, hd, kw, lane, acc[hd], m[hd],
                          pair_sum(l[hd]), smem);
  }
}

// Joins the splits of a row.  Few of them: a wave a row, in split order.
template <typename T>
__global__ __launch_bounds__(kThreads) void attn_join_few(AttnArgs a) {
  const int64_t rows = (int64_t)a.B * a.Hk * a.R, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int lane = threadIdx.x & 63;
  const int64_t stride = rows * (a.D + 2);
  const float* p = a.part + row * (a.D + 2);
  float m[kFewSplits], top = kNegInf;
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    m[s] = s < a.splits ? p[s * stride + a.D] : kNegInf;
    top = fmaxf(top, m[s]);
  }
  const float base = top == kNegInf ? 0.0f : top;
  float tot = 0.0f, o[2] = {0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s)
    if (s < a.splits) {
      const float f = __builtin_amdgcn_exp2f(m[s] - base);
      tot = fmaf(p[s * stride + a.D + 1], f, tot);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (lane + 64 * j < a.D) o[j] = fmaf(p[s * stride + lane + 64 * j], f, o[j]);
    }
  const int64_t bh = row / a.R;
  const int r = (int)(row - bh * a.R), t = r / a.G, b = (int)(bh / a.Hk);
  const int head = (int)(bh - (int64_t)b * a.Hk) * a.G + (r - t * a.G);
  const float inv = tot > 0.0f || tot != tot ? 1.0f / tot : 0.0f;
  T* out = (T*)a.out + (((int64_t)b * a.Tq + t) * a.Hq + head) * a.D;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 64 * j < a.D) out[lane + 64 * j] = (T)(o[j] * inv);
  if (lane == 0) a.stats[((int64_t)b * a.Hq + head) * a.Tq + t] = make_float2(top, tot);
}

// Many: one workgroup a row.  Wave w joins splits w, w + WAVES, ... with a running maximum, kJoinRun of them at a time whose
// loads all go out at once (what they wait for is the time: 79 splits of 16 rows took 13 us when the maximum, and then four
// splits at a time, were waited for in turn); the waves' results are joined in wave order.
constexpr int kJoinRun = 8;

template <typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void attn_join(AttnArgs a) {
  __shared__ float tops[WAVES], sums[WAVES], part[WAVES][128];
  const int64_t rows = (int64_t)a.B * a.Hk * a.R, row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t stride = rows * (a.D + 2);
  const float* p = a.part + row * (a.D + 2);
  float top = kNegInf, tot = 0.0f, o[2] = {0.0f, 0.0f};
#pragma unroll 1
  for (int s0 = wave; s0 < a.splits; s0 += WAVES * kJoinRun) {
    float m[kJoinRun], l[kJoinRun], x[kJoinRun][2];
    float next = top;
#pragma unroll
    for (int i = 0; i < kJoinRun; ++i) {
      const int s = s0 + i * WAVES;
      const bool in = s < a.splits;
      const float* q = p + (in ? s : s0) * stride;
      m[i] = in ? q[a.D] : kNegInf;
      l[i] = q[a.D + 1];
#pragma unroll
      for (int j = 0; j < 2; ++j) x[i][j] = lane + 64 * j < a.D ? q[lane + 64 * j] : 0.0f;
      next = fmaxf(next, m[i]);
      if (!in) l[i] = x[i][0] = x[i][1] = 0.0f;
    }
    const float base = next == kNegInf ? 0.0f : next, back = __builtin_amdgcn_exp2f(top - base);
    top = next;
    tot *= back, o[0] *= back, o[1] *= back;
#pragma unroll
    for (int i = 0; i < kJoinRun; ++i) {
      const float f = __builtin_amdgcn_exp2f(m[i] - base);
      tot = fmaf(l[i], f, tot);
      o[0] = fmaf(x[i][0], f, o[0]);
      o[1] = fmaf(x[i][1], f, o[1]);
    }
  }
  if (lane == 0) tops[wave] = top, sums[wave] = tot;
  part[wave][lane] = o[0], part[wave][lane + 64] = o[1];
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= 128) return;
  top = tops[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) top = fmaxf(top, tops[w]);
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
  tot = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const float f = __builtin_amdgcn_exp2f(tops[w] - base);
    tot = fmaf(sums[w], f, tot);
    sum = fmaf(part[w][c], f, sum);
  }
  const int64_t bh = row / a.R;
  const int r = (int)(row - bh * a.R), t = r / a.G, b = (int)(bh / a.Hk);
  const int head = (int)(bh - (int64_t)b * a.Hk) * a.G + (r - t * a.G);
  const float inv = tot > 0.0f || tot != tot ? 1.0f / tot : 0.0f;
  if (c < a.D) ((T*)a.out)[(((int64_t)b * a.Tq + t) * a.Hq + head) * a.D + c] = (T)(sum * inv);
  if (c == 0) a.stats[((int64_t)b * a.Hq + head) * a.Tq + t] = make_float2(top, tot);
}

struct Plan {
  int kw, hb, tiles, splits, split_keys;
};

Plan make_plan(const AttnArgs& a) {
  Plan p;
  const int64_t bh = (int64_t)a.B * a.Hk;
  // two heads a wave where they share the distances and there are enough of them to fill the card
  p.hb = a.dims > 0 && a.G == 1 && a.Hk % 2 == 0 && a.D <= 32 && bh * ((a.R + 31) / 32) >= 1024 ? 2 : 1;
  // row tiles that share staged keys when they fill the card several times over, else keys over the waves
  p.kw = bh / p.hb * ((a.R + 127) / 128) >= (a.D <= 64 ? 2048 : 512) ? 1 : 4;
  const int64_t row_tiles = bh * ((a.R + 31) / 32);
  // under 512 workgroups of four waves a SIMD has one wave or none: eight a workgroup (900 fp32 queries, 232 workgroups:
  // 22.4 us against 25.7 us with the keys in two splits); 928 workgroups lose by it (32.1 against 27.3 us)
  const int dp = a.D <= 32 ? 32 : a.D <= 64 ? 64 : 128;
  if (p.kw == 4 && p.hb == 1 && (a.elem_bytes == 4 ? eight_waves<float>(dp) : eight_waves<__bf16>(dp)) &&
      row_tiles >= 128 && row_tiles < 512)
    p.kw = 8;
  const int rows = p.kw == 1 ? 128 : 32, kt = p.kw == 1 ? 128 : 32 * p.kw;
  p.tiles = (a.R + rows - 1) / rows;
  // under 128 workgroups the keys are split over several and joined: at least 512 keys each and four workgroups a CU at most,
  // but down to a stage of 128 keys while there is not a workgroup a CU (one token over 8000 keys of 2 heads: 32 workgroups
  // take 10.9 us, 126 take 8.8 us; beyond that the join costs what shorter walks gain)
  const int64_t blocks = bh / p.hb * p.tiles;
  p.splits = 1;
  if (blocks < 128) {
    const auto at_most = [](int64_t x, int64_t y) { return x < y ? x : y; };
    const int64_t keys = a.Tk;
    const int64_t want = at_most((1024 + blocks - 1) / blocks, (keys + 511) / 512);
    const int64_t fill = at_most((256 + blocks - 1) / blocks, (keys + 127) / 128);
    p.splits = (int)(want > fill ? want : fill);
    if (p.splits < 1) p.splits = 1;
  }
  const int per = (a.Tk + p.splits - 1) / p.splits;
  p.split_keys = (per + kt - 1) / kt * kt;
  if (p.split_keys < kt) p.split_keys = kt;
  p.splits = a.Tk > 0 ? (a.Tk + p.split_keys - 1) / p.split_keys : 1;
  return p;
}

template <typename T, int DP, int HB, bool BIAS>
void launch(const AttnArgs& a, const Plan& p, hipStream_t stream) {
  const int blocks = (int)((int64_t)a.B * a.Hk / HB * p.tiles * p.splits);
  const dim3 grid = grid_rows(blocks);
  if (p.kw == 1) {
    attn_fwd<T, DP, 1, HB, BIAS><<<grid, 256, 0, stream>>>(a, p.tiles, blocks);
  } else if (p.kw == 4) {
    attn_fwd<T, DP, 4, HB, BIAS><<<grid, 256, 0, stream>>>(a, p.tiles, blocks);
  } else {
    if constexpr (HB == 1 && eight_waves<T>(DP)) attn_fwd<T, DP, 8, HB, BIAS><<<grid, 512, 0, stream>>>(a, p.tiles, blocks);
  }
}

template <typename T, int DP>
hipError_t run(AttnArgs& a, const Plan& p, hipStream_t stream) {
  if (a.dims == 0) {
    launch<T, DP, 1, false>(a, p, stream);
  } else if (p.hb == 1) {
    launch<T, DP, 1, true>(a, p, stream);
  } else {
    if constexpr (DP == 32) launch<T, DP, 2, true>(a, p, stream);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)a.B * a.Hk * a.R;
  if (p.splits <= kFewSplits)
    attn_join_few<T><<<dim3((unsigned)((rows + 3) / 4)), kThreads, 0, stream>>>(a);
  else if (p.splits <= 4 * kJoinRun)
    attn_join<T, 4><<<dim3((unsigned)rows), 256, 0, stream>>>(a);
  else
    attn_join<T, 16><<<dim3((unsigned)rows), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t by_width(AttnArgs& a, const Plan& p, hipStream_t stream) {
  if (a.D <= 32) return run<T, 32>(a, p, stream);
  if (a.D <= 64) return run<T, 64>(a, p, stream);
  return run<T, 128>(a, p, stream);
}

}  // namespace

size_t attention_forward_workspace_bytes(const AttnArgs& a) {
  const Plan p = make_plan(a);
  return p.splits == 1 ? 0 : (size_t)p.splits * a.B * a.Hk * a.R * (a.D + 2) * sizeof(float);
}

hipError_t launch_attention_forward(AttnArgs a, hipStream_t stream) {
  const Plan p = make_plan(a);
  a.splits = p.splits;
  a.split_keys = p.split_keys;
  return a.elem_bytes == 4 ? by_width<float>(a, p, stream) : by_width<__bf16>(a, p, stream);
}

}  // namespace fbev
