// Attention between queries, cells and tokens, forward.
//
//   s_ij = cap tanh(scale q_i . k_j / cap) - slope_i |pos_i - pos_j|     (cap and bias optional)
//   o_i  = sum_j p_ij v_j,  p = softmax of s over the keys row i sees,  lse_i = log sum_j exp(s_ij)
//
// One pass over the keys with a running maximum and sum per row (in fp32, base-2 exponentials).  A key
// head's G query heads are rows of one problem (row = token G + head), so single tokens with grouped heads
// still fill a tile and keys are read once for the group.
#include "attention_core.h"

namespace fbev {
namespace {

constexpr int kThreads = 256;

template <typename T, int DP, int KW>
struct Fwd {
  static constexpr int RW = 4 / KW;                       // row tiles of a workgroup
  static constexpr int KT = KW == 1 ? 64 : 32 * KW;       // keys staged at a time
  static constexpr int kPad = Mma<T, DP>::kPadRow;
  static constexpr size_t kTiles = (size_t)2 * KT * kPad * sizeof(T);
  static constexpr size_t kMerge = (size_t)4 * 32 * (DP + 4) * 4 + 4 * 32 * 8;
  static constexpr size_t kBytes = KW == 1 || kTiles > kMerge ? kTiles : kMerge;
};

template <typename T, int DP, int KW>
__global__ __launch_bounds__(kThreads) void attn_fwd(AttnArgs a, int tiles) {
  using C = Fwd<T, DP, KW>;
  using M = Mma<T, DP>;
  constexpr int NB = DP / 32, KT = C::KT, RW = C::RW;
  __shared__ alignas(16) char smem[C::kBytes];
  __shared__ alignas(16) float pos[3][KT];
  __shared__ alignas(16) int docs[KT];
  __shared__ int doc_range[4][2];
  T* Ks = (T*)smem;
  T* Vs = Ks + KT * C::kPad;

  const int bid = xcd_block(blockIdx.x, gridDim.x);
  const int split = bid % a.splits, tile = bid / a.splits % tiles, bh = bid / a.splits / tiles;
  const int b = bh / a.Hk, hk = bh - b * a.Hk;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, h = lane >> 5;
  const int rw = wave / KW, kw = wave - rw * KW;
  const int first = tile * 32 * RW + rw * 32;            // the wave's rows
  const Row w = make_row(a, b, hk, min(first + n, a.R - 1));
  typename M::Frag q[M::kFrags];
  load_row<T, DP>((const T*)a.q + b * a.qs[0] + w.t * a.qs[1] + w.head * a.qs[2], true, a.vec, a.D, h, q);

  float own[3] = {0.0f, 0.0f, 0.0f}, slope2 = 0.0f;
  if (a.dims) {
    for (int ax = 0; ax < a.dims; ++ax) own[ax] = a.pos_q[((int64_t)b * a.Tq + w.t) * a.dims + ax];
    slope2 = a.slope[((int64_t)b * a.Tq + w.t) * a.Hq + w.head] * kLog2e;
  }
  for (int e = threadIdx.x; e < KT; e += kThreads) pos[0][e] = pos[1][e] = pos[2][e] = 0.0f, docs[e] = 0;
  // the keys the workgroup's and the wave's rows can see by order
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
  const bool one_doc = dmin == dmax && wave_min(w.doc) == dmin;   // every row of the wave in one document

  f32x16 acc[NB] = {};
  float m = kNegInf, l = 0.0f;
  const float c1 = a.scale * kLog2e, inv_cap = a.cap > 0.0f ? a.scale / a.cap : 0.0f, c0 = a.cap * kLog2e;
  const int k_begin = split * a.split_keys;
  const int k_end = min(min(a.Tk, blk_hi + 1), (split + 1) * a.split_keys);
  for (int s0 = k_begin; s0 < k_end; s0 += KT) {
    const int nk = min(KT, a.Tk - s0);
    int my_doc = -1;
    if (a.doc_q) {
      if ((int)threadIdx.x < nk) my_doc = a.doc_k[(int64_t)b * a.Tk + s0 + threadIdx.x];
      if (!__syncthreads_or(my_doc >= bmin && my_doc <= bmax)) continue;
    } else {
      __syncthreads();
    }
    stage_rows<T, DP, KT, kThreads>(Ks, nk, a.vec, a.D, [&](int r) {
      return (const T*)a.k + b * a.ks[0] + (int64_t)(s0 + r) * a.ks[1] + hk * a.ks[2];
    });
    stage_rows<T, DP, KT, kThreads>(Vs, nk, a.vec, a.D, [&](int r) {
      return (const T*)a.v + b * a.vs[0] + (int64_t)(s0 + r) * a.vs[1] + hk * a.vs[2];
    });
    if ((int)threadIdx.x < KT) {
      if (a.doc_q) docs[threadIdx.x] = my_doc;
      if (a.dims && (int)threadIdx.x < nk)
        for (int ax = 0; ax < a.dims; ++ax)
          pos[ax][threadIdx.x] = a.pos_k[((int64_t)b * a.Tk + s0 + threadIdx.x) * a.dims + ax];
    }
    __syncthreads();
#pragma unroll 1
    for (int at = 32 * kw; at < KT; at += 32 * KW) {
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
      f32x16 s = {};
#pragma unroll
      for (int f = 0; f < M::kFrags; ++f) s = M::dot(tile_frag<T, DP>(kt, f, lane), q[f], s);
      if (a.cap > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = c0 * tanh_fast<sizeof(T) == 4>(s[i] * inv_cap);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= c1;
      }
      if (a.dims) {
        f32x16 d;
        distances<KT>(pos, at, a.dims, own, h, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = fmaf(-slope2, d[i], s[i]);
      }
      f32x16 seen;
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int kr = acc_row(i, h);
          const bool vis = key0 + kr <= w.lim && docs[at + kr] == w.doc;
          seen[i] = vis ? 1.0f : 0.0f;
          s[i] = vis ? s[i] : kNegInf;
        }
      }
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
      top = pair_max(top);
      // the maximum is only moved when some row's grew by more than 2^8: sums and products stay in range
      if (__any(top > m + 8.0f)) {
        const float m2 = fmaxf(m, top);
        const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - m2);
        m = m2;
        l *= f;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[blk][i] *= f;
      }
      const float base = m == kNegInf ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(s[i] - base);
        sum += s[i];
      }
      l += sum;
      if (whole)
        M::template accumulate<NB>(acc, M::pack(s), vt, lane);
      else
        M::template accumulate_masked<NB>(acc, M::pack(s), M::pack(seen), vt, lane);
    }
  }
  l = pair_sum(l);

  const bool part = a.splits > 1;
  if constexpr (KW == 1) {
    if (first + n < a.R) {
      float* po = part ? a.part + (((int64_t)split * a.B * a.Hk + bh) * a.R + w.r) * (a.D + 2) : nullptr;
      T* out = (T*)a.out + (((int64_t)b * a.Tq + w.t) * a.Hq + w.head) * a.D;
      const float inv = part ? 1.0f : (l > 0.0f || l != l ? 1.0f / l : 0.0f);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = 32 * blk + 8 * u + 4 * h;
          if (part) {
            for (int j = 0; j < 4; ++j)
              if (c + j < a.D) po[c + j] = acc[blk][4 * u + j];
          } else if (a.vec_out) {
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
      if (h == 0) {
        if (part)
          po[a.D] = m, po[a.D + 1] = l;
        else
          a.lse[((int64_t)b * a.Hq + w.head) * a.Tq + w.t] = l == 0.0f ? kNegInf : m * kLn2 + logf(l);
      }
    }
  } else {
    // the four waves' sums over their keys, added in wave order
    float* mo = (float*)smem;                       // [4][32][DP + 4]
    float* ml = mo + 4 * 32 * (DP + 4);             // [4][32][2]
    __syncthreads();
    if (h == 0) ml[(kw * 32 + n) * 2] = m, ml[(kw * 32 + n) * 2 + 1] = l;
    __syncthreads();
    float top = kNegInf;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[(k * 32 + n) * 2]);
    float tot = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
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
        a.lse[((int64_t)b * a.Hq + w.head) * a.Tq + w.t] = tot == 0.0f ? kNegInf : top * kLn2 + logf(tot);
      }
    }
    __syncthreads();
    if (kw == 0 && h == 0) ml[n * 2] = part ? 1.0f : (tot > 0.0f || tot != tot ? 1.0f / tot : 0.0f);
    __syncthreads();
    const int rows = min(32, a.R - first);
    for (int e = threadIdx.x; e < rows * DP; e += kThreads) {
      const int r = e / DP, c = e - r * DP;
      if (c >= a.D) continue;
      float o = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) o += mo[(k * 32 + r) * (DP + 4) + c];
      const int row = first + r, t = row / a.G, head = hk * a.G + (row - t * a.G);
      if (part)
        a.part[(((int64_t)split * a.B * a.Hk + bh) * a.R + row) * (a.D + 2) + c] = o;
      else
        ((T*)a.out)[(((int64_t)b * a.Tq + t) * a.Hq + head) * a.D + c] = (T)(o * ml[r * 2]);
    }
  }
}

// Joins the splits of a row, in split order: one wave a row.
template <typename T>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  const int64_t rows = (int64_t)a.B * a.Hk * a.R, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int lane = threadIdx.x & 63;
  const int64_t stride = rows * (a.D + 2);
  const float* p = a.part + row * (a.D + 2);
  float top = kNegInf;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, p[s * stride + a.D]);
  float tot = 0.0f, o[2] = {0.0f, 0.0f};
  for (int s = 0; s < a.splits; ++s) {
    const float mk = p[s * stride + a.D];
    const float f = mk == kNegInf ? (top == kNegInf ? 1.0f : 0.0f) : __builtin_amdgcn_exp2f(mk - top);
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
  if (lane == 0) a.lse[((int64_t)b * a.Hq + head) * a.Tq + t] = tot == 0.0f ? kNegInf : top * kLn2 + logf(tot);
}

struct Plan {
  int kw, tiles, splits, split_keys;
};

Plan make_plan(const AttnArgs& a) {
  Plan p;
  const int64_t bh = (int64_t)a.B * a.Hk;
  // row tiles that share staged keys when they fill the card (two workgroups a CU), else keys over the waves
  p.kw = bh * ((a.R + 127) / 128) >= 512 ? 1 : 4;
  const int rows = 32 * (4 / p.kw), kt = p.kw == 1 ? 64 : 128;
  p.tiles = (a.R + rows - 1) / rows;
  const int64_t blocks = bh * p.tiles;
  p.splits = 1;
  if (blocks < 256) {
    int64_t want = (1024 + blocks - 1) / blocks;
    const int64_t most = (a.Tk + 4 * kt - 1) / (4 * kt);
    if (want > most) want = most;
    p.splits = want < 1 ? 1 : (int)want;
  }
  const int per = (a.Tk + p.splits - 1) / p.splits;
  p.split_keys = (per + kt - 1) / kt * kt;
  if (p.split_keys < kt) p.split_keys = kt;
  p.splits = a.Tk > 0 ? (a.Tk + p.split_keys - 1) / p.split_keys : 1;
  return p;
}

template <typename T, int DP>
hipError_t run(AttnArgs& a, const Plan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.B * a.Hk * p.tiles * p.splits));
  if (p.kw == 1)
    attn_fwd<T, DP, 1><<<grid, kThreads, 0, stream>>>(a, p.tiles);
  else
    attn_fwd<T, DP, 4><<<grid, kThreads, 0, stream>>>(a, p.tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)a.B * a.Hk * a.R;
  attn_join<T><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, stream>>>(a);
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
