// Group norm with an activation on channels-last maps, forward and backward.
//
//   xh = (x - mean) rstd   (mean, variance over the pixels and channels of an (image, group)),
//   z = weight xh + bias,  y = act(z);
//   dz = gy act'(z),  gbias = sum dz,  gweight = sum dz xh,  u = weight dz,
//   gx = rstd (u - mean(u) - xh mean(u xh)).
//
// What bounds it: memory.  A workgroup holds its part of an image in registers (R pieces of 16 bytes a
// thread, all loaded before the first is used), so within it the mean comes first and the squares are
// taken around it.  Two forms, by the bytes of an image's slab of whole groups:
//   - a slab that fits one workgroup's registers is normalised in one launch with one read;
//   - otherwise one launch leaves each chunk's (mean, sum of squares around it) in the workspace, and the
//     next merges an image's chunks (pairwise formula, in their order) and normalises; its blocks take the
//     chunks in the same order, so the second read finds much of them in the same L2.
// The backward has the same two forms with the per-channel sums of dz and dz xh; the parameters'
// gradients are column sums over chunks and images in a fixed order.  All results are deterministic.
#include "encoder.h"

#include "../../include/flashbev.h"

namespace fbev {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T e[V];
};

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == FBEV_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == FBEV_ACT_SILU) return z / (1.0f + __expf(-z));
  if constexpr (ACT == FBEV_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == FBEV_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == FBEV_ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (ACT == FBEV_ACT_GELU)
    return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
  return 1.0f;
}

// A workgroup's share: channels [c0, c0 + nv V) (whole groups) of pixels [s0, s0 + ns).  Thread (ty, cv)
// holds channel piece cv of pixels s0 + ty, s0 + ty + TY, ...
struct Share {
  int img, c0, nv, s0, ns, TY, ty, cv;
  bool active;
};

// Sums over the workgroup per group, for two values a channel: buf[(ty nv + cv) per + j] holds a thread's
// value for channel c0 + cv V + j.  out[g] = sums of the share's groups, valid in all threads after the call.
// `per` is 1 when a piece lies inside one group (its channels were summed first) and V otherwise.
template <int BLOCK>
__device__ __forceinline__ void group_sums(const float* buf, float* out, int TY, int cols, int gcols) {
  const int ng = cols / gcols;
  int gt = 64;
  while (gt > 1 && gt * ng > BLOCK) gt >>= 1;
  __syncthreads();
  for (int g0 = 0; g0 < ng; g0 += BLOCK / gt) {
    const int g = g0 + (int)threadIdx.x / gt, l = threadIdx.x & (gt - 1);
    float s = 0.0f;
    if (g < ng) {
      const int n = TY * gcols;
      for (int e = l; e < n; e += gt) {
        const int ty = e / gcols, c = e - ty * gcols;
        s += buf[ty * cols + g * gcols + c];
      }
    }
    for (int o = gt >> 1; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (g < ng && l == 0) out[g] = s;
  }
  __syncthreads();
}

template <int BLOCK, int V>
struct Lds {
  float buf[BLOCK * V];
  float g1[BLOCK * V];     // per group of the share (at most one group a channel)
  float g2[BLOCK * V];
};

template <int BLOCK, int V>
__device__ __forceinline__ Share make_share(int img, int c0, int nch, int s0, int ns) {
  Share w;
  w.img = img;
  w.c0 = c0;
  w.nv = nch / V;
  w.s0 = s0;
  w.ns = ns;
  w.TY = BLOCK / w.nv;
  w.ty = threadIdx.x / w.nv;
  w.cv = threadIdx.x - w.ty * w.nv;
  w.active = w.ty < w.TY;
  return w;
}

template <typename T, int V, int R>
__device__ __forceinline__ void load_share(const NormArgs& a, const Share& w, Piece<T, V> (&x)[R]) {
  const T* base = (const T*)a.x + w.img * a.x_image + w.c0 + w.cv * V;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s = w.ty + r * w.TY;
    if (w.active && s < w.ns) x[r] = *(const Piece<T, V>*)(base + (int64_t)(w.s0 + s) * a.x_pixel);
  }
}

// The same rows of a contiguous tensor.
template <typename T, int V, int R>
__device__ __forceinline__ void load_rows(const void* src, const NormArgs& a, const Share& w, Piece<T, V> (&x)[R]) {
  const T* base = (const T*)src + (int64_t)w.img * a.pixels * a.C + w.c0 + w.cv * V;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s = w.ty + r * w.TY;
    if (w.active && s < w.ns) x[r] = *(const Piece<T, V>*)(base + (int64_t)(w.s0 + s) * a.C);
  }
}

// Writes a thread's per-channel values into the buffer (summed over the piece when per is 1).
template <int V>
__device__ __forceinline__ void put_sums(float* buf, const Share& w, int per, const float (&v)[V]) {
  if (!w.active) return;
  float* at = buf + (w.ty * w.nv + w.cv) * per;
  if (per == 1) {
    float s = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) s += v[j];
    at[0] = s;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) at[j] = v[j];
  }
}

// Mean and sum of squares around it of every group of the share, into L.g1 and L.g2.
template <int BLOCK, typename T, int V, int R>
__device__ __forceinline__ void share_moments(const NormArgs& a, const Share& w, const Piece<T, V> (&x)[R],
                                              Lds<BLOCK, V>& L, int cg, int per) {
  const int cols = w.nv * per, gcols = per == 1 ? cg / V : cg;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (w.ty + r * w.TY < w.ns)
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += to_f32(x[r].e[j]);
  put_sums<V>(L.buf, w, per, v);
  group_sums<BLOCK>(L.buf, L.g1, w.TY, cols, gcols);
  const float inv = 1.0f / ((float)w.ns * (float)cg);
  float m[V];
#pragma unroll
  for (int j = 0; j < V; ++j) m[j] = w.active ? L.g1[(w.cv * V + j) / cg] * inv : 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (w.ty + r * w.TY < w.ns)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = to_f32(x[r].e[j]) - m[j];
        v[j] = fmaf(d, d, v[j]);
      }
  put_sums<V>(L.buf, w, per, v);
  group_sums<BLOCK>(L.buf, L.g2, w.TY, cols, gcols);
  const int ng = w.nv * V / cg;
  for (int g = threadIdx.x; g < ng; g += BLOCK) L.g1[g] *= inv;
  __syncthreads();
}

template <typename T, int V, int R, int ACT>
__device__ __forceinline__ void write_normed(const NormArgs& a, const Share& w, const Piece<T, V> (&x)[R],
                                             const float (&mul)[V], const float (&add)[V]) {
  T* base = (T*)a.y + (int64_t)w.img * a.pixels * a.C + w.c0 + w.cv * V;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s = w.ty + r * w.TY;
    if (w.active && s < w.ns) {
      Piece<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.e[j] = (T)act_fwd<ACT>(fmaf(to_f32(x[r].e[j]), mul[j], add[j]));
      *(Piece<T, V>*)(base + (int64_t)(w.s0 + s) * a.C) = o;
    }
  }
}

// z = x mul + add for the thread's channels, from its groups' mean and rstd in L.g1, L.g2.
template <int BLOCK, int V>
__device__ __forceinline__ void affine(const NormArgs& a, const Share& w, const Lds<BLOCK, V>& L, int cg,
                                       float (&mul)[V], float (&add)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mul[j] = add[j] = 0.0f;
    if (w.active) {
      const int c = w.cv * V + j, g = c / cg;
      mul[j] = L.g2[g] * (a.weight ? a.weight[w.c0 + c] : 1.0f);
      add[j] = (a.bias ? a.bias[w.c0 + c] : 0.0f) - L.g1[g] * mul[j];
    }
  }
}

// One launch: block (slab, image) normalises all pixels of `nch` channels.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_whole(NormArgs a, int nch, int slabs) {
  __shared__ Lds<BLOCK, V> L;
  const int img = blockIdx.x / slabs, c0 = (blockIdx.x - img * slabs) * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), 0, a.pixels);
  const int cg = a.C / a.groups, per = cg % V == 0 ? 1 : V;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  share_moments<BLOCK, T, V, R>(a, w, x, L, cg, per);
  const int ng = w.nv * V / cg;
  const float inv = 1.0f / ((float)w.ns * (float)cg);
  for (int g = threadIdx.x; g < ng; g += BLOCK) {
    const float rstd = 1.0f / sqrtf(L.g2[g] * inv + a.eps);
    L.g2[g] = rstd;
    float* st = a.stats + ((int64_t)img * a.groups + c0 / cg + g) * 2;
    st[0] = L.g1[g];
    st[1] = rstd;
  }
  __syncthreads();
  float mul[V], add[V];
  affine<BLOCK, V>(a, w, L, cg, mul, add);
  write_normed<T, V, R, ACT>(a, w, x, mul, add);
}

// Two launches, the first: block (chunk, image, slab) leaves (mean, squares) of its groups.
template <int BLOCK, typename T, int V, int R>
__global__ __launch_bounds__(BLOCK) void norm_moments(NormArgs a, int nch, int slabs, int chunk, int chunks) {
  __shared__ Lds<BLOCK, V> L;
  const int per_img = slabs * chunks, img = blockIdx.x / per_img, rest = blockIdx.x - img * per_img;
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups, per = cg % V == 0 ? 1 : V;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  share_moments<BLOCK, T, V, R>(a, w, x, L, cg, per);
  const int ng = w.nv * V / cg;
  float* part = a.part + (((int64_t)img * chunks + ch) * a.groups + c0 / cg) * 2;
  for (int g = threadIdx.x; g < ng; g += BLOCK) {
    part[2 * g] = L.g1[g];
    part[2 * g + 1] = L.g2[g];
  }
}

// The second: merges the image's chunks and normalises.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_apply(NormArgs a, int nch, int slabs, int chunk, int chunks) {
  __shared__ Lds<BLOCK, V> L;
  const int per_img = slabs * chunks, img = blockIdx.x / per_img, rest = blockIdx.x - img * per_img;
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  const int ng = w.nv * V / cg;
  // lanes of a group take every gt-th chunk and merge their (n, mean, squares) in a fixed tree
  int gt = 64;
  while (gt > 1 && gt * ng > BLOCK) gt >>= 1;
  for (int g0 = 0; g0 < ng; g0 += BLOCK / gt) {
    const int g = g0 + (int)threadIdx.x / gt, l = threadIdx.x & (gt - 1);
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    if (g < ng)
      for (int k = l; k < chunks; k += gt) {
        const float* p = a.part + (((int64_t)img * chunks + k) * a.groups + c0 / cg + g) * 2;
        const float nk = (float)min(chunk, a.pixels - k * chunk) * (float)cg;
        const float tot = n + nk, d = p[0] - mean;
        mean += d * (nk / tot);
        m2 += p[1] + d * d * (n * (nk / tot));
        n = tot;
      }
    for (int o = 1; o < gt; o <<= 1) {
      const float on = __shfl_xor(n, o), om = __shfl_xor(mean, o), o2 = __shfl_xor(m2, o);
      const float tot = n + on;
      const bool low = (l & o) == 0;          // both sides merge (lower, upper) in the same order
      const float na = low ? n : on, ma = low ? mean : om, sa = low ? m2 : o2;
      const float nb = low ? on : n, mb = low ? om : mean, sb = low ? o2 : m2;
      const float f = tot > 0.0f ? nb / tot : 0.0f, d = mb - ma;
      mean = nb > 0.0f ? ma + d * f : ma;
      m2 = sa + sb + (nb > 0.0f ? d * d * (na * f) : 0.0f);
      n = tot;
    }
    if (g < ng && l == 0) {
      const float rstd = 1.0f / sqrtf(m2 / n + a.eps);
      L.g1[g] = mean;
      L.g2[g] = rstd;
      if (ch == 0) {
        float* st = a.stats + ((int64_t)img * a.groups + c0 / cg + g) * 2;
        st[0] = mean;
        st[1] = rstd;
      }
    }
  }
  __syncthreads();
  float mul[V], add[V];
  affine<BLOCK, V>(a, w, L, cg, mul, add);
  write_normed<T, V, R, ACT>(a, w, x, mul, add);
}

// ---- backward

// dz and xh of element j of piece r, from the group's mean / rstd and the channel's weight / bias.
template <int V>
struct Channel {
  float mean[V], rstd[V], wt[V], bs[V];
};

template <int V>
__device__ __forceinline__ Channel<V> load_channel(const NormArgs& a, const Share& w, int cg) {
  Channel<V> p;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    p.mean[j] = p.rstd[j] = p.wt[j] = p.bs[j] = 0.0f;
    if (w.active) {
      const int c = w.c0 + w.cv * V + j;
      const float* st = a.stats + ((int64_t)w.img * a.groups + c / cg) * 2;
      p.mean[j] = st[0];
      p.rstd[j] = st[1];
      p.wt[j] = a.weight ? a.weight[c] : 1.0f;
      p.bs[j] = a.bias ? a.bias[c] : 0.0f;
    }
  }
  return p;
}

template <typename T, int V, int R, int ACT>
__device__ __forceinline__ void channel_sums(const Share& w, const Piece<T, V> (&x)[R], const Piece<T, V> (&gy)[R],
                                             const Channel<V>& p, float (&sb)[V], float (&sw)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) sb[j] = sw[j] = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (w.ty + r * w.TY < w.ns)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (to_f32(x[r].e[j]) - p.mean[j]) * p.rstd[j];
        const float dz = to_f32(gy[r].e[j]) * act_grad<ACT>(fmaf(xh, p.wt[j], p.bs[j]));
        sb[j] += dz;
        sw[j] = fmaf(dz, xh, sw[j]);
      }
}

// Column sums over ty of a [TY][cols] buffer into out[cols].
template <int BLOCK>
__device__ __forceinline__ void column_sums(const float* buf, float* out, int TY, int cols) {
  group_sums<BLOCK>(buf, out, TY, cols, 1);
}

template <typename T, int V, int R, int ACT>
__device__ __forceinline__ void write_gx(const NormArgs& a, const Share& w, const Piece<T, V> (&x)[R],
                                         const Piece<T, V> (&gy)[R], const Channel<V>& p, const float (&m1)[V],
                                         const float (&m2)[V]) {
  T* base = (T*)a.gx + (int64_t)w.img * a.pixels * a.C + w.c0 + w.cv * V;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s = w.ty + r * w.TY;
    if (w.active && s < w.ns) {
      Piece<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (to_f32(x[r].e[j]) - p.mean[j]) * p.rstd[j];
        const float u = to_f32(gy[r].e[j]) * act_grad<ACT>(fmaf(xh, p.wt[j], p.bs[j])) * p.wt[j];
        o.e[j] = (T)(p.rstd[j] * (u - m1[j] - xh * m2[j]));
      }
      *(Piece<T, V>*)(base + (int64_t)(w.s0 + s) * a.C) = o;
    }
  }
}

// Group means of u and u xh for the thread's channels, from per-channel sums of dz (L.g1) and dz xh (L.g2)
// over the image, which the threads of a group add up in channel order.
template <int BLOCK, int V>
__device__ __forceinline__ void group_means(const NormArgs& a, const Share& w, const Lds<BLOCK, V>& L, int cg,
                                            float (&m1)[V], float (&m2)[V]) {
  const float inv = 1.0f / ((float)a.pixels * (float)cg);
  int last = -1;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    m1[j] = m2[j] = 0.0f;
    if (w.active) {
      const int g = (w.cv * V + j) / cg;
      if (g != last) {
        s1 = s2 = 0.0f;
        for (int c = g * cg; c < (g + 1) * cg; ++c) {
          const float wt = a.weight ? a.weight[w.c0 + c] : 1.0f;
          s1 = fmaf(wt, L.g1[c], s1);
          s2 = fmaf(wt, L.g2[c], s2);
        }
        last = g;
      }
      m1[j] = s1 * inv;
      m2[j] = s2 * inv;
    }
  }
}

// One read: block (slab, image) has all pixels of its channels; leaves the image's channel sums too.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_bwd_whole(NormArgs a, int nch, int slabs) {
  __shared__ Lds<BLOCK, V> L;
  const int img = blockIdx.x / slabs, c0 = (blockIdx.x - img * slabs) * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), 0, a.pixels);
  const int cg = a.C / a.groups, cols = w.nv * V;
  Piece<T, V> x[R], gy[R];
  load_share<T, V, R>(a, w, x);
  load_rows<T, V, R>(a.gy, a, w, gy);
  const Channel<V> p = load_channel<V>(a, w, cg);
  float sb[V], sw[V];
  channel_sums<T, V, R, ACT>(w, x, gy, p, sb, sw);
  put_sums<V>(L.buf, w, V, sb);
  column_sums<BLOCK>(L.buf, L.g1, w.TY, cols);
  put_sums<V>(L.buf, w, V, sw);
  column_sums<BLOCK>(L.buf, L.g2, w.TY, cols);
  float* part = a.part + (int64_t)img * 2 * a.C + c0;
  for (int c = threadIdx.x; c < cols; c += BLOCK) {
    part[c] = L.g1[c];
    part[a.C + c] = L.g2[c];
  }
  float m1[V], m2[V];
  group_means<BLOCK, V>(a, w, L, cg, m1, m2);
  write_gx<T, V, R, ACT>(a, w, x, gy, p, m1, m2);
}

// Chunked, the first launch: each chunk's channel sums.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_bwd_sums(NormArgs a, int nch, int slabs, int chunk, int chunks) {
  __shared__ Lds<BLOCK, V> L;
  const int per_img = slabs * chunks, img = blockIdx.x / per_img, rest = blockIdx.x - img * per_img;
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups, cols = w.nv * V;
  Piece<T, V> x[R], gy[R];
  load_share<T, V, R>(a, w, x);
  load_rows<T, V, R>(a.gy, a, w, gy);
  const Channel<V> p = load_channel<V>(a, w, cg);
  float sb[V], sw[V];
  channel_sums<T, V, R, ACT>(w, x, gy, p, sb, sw);
  put_sums<V>(L.buf, w, V, sb);
  column_sums<BLOCK>(L.buf, L.g1, w.TY, cols);
  put_sums<V>(L.buf, w, V, sw);
  column_sums<BLOCK>(L.buf, L.g2, w.TY, cols);
  float* part = a.part + ((int64_t)img * chunks + ch) * 2 * a.C + c0;
  for (int c = threadIdx.x; c < cols; c += BLOCK) {
    part[c] = L.g1[c];
    part[a.C + c] = L.g2[c];
  }
}

// Sums of one column of the [rows][2 C] partial sums, by a wave.
__device__ __forceinline__ float wave_column(const float* part, int64_t rows, int stride, int col) {
  float s = 0.0f;
  for (int64_t r = threadIdx.x & 63; r < rows; r += 64) s += part[r * stride + col];
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

template <int BLOCK>
__device__ __forceinline__ void param_grads(const NormArgs& a, int64_t rows, int block) {
  const int col = block * (BLOCK / 64) + (int)(threadIdx.x >> 6);     // 0 .. 2 C - 1
  if (col >= 2 * a.C) return;
  float* out = col < a.C ? a.gbias : a.gweight;
  if (out == nullptr) return;
  const float s = wave_column(a.part, rows, 2 * a.C, col);
  if ((threadIdx.x & 63) == 0) out[col < a.C ? col : col - a.C] = s;
}

template <int BLOCK>
__global__ __launch_bounds__(BLOCK) void norm_param_grads(NormArgs a, int64_t rows) {
  param_grads<BLOCK>(a, rows, blockIdx.x);
}

// The second: gx from the image's sums; the blocks behind the last chunk add up the parameters' gradients.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_bwd_apply(NormArgs a, int nch, int slabs, int chunk, int chunks) {
  __shared__ Lds<BLOCK, V> L;
  const int per_img = slabs * chunks, img = blockIdx.x / per_img, rest = blockIdx.x - img * per_img;
  if (img >= a.images) {
    param_grads<BLOCK>(a, (int64_t)a.images * chunks, blockIdx.x - a.images * per_img);
    return;
  }
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups, cols = w.nv * V;
  Piece<T, V> x[R], gy[R];
  load_share<T, V, R>(a, w, x);
  load_rows<T, V, R>(a.gy, a, w, gy);
  const Channel<V> p = load_channel<V>(a, w, cg);
  for (int c = threadIdx.x; c < 2 * cols; c += BLOCK) {
    const int col = c < cols ? c : a.C + c - cols;
    float s = 0.0f;
    for (int k = 0; k < chunks; ++k) s += a.part[((int64_t)img * chunks + k) * 2 * a.C + c0 + col];
    (c < cols ? L.g1 : L.g2)[c < cols ? c : c - cols] = s;
  }
  __syncthreads();
  float m1[V], m2[V];
  group_means<BLOCK, V>(a, w, L, cg, m1, m2);
  write_gx<T, V, R, ACT>(a, w, x, gy, p, m1, m2);
}

// ---- launch plan

constexpr int kR = 16;          // pieces a thread holds (forward)
constexpr int kRB = 8;          // pieces of x and of gy a thread holds (backward)
constexpr int kSmall = 256, kBig = 1024;

struct Plan {
  bool whole;
  int nch, slabs;               // channels of a slab (whole groups, whole pieces)
  int chunk, chunks;            // pixels of a chunk
  bool big;
};

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// A slab is a multiple of `unit` channels, the least that holds whole groups and whole pieces.
Plan make_plan(const NormArgs& a, int R) {
  Plan p{};
  const int cg = a.C / a.groups;
  const int unit = cg / gcd(cg, a.vec) * a.vec;
  // whole images: slabs of at least 64 bytes a pixel that fit kBig threads' registers
  int want = 64 / a.elem_bytes;
  int nch = unit;
  while (nch < want && nch < a.C) nch += unit;
  if (nch > a.C) nch = a.C;
  const int64_t fit = (int64_t)R * (kBig / (nch / a.vec > kBig ? kBig : nch / a.vec));
  if (nch / a.vec <= kBig && a.pixels <= fit) {
    p.whole = true;
    p.nch = nch;
    p.slabs = (a.C + nch - 1) / nch;
    p.big = a.pixels > (int64_t)R * (kSmall / (nch / a.vec > kSmall ? kSmall + 1 : nch / a.vec));
    return p;
  }
  // chunks: all channels, or as many whole units as kSmall pieces hold
  nch = a.C;
  if (nch / a.vec > kSmall) {
    nch = kSmall * a.vec / unit * unit;
    p.big = nch == 0;
    if (nch == 0) nch = unit;
  }
  p.nch = nch;
  p.slabs = (a.C + nch - 1) / nch;
  const int block = p.big ? kBig : kSmall;
  p.chunk = R * (block / (nch / a.vec));
  p.chunks = (a.pixels + p.chunk - 1) / p.chunk;
  return p;
}

template <int BLOCK, typename T, int V, int ACT>
hipError_t forward(const NormArgs& a, const Plan& p, hipStream_t stream) {
  if (p.whole) {
    norm_whole<BLOCK, T, V, kR, ACT><<<dim3((unsigned)(a.images * p.slabs)), BLOCK, 0, stream>>>(a, p.nch, p.slabs);
  } else {
    const dim3 grid((unsigned)(a.images * p.slabs * p.chunks));
    norm_moments<BLOCK, T, V, kR><<<grid, BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks);
    norm_apply<BLOCK, T, V, kR, ACT><<<grid, BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks);
  }
  return hipGetLastError();
}

template <int BLOCK, typename T, int V, int ACT>
hipError_t backward(const NormArgs& a, const Plan& p, hipStream_t stream) {
  const unsigned extra = (unsigned)((2 * a.C + BLOCK / 64 - 1) / (BLOCK / 64));
  if (p.whole) {
    norm_bwd_whole<BLOCK, T, V, kRB, ACT><<<dim3((unsigned)(a.images * p.slabs)), BLOCK, 0, stream>>>(a, p.nch,
                                                                                                      p.slabs);
    if (a.gweight || a.gbias)
      norm_param_grads<BLOCK><<<dim3(extra), BLOCK, 0, stream>>>(a, a.images);
  } else {
    const unsigned n = (unsigned)(a.images * p.slabs * p.chunks);
    norm_bwd_sums<BLOCK, T, V, kRB, ACT><<<dim3(n), BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks);
    norm_bwd_apply<BLOCK, T, V, kRB, ACT>
        <<<dim3(n + (a.gweight || a.gbias ? extra : 0)), BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks);
  }
  return hipGetLastError();
}

template <typename T, int V, int ACT>
hipError_t run(const NormArgs& a, bool bwd, hipStream_t stream) {
  const Plan p = make_plan(a, bwd ? kRB : kR);
  if (bwd) return p.big ? backward<kBig, T, V, ACT>(a, p, stream) : backward<kSmall, T, V, ACT>(a, p, stream);
  return p.big ? forward<kBig, T, V, ACT>(a, p, stream) : forward<kSmall, T, V, ACT>(a, p, stream);
}

template <typename T, int V>
hipError_t by_act(const NormArgs& a, bool bwd, hipStream_t stream) {
  switch (a.act) {
    case FBEV_ACT_RELU: return run<T, V, FBEV_ACT_RELU>(a, bwd, stream);
    case FBEV_ACT_SILU: return run<T, V, FBEV_ACT_SILU>(a, bwd, stream);
    case FBEV_ACT_GELU: return run<T, V, FBEV_ACT_GELU>(a, bwd, stream);
  }
  return run<T, V, FBEV_ACT_NONE>(a, bwd, stream);
}

hipError_t by_type(const NormArgs& a, bool bwd, hipStream_t stream) {
  if (a.elem_bytes == 4) {
    if (a.vec == 4) return by_act<float, 4>(a, bwd, stream);
    if (a.vec == 2) return by_act<float, 2>(a, bwd, stream);
    return by_act<float, 1>(a, bwd, stream);
  }
  if (a.vec == 8) return by_act<__bf16, 8>(a, bwd, stream);
  if (a.vec == 4) return by_act<__bf16, 4>(a, bwd, stream);
  if (a.vec == 2) return by_act<__bf16, 2>(a, bwd, stream);
  return by_act<__bf16, 1>(a, bwd, stream);
}

}  // namespace

size_t group_norm_workspace_bytes(const NormArgs& a, bool backward) {
  const Plan p = make_plan(a, backward ? kRB : kR);
  if (backward) return (size_t)a.images * (p.whole ? 1 : p.chunks) * 2 * a.C * sizeof(float);
  return p.whole ? 0 : (size_t)a.images * p.chunks * 2 * a.groups * sizeof(float);
}

hipError_t launch_group_norm_forward(const NormArgs& a, hipStream_t stream) { return by_type(a, false, stream); }

hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream) {
  if ((int64_t)a.images * a.pixels > 0) return by_type(a, true, stream);
  norm_param_grads<kSmall><<<dim3((unsigned)((2 * a.C + 3) / 4)), kSmall, 0, stream>>>(a, 0);   // sums of nothing
  return hipGetLastError();
}

}  // namespace fbev
