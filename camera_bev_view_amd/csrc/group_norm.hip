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
//   - a slab of at most 32 KB (two pieces a thread of 1024) is normalised in one launch with one read: the
//     8 x 22 maps of six images, 64 channels, take 6 us, of which a launch is 4; for larger slabs too few
//     workgroups are at work and the other form is faster although it reads twice;
//   - otherwise one launch leaves each chunk's (mean, sum of squares around it) in the workspace, and the
//     next merges an image's chunks (pairwise formula, in their order) and normalises; its blocks take the
//     chunks in the same order, so the second read finds much of them in the same L2.  Many chunks are merged by a
//     launch between the two.
// The backward has the same two forms with the per-channel sums of dz and dz xh; the parameters'
// gradients are column sums over chunks and images in a fixed order.  All results are deterministic.
//
// Measured: bf16, 24 maps of 32 x 88 with 80 channels (10.8 MB): moments 9.4, apply 10.3, backward 13.4 and 16.7 us;
// six maps of 64 x 176 with 128 channels (17.3 MB): 9.4 and 18.1 us.  The second read comes out of the caches (the
// counters see each kernel fetch its input once); a launch costs about 4 us of each, the chunks' merge by every workgroup
// about 7 us of the 18 (20 us forward with it left out), the rest is one round of loads and stores by all workgroups at once.
#include "encoder.h"

#include "../../include/flashbev.h"
#include "pieces.h"

namespace fbev {
namespace {

// The workgroup's number in a grid_rows() launch.
__device__ __forceinline__ uint32_t row_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == FBEV_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == FBEV_ACT_SILU) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
  if constexpr (ACT == FBEV_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == FBEV_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == FBEV_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (ACT == FBEV_ACT_GELU)
    return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
  return 1.0f;
}

// i / n for 0 <= i < 2^20, n >= 1 from 1 / n in fp32: (i + 1/2) / n is at least 1 / (2 n) away from a whole number, far
// more than the product's rounding.
__device__ __forceinline__ int small_div(int i, float inv) { return (int)(((float)i + 0.5f) * inv); }

// A workgroup's share: channels [c0, c0 + nv V) (whole groups) of pixels [s0, s0 + ns).  Thread (ty, cv)
// holds channel piece cv of pixels s0 + ty, s0 + ty + TY, ...
struct Share {
  int img, c0, nv, s0, ns, TY, ty, cv;
  bool active;
};

// Per group or channel of the share, two results.
template <int BLOCK, int V>
struct Groups {
  float g1[BLOCK * V], g2[BLOCK * V];
};
template <int BLOCK, int V>
struct Lds : Groups<BLOCK, V> {
  float buf[BLOCK * V], buf2[BLOCK * V];
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
  w.ty = small_div(threadIdx.x, 1.0f / (float)w.nv);
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

// Mean and sum of squares around it of every group of the share, into L.g1 and L.g2.  A thread takes its own values'
// mean and squares first (of a channel, or of the piece when it lies inside one group); a group's lanes then join them:
//   mean = sum n_i m_i / n,  squares = sum (q_i + n_i (m_i - mean)^2).
template <int BLOCK, typename T, int V, int R>
__device__ __forceinline__ void share_moments(const Share& w, const Piece<T, V> (&x)[R], Lds<BLOCK, V>& L, int cg,
                                              int per) {
  const int base = w.ns / w.TY, rem = w.ns - base * w.TY;
  const int rows = w.active ? base + (w.ty < rem ? 1 : 0) : 0;          // this thread's
  if (w.active) {
    float m[V], q[V];
    const float inv = rows > 0 ? 1.0f / (float)rows : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = q[j] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < rows)
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] += to_f32(x[r].e[j]);
    if (per == 1) {
      float t = m[0];
#pragma unroll
      for (int j = 1; j < V; ++j) t += m[j];
      t *= inv / (float)V;
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] = t;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] *= inv;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < rows)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = to_f32(x[r].e[j]) - m[j];
          q[j] = fmaf(d, d, q[j]);
        }
    const int at = (w.ty * w.nv + w.cv) * per;
    if (per == 1) {
      float t = q[0];
#pragma unroll
      for (int j = 1; j < V; ++j) t += q[j];
      L.buf[at] = m[0];
      L.buf2[at] = t;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        L.buf[at + j] = m[j];
        L.buf2[at + j] = q[j];
      }
    }
  }
  __syncthreads();
  const int cols = w.nv * per, gcols = per == 1 ? cg / V : cg, ng = cols / gcols;
  const int ty_n = min(w.TY, w.ns);
  const float each = (float)base * (per == 1 ? (float)V : 1.0f);        // elements of an entry
  const float more = (float)(base + 1) * (per == 1 ? (float)V : 1.0f);
  int gt = 64;
  while (gt > 1 && gt * ng > BLOCK) gt >>= 1;
  const int dty = gt / gcols, dc = gt - dty * gcols;
  for (int g0 = 0; g0 < ng; g0 += BLOCK / gt) {
    const int g = g0 + (int)threadIdx.x / gt, l = threadIdx.x & (gt - 1);
    float s = 0.0f, q = 0.0f;
    // entries l, l + gt, ... of the group's gcols columns by ty_n rows; a row has base or base + 1 pixels
    const int ty0 = l / gcols, c0 = l - ty0 * gcols;
    if (g < ng)
      for (int ty = ty0, c = c0; ty < ty_n;) {
        s = fmaf(ty < rem ? more : each, L.buf[ty * cols + g * gcols + c], s);
        ty += dty;
        c += dc;
        if (c >= gcols) c -= gcols, ++ty;
      }
    for (int o = gt >> 1; o > 0; o >>= 1) s += __shfl_xor(s, o);
    const float mean = s / ((float)w.ns * (float)cg);
    if (g < ng)
      for (int ty = ty0, c = c0; ty < ty_n;) {
        const int at = ty * cols + g * gcols + c;
        const float d = L.buf[at] - mean;
        q += fmaf((ty < rem ? more : each) * d, d, L.buf2[at]);
        ty += dty;
        c += dc;
        if (c >= gcols) c -= gcols, ++ty;
      }
    for (int o = gt >> 1; o > 0; o >>= 1) q += __shfl_xor(q, o);
    if (g < ng && l == 0) {
      L.g1[g] = mean;
      L.g2[g] = q;
    }
  }
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

// The thread's channels' weight and bias, and z = x mul + add from its groups' mean and rstd in L.g1, L.g2.
template <int V>
struct Affine {
  float mul[V], add[V];

  __device__ __forceinline__ void load(const NormArgs& a, const Share& w) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = w.c0 + w.cv * V + j;
      mul[j] = w.active && a.weight ? a.weight[c] : 1.0f;
      add[j] = w.active && a.bias ? a.bias[c] : 0.0f;
    }
  }
  template <int BLOCK>
  __device__ __forceinline__ void finish(const Share& w, const Groups<BLOCK, V>& L, int cg) {
    const float inv = 1.0f / (float)cg;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int g = w.active ? small_div(w.cv * V + j, inv) : 0;
      mul[j] *= L.g2[g];
      add[j] -= L.g1[g] * mul[j];
    }
  }
};

// One launch: block (slab, image) normalises all pixels of `nch` channels.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_whole(NormArgs a, int nch, int slabs) {
  __shared__ Lds<BLOCK, V> L;
  const uint32_t block = row_block();
  const int img = block / slabs, c0 = (block - img * slabs) * nch;
  if (img >= a.images) return;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), 0, a.pixels);
  const int cg = a.C / a.groups, per = cg % V == 0 ? 1 : V;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  Affine<V> af;
  af.load(a, w);
  share_moments<BLOCK, T, V, R>(w, x, L, cg, per);
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
  af.template finish<BLOCK>(w, L, cg);
  write_normed<T, V, R, ACT>(a, w, x, af.mul, af.add);
}

// Two launches, the first: block (chunk, image, slab) leaves (mean, squares) of its groups.
template <int BLOCK, typename T, int V, int R>
__global__ __launch_bounds__(BLOCK) void norm_moments(NormArgs a, int nch, int slabs, int chunk, int chunks) {
  __shared__ Lds<BLOCK, V> L;
  const uint32_t block = row_block();
  const int per_img = slabs * chunks, img = block / per_img, rest = block - img * per_img;
  if (img >= a.images) return;
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups, per = cg % V == 0 ? 1 : V;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  share_moments<BLOCK, T, V, R>(w, x, L, cg, per);
  const int ng = w.nv * V / cg;
  float* part = a.part + (((int64_t)img * chunks + ch) * a.groups + c0 / cg) * 2;
  for (int g = threadIdx.x; g < ng; g += BLOCK) {
    part[2 * g] = L.g1[g];
    part[2 * g + 1] = L.g2[g];
  }
}

// An image's chunks joined once, for all workgroups that normalise it: a wave a group, its lanes as share_moments joins
// threads.  Writes the statistics.
__global__ __launch_bounds__(512) void norm_join(NormArgs a, int chunk, int chunks) {
  const int64_t at = (int64_t)row_block() * 8 + (threadIdx.x >> 6);
  if (at >= (int64_t)a.images * a.groups) return;
  const int img = (int)(at / a.groups), g = (int)(at - (int64_t)img * a.groups), lane = threadIdx.x & 63;
  const int cg = a.C / a.groups;
  const float2* p = (const float2*)a.part + (int64_t)img * chunks * a.groups + g;
  const float n = (float)a.pixels * (float)cg;
  const float full = (float)chunk * (float)cg, rest = (float)(a.pixels - (chunks - 1) * chunk) * (float)cg;
  auto size = [&](int k) { return k < chunks - 1 ? full : (k == chunks - 1 ? rest : 0.0f); };
  float mean = 0.0f, m2 = 0.0f;
  for (int k0 = lane; k0 < chunks; k0 += 64 * 8) {        // eight loads in flight at once
    float2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = p[(int64_t)min(k0 + 64 * i, chunks - 1) * a.groups];
#pragma unroll
    for (int i = 0; i < 8; ++i) mean = fmaf(size(k0 + 64 * i), c[i].x, mean);
  }
  for (int o = 32; o > 0; o >>= 1) mean += __shfl_xor(mean, o);
  mean /= n;
  for (int k0 = lane; k0 < chunks; k0 += 64 * 8) {
    float2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = p[(int64_t)min(k0 + 64 * i, chunks - 1) * a.groups];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = c[i].x - mean, q = fmaf(size(k0 + 64 * i) * d, d, c[i].y);
      if (k0 + 64 * i < chunks) m2 += q;
    }
  }
  for (int o = 32; o > 0; o >>= 1) m2 += __shfl_xor(m2, o);
  if (lane == 0) {
    a.stats[2 * at] = mean;
    a.stats[2 * at + 1] = 1.0f / sqrtf(m2 / n + a.eps);
  }
}

constexpr int kKeep = 12;

// The second: merges the image's chunks and normalises.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_apply(NormArgs a, int nch, int slabs, int chunk, int chunks, int share,
                                                   int shares, bool joined) {
  __shared__ Groups<BLOCK, V> L;
  const uint32_t block = row_block();
  const int per_img = slabs * shares, img = block / per_img, rest = block - img * per_img;
  if (img >= a.images) return;
  const int slab = rest / shares, ch = rest - slab * shares, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * share, min(share, a.pixels - ch * share));
  const int cg = a.C / a.groups;
  Piece<T, V> x[R];
  load_share<T, V, R>(a, w, x);
  Affine<V> af;
  af.load(a, w);
  const int ng = w.nv * V / cg;
  // the lanes of a group join its chunks as share_moments joins threads
  int gt = 64;
  while (gt > 1 && gt * ng > BLOCK) gt >>= 1;
  const float n = (float)a.pixels * (float)cg;
  if (joined) {
    for (int g = threadIdx.x; g < ng; g += BLOCK) {
      const float* st = a.stats + ((int64_t)img * a.groups + c0 / cg + g) * 2;
      L.g1[g] = st[0];
      L.g2[g] = st[1];
    }
  }
  for (int g0 = joined ? ng : 0; g0 < ng; g0 += BLOCK / gt) {
    const int g = g0 + (int)threadIdx.x / gt, l = threadIdx.x & (gt - 1);
    const float2* p = (const float2*)a.part + (int64_t)img * chunks * a.groups + c0 / cg + g;
    float mean = 0.0f, m2 = 0.0f;
    // the first kKeep of a lane's chunks stay in registers, all their loads in flight at once
    float2 c[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int k = l + i * gt;
      c[i] = g < ng && k < chunks ? p[(int64_t)k * a.groups] : make_float2(0.0f, 0.0f);
    }
    const float full = (float)chunk * (float)cg, rest = (float)(a.pixels - (chunks - 1) * chunk) * (float)cg;
    auto size = [&](int k) { return k < chunks - 1 ? full : (k == chunks - 1 ? rest : 0.0f); };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) mean = fmaf(size(l + i * gt), c[i].x, mean);
    if (g < ng)
      for (int k = l + kKeep * gt; k < chunks; k += gt) mean = fmaf(size(k), p[(int64_t)k * a.groups].x, mean);
    for (int o = gt >> 1; o > 0; o >>= 1) mean += __shfl_xor(mean, o);
    mean /= n;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const float d = c[i].x - mean;
      m2 += fmaf(size(l + i * gt) * d, d, c[i].y);
    }
    if (g < ng)
      for (int k = l + kKeep * gt; k < chunks; k += gt) {
        const float2 x = p[(int64_t)k * a.groups];
        const float d = x.x - mean;
        m2 += fmaf(size(k) * d, d, x.y);
      }
    for (int o = gt >> 1; o > 0; o >>= 1) m2 += __shfl_xor(m2, o);
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
  af.template finish<BLOCK>(w, L, cg);
  write_normed<T, V, R, ACT>(a, w, x, af.mul, af.add);
}

// Images without pixels: mean 0, variance 0.
__global__ __launch_bounds__(256) void norm_empty_stats(NormArgs a) {
  const int64_t at = (int64_t)row_block() * 256 + threadIdx.x;
  if (at >= (int64_t)a.images * a.groups) return;
  a.stats[2 * at] = 0.0f;
  a.stats[2 * at + 1] = 1.0f / sqrtf(a.eps);
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
  const float inv = 1.0f / (float)cg;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    p.mean[j] = p.rstd[j] = p.wt[j] = p.bs[j] = 0.0f;
    if (w.active) {
      const int c = w.c0 + w.cv * V + j;
      const float* st = a.stats + ((int64_t)w.img * a.groups + w.c0 / cg + small_div(w.cv * V + j, inv)) * 2;
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

// The workgroup's sums of two values a channel, into L.g1 and L.g2: gt lanes a channel, in a fixed order.
template <int BLOCK, int V>
__device__ __forceinline__ void channel_totals(const Share& w, const float (&a)[V], const float (&b)[V],
                                               Lds<BLOCK, V>& L) {
  const int cols = w.nv * V;
  if (w.active) {
    const int at = w.ty * cols + w.cv * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      L.buf[at + j] = a[j];
      L.buf2[at + j] = b[j];
    }
  }
  __syncthreads();
  int gt = 64;
  while (gt > 1 && gt * cols > BLOCK) gt >>= 1;
  for (int c0 = 0; c0 < cols; c0 += BLOCK / gt) {
    const int c = c0 + (int)threadIdx.x / gt, l = threadIdx.x & (gt - 1);
    float s = 0.0f, t = 0.0f;
    if (c < cols)
      for (int ty = l; ty < w.TY; ty += gt) {
        s += L.buf[ty * cols + c];
        t += L.buf2[ty * cols + c];
      }
    for (int o = gt >> 1; o > 0; o >>= 1) {
      s += __shfl_xor(s, o);
      t += __shfl_xor(t, o);
    }
    if (c < cols && l == 0) {
      L.g1[c] = s;
      L.g2[c] = t;
    }
  }
  __syncthreads();
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
__device__ __forceinline__ void group_means(const NormArgs& a, const Share& w, const Groups<BLOCK, V>& L, int cg,
                                            float (&m1)[V], float (&m2)[V]) {
  const float inv = 1.0f / ((float)a.pixels * (float)cg), inv_cg = 1.0f / (float)cg;
  int last = -1;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    m1[j] = m2[j] = 0.0f;
    if (w.active) {
      const int g = small_div(w.cv * V + j, inv_cg);
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
  const uint32_t block = row_block();
  const int img = block / slabs, c0 = (block - img * slabs) * nch;
  if (img >= a.images) return;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), 0, a.pixels);
  const int cg = a.C / a.groups, cols = w.nv * V;
  Piece<T, V> x[R], gy[R];
  load_share<T, V, R>(a, w, x);
  load_rows<T, V, R>(a.gy, a, w, gy);
  const Channel<V> p = load_channel<V>(a, w, cg);
  float sb[V], sw[V];
  channel_sums<T, V, R, ACT>(w, x, gy, p, sb, sw);
  channel_totals<BLOCK, V>(w, sb, sw, L);
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
  const uint32_t block = row_block();
  const int per_img = slabs * chunks, img = block / per_img, rest = block - img * per_img;
  if (img >= a.images) return;
  const int slab = rest / chunks, ch = rest - slab * chunks, c0 = slab * nch;
  const Share w = make_share<BLOCK, V>(img, c0, min(nch, a.C - c0), ch * chunk, min(chunk, a.pixels - ch * chunk));
  const int cg = a.C / a.groups, cols = w.nv * V;
  Piece<T, V> x[R], gy[R];
  load_share<T, V, R>(a, w, x);
  load_rows<T, V, R>(a.gy, a, w, gy);
  const Channel<V> p = load_channel<V>(a, w, cg);
  float sb[V], sw[V];
  channel_sums<T, V, R, ACT>(w, x, gy, p, sb, sw);
  channel_totals<BLOCK, V>(w, sb, sw, L);
  float* part = a.part + ((int64_t)img * chunks + ch) * 2 * a.C + c0;
  for (int c = threadIdx.x; c < cols; c += BLOCK) {
    part[c] = L.g1[c];
    part[a.C + c] = L.g2[c];
  }
}

// Sums of one column of the [rows][2 C] partial sums, by a wave.
__device__ __forceinline__ float wave_column(const float* part, int64_t rows, int stride, int col) {
  float s = 0.0f;
  for (int64_t r0 = threadIdx.x & 63; r0 < rows; r0 += 64 * 8) {      // eight loads in flight at once
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[(r0 + 64 * i < rows ? r0 + 64 * i : rows - 1) * stride + col];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += r0 + 64 * i < rows ? v[i] : 0.0f;
  }
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

template <int BLOCK>
__device__ __forceinline__ void param_grads(const NormArgs& a, const float* sums, int64_t rows, int block) {
  const int col = block * (BLOCK / 64) + (int)(threadIdx.x >> 6);     // 0 .. 2 C - 1
  if (col >= 2 * a.C) return;
  float* out = col < a.C ? a.gbias : a.gweight;
  if (out == nullptr) return;
  const float s = wave_column(sums, rows, 2 * a.C, col);
  if ((threadIdx.x & 63) == 0) out[col < a.C ? col : col - a.C] = s;
}

template <int BLOCK>
__global__ __launch_bounds__(BLOCK) void norm_param_grads(NormArgs a, int64_t rows) {
  param_grads<BLOCK>(a, a.part, rows, blockIdx.x);
}

// An image's chunks joined once, for all workgroups of the next launch: 32 columns by 32 chunks a workgroup.
__global__ __launch_bounds__(1024) void norm_bwd_join(NormArgs a, int chunks, float* sums) {
  __shared__ float part[32][33];
  const uint32_t block = row_block();
  const int per_img = (2 * a.C + 31) / 32, img = block / per_img;
  if (img >= a.images) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = (block - img * per_img) * 32 + x;
  const float* p = a.part + (int64_t)img * chunks * 2 * a.C + min(col, 2 * a.C - 1);
  float s = 0.0f;
  for (int k0 = y; k0 < chunks; k0 += 32 * 8) {           // eight loads in flight at once
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(int64_t)min(k0 + 32 * i, chunks - 1) * 2 * a.C];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += k0 + 32 * i < chunks ? v[i] : 0.0f;
  }
  part[y][x] = s;
  __syncthreads();
  if (y > 0 || col >= 2 * a.C) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += part[i][x];
  sums[(int64_t)img * 2 * a.C + col] = s;
}

// The second: gx from the image's sums; the blocks behind the last chunk add up the parameters' gradients.
template <int BLOCK, typename T, int V, int R, int ACT>
__global__ __launch_bounds__(BLOCK) void norm_bwd_apply(NormArgs a, int nch, int slabs, int chunk, int chunks,
                                                       const float* sums, int rows) {
  __shared__ Groups<BLOCK, V> L;
  const uint32_t block = row_block();
  const int per_img = slabs * chunks, img = block / per_img, rest = block - img * per_img;
  if (img >= a.images) {
    param_grads<BLOCK>(a, sums, (int64_t)a.images * rows, (int)(block - (uint32_t)a.images * per_img));
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
    const float* q = sums + (int64_t)img * rows * 2 * a.C + c0 + col;
    float s = 0.0f;
    for (int k0 = 0; k0 < rows; k0 += 16) {               // sixteen loads in flight at once
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = q[(int64_t)min(k0 + i, rows - 1) * 2 * a.C];
#pragma unroll
      for (int i = 0; i < 16; ++i) s += k0 + i < rows ? v[i] : 0.0f;
    }
    (c < cols ? L.g1 : L.g2)[c < cols ? c : c - cols] = s;
  }
  __syncthreads();
  float m1[V], m2[V];
  group_means<BLOCK, V>(a, w, L, cg, m1, m2);
  write_gx<T, V, R, ACT>(a, w, x, gy, p, m1, m2);
}

// ---- launch plan

constexpr int kSmall = 256, kBig = 1024;
constexpr int kWhole = 2;       // pieces a thread of a kBig workgroup holds of a whole slab (32 KB)
// Eight pieces were faster than 16 in the moments (which leave CUs idle) and than 2 or 4 in the second launch (more
// workgroups, each of which merges the chunks).  The backward holds two tensors, four or six
// pieces of each.
constexpr int kR = 8;           // pieces a thread holds of a chunk (forward)
constexpr int kRA = 8;          // pieces a thread normalises (forward, the second launch)
constexpr int kRB = 4, kRBMany = 6;       // pieces of x and of gy a thread holds of a chunk (backward)

// An image's chunks are joined by a launch of their own above so many of them: every workgroup of the next launch joins them
// by itself below, which is a launch less but grows with the square (bf16, 200 x 200 cells, 128 channels, 313 chunks forward
// and 417 backward: 31.3 -> 21.9 us and 48.7 -> 30.3 us; four maps with 256 channels 232.6 -> 75.6 us and 630 -> 157 us;
// 400 x 400 cells, 128 channels, 220 -> 55 us and 329 -> 91 us; 88 chunks forward 27.7 and 28.0 us, 29 backward 29.9 and
// 31.2 us, 79 backward 16.5 and 17.0 us).
constexpr int kJoinMoments = 96, kJoinSums = 64;

struct Plan {
  bool whole;
  int nch, slabs;               // channels of a slab (whole groups, whole pieces)
  int chunk, chunks;            // pixels of a chunk
  bool big;
};

// A slab is a multiple of `unit` channels, the least that holds whole groups and whole pieces.
Plan make_plan(const NormArgs& a, int R) {
  Plan p{};
  const int cg = a.C / a.groups;
  const int unit = cg / gcd(cg, a.vec) * a.vec;
  // whole images: slabs of at least 64 bytes a pixel, up to kWhole pieces for each of kBig threads
  const int want = 64 / a.elem_bytes;
  int nch = unit;
  while (nch < want && nch < a.C) nch += unit;
  if (nch > a.C) nch = a.C;
  if (nch / a.vec <= kBig && a.pixels <= (int64_t)kWhole * (kBig / (nch / a.vec))) {
    p.whole = true;
    p.nch = nch;
    p.slabs = (a.C + nch - 1) / nch;
    return p;
  }
  // chunks: all channels, or as many whole units as kSmall pieces hold (as kBig pieces, for a wide unit)
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

// The backward's plan, and the pieces it was made for: six of each tensor where there are workgroups enough with four (bf16,
// six maps of 64 x 176, 128 channels: 53 -> 41 us; four of 200 x 200, 256 channels: 177 -> 158 us), four where there are
// not (six of 32 x 88, 80 channels: 18.9 us against 21.2 us; 174 workgroups).
Plan backward_plan(const NormArgs& a, int* pieces) {
  const Plan p = make_plan(a, kRB);
  *pieces = !p.whole && (int64_t)a.images * p.slabs * p.chunks >= 512 ? kRBMany : kRB;
  return *pieces == kRB ? p : make_plan(a, kRBMany);
}

template <int BLOCK, typename T, int V, int ACT>
void forward(const NormArgs& a, const Plan& p, hipStream_t stream) {
  const int share = kRA * (BLOCK / (p.nch / V)), shares = (a.pixels + share - 1) / share;
  norm_moments<BLOCK, T, V, kR><<<grid_rows((int64_t)a.images * p.slabs * p.chunks), BLOCK, 0, stream>>>(
      a, p.nch, p.slabs, p.chunk, p.chunks);
  const bool joined = p.chunks > kJoinMoments;
  if (joined)
    norm_join<<<grid_rows(((int64_t)a.images * a.groups + 7) / 8), 512, 0, stream>>>(a, p.chunk, p.chunks);
  norm_apply<BLOCK, T, V, kRA, ACT><<<grid_rows((int64_t)a.images * p.slabs * shares), BLOCK, 0, stream>>>(
      a, p.nch, p.slabs, p.chunk, p.chunks, share, shares, joined);
}

template <int BLOCK, typename T, int V, int ACT, int R>
void backward(const NormArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t extra = a.gweight || a.gbias ? (2 * a.C + BLOCK / 64 - 1) / (BLOCK / 64) : 0;
  const int64_t n = (int64_t)a.images * p.slabs * p.chunks;
  norm_bwd_sums<BLOCK, T, V, R, ACT><<<grid_rows(n), BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks);
  const float* sums = a.part;
  int rows = p.chunks;
  if (p.chunks > kJoinSums) {
    float* joined = a.part + (int64_t)a.images * p.chunks * 2 * a.C;
    norm_bwd_join<<<grid_rows((int64_t)a.images * ((2 * a.C + 31) / 32)), 1024, 0, stream>>>(a, p.chunks, joined);
    sums = joined;
    rows = 1;
  }
  norm_bwd_apply<BLOCK, T, V, R, ACT><<<grid_rows(n + extra), BLOCK, 0, stream>>>(a, p.nch, p.slabs, p.chunk, p.chunks,
                                                                               sums, rows);
}

template <typename T, int V, int ACT>
hipError_t run(const NormArgs& a, bool bwd, hipStream_t stream) {
  int pieces = kR;
  const Plan p = bwd ? backward_plan(a, &pieces) : make_plan(a, kR);
  const dim3 whole = grid_rows((int64_t)a.images * p.slabs);
  if (p.whole && !bwd) {
    norm_whole<kBig, T, V, kWhole, ACT><<<whole, kBig, 0, stream>>>(a, p.nch, p.slabs);
  } else if (p.whole) {
    norm_bwd_whole<kBig, T, V, kWhole, ACT><<<whole, kBig, 0, stream>>>(a, p.nch, p.slabs);
    if (a.gweight || a.gbias)
      norm_param_grads<kSmall><<<dim3((unsigned)((2 * a.C + 3) / 4)), kSmall, 0, stream>>>(a, a.images);
  } else if (bwd) {
    if (p.big)
      pieces == kRB ? backward<kBig, T, V, ACT, kRB>(a, p, stream) : backward<kBig, T, V, ACT, kRBMany>(a, p, stream);
    else
      pieces == kRB ? backward<kSmall, T, V, ACT, kRB>(a, p, stream)
                    : backward<kSmall, T, V, ACT, kRBMany>(a, p, stream);
  } else {
    p.big ? forward<kBig, T, V, ACT>(a, p, stream) : forward<kSmall, T, V, ACT>(a, p, stream);
  }
  return hipGetLastError();
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
  int pieces;
  const Plan p = backward ? backward_plan(a, &pieces) : make_plan(a, kR);
  if (backward)
    return (size_t)a.images * (p.whole ? 1 : p.chunks + (p.chunks > kJoinSums ? 1 : 0)) * 2 * a.C * sizeof(float);
  return p.whole ? 0 : (size_t)a.images * p.chunks * 2 * a.groups * sizeof(float);
}

hipError_t launch_group_norm_forward(const NormArgs& a, hipStream_t stream) {
  if (a.pixels > 0) return by_type(a, false, stream);
  norm_empty_stats<<<grid_rows(((int64_t)a.images * a.groups + kSmall - 1) / kSmall), kSmall, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream) {
  if ((int64_t)a.images * a.pixels > 0) return by_type(a, true, stream);
  norm_param_grads<kSmall><<<dim3((unsigned)((2 * a.C + 3) / 4)), kSmall, 0, stream>>>(a, 0);   // sums of nothing
  return hipGetLastError();
}

}  // namespace fbev
