// Rotary positions with several axes.
//
//   theta[b,t,i] = sum_a pos[b,t,a] freqs[a,i]            (i < P pairs of channels)
//   (x1, x2)    -> (x1 cos - x2 sin, x2 cos + x1 sin)     per pair; the inverse turns by -theta
//
// Pairs are channels (i, i + P), or (2i, 2i + 1) when interleaved; channels from 2P on pass unchanged.
// Angles are formed and reduced to a quarter turn in double precision (a position of 1e6 at one radian
// a unit loses nothing but the final rounding), sine and cosine of the rest are Taylor polynomials in
// fp32, and a pair is rotated in fp32 and rounded once to its type.
//
// What bounds it: memory (every element is read and written once), so the angles are computed once per
// (token, pair) into LDS and shared by all query and key heads of the token: with ten heads the ~45
// vector instructions of an angle cost a tenth of that per rotated pair.
#include "encoder.h"

namespace fbev {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxTokens = 16;        // tokens of a workgroup at most
constexpr int kTableMax = 2048;       // (token, pair) angles of a workgroup at most

// sin and cos of `turns` whole turns (any magnitude below 2^50).
__device__ __forceinline__ float2 sincos_turns(double turns) {
  const double quarters = turns * 4.0;
  const double k = rint(quarters);
  const float x = (float)((quarters - k) * 1.5707963267948966);   // |x| <= pi/4
  const int n = (int)(int64_t)(k - 4.0 * floor(k * 0.25));
  const float x2 = x * x;
  // Taylor: the first term left out is below 2e-9 of the value at pi/4
  float s = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(x2, s, 8.3333333e-3f);
  s = fmaf(x2, s, -1.6666667e-1f);
  s = fmaf(x2 * x, s, x);
  float c = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(x2, c, -1.3888889e-3f);
  c = fmaf(x2, c, 4.1666667e-2f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.0f);
  const float ss = (n & 1) ? c : s, cc = (n & 1) ? s : c;
  return make_float2((n & 2) ? -ss : ss, ((n + 1) & 2) ? -cc : cc);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
  T e[V];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }

// A workgroup takes `tokens` tokens of one sample; items are (token, head, piece of V channels' pairs).
template <typename T, int V, bool IL>
__global__ __launch_bounds__(kBlock) void rotary_kernel(RotaryArgs a, int tokens, int blocks_per_sample) {
  __shared__ float2 table[kTableMax];
  const int b = blockIdx.x / blocks_per_sample;
  const int t0 = (blockIdx.x - b * blocks_per_sample) * tokens;
  const int nt = min(tokens, a.T - t0);
  for (int e = threadIdx.x; e < nt * a.P; e += kBlock) {
    const int t = e / a.P, i = e - t * a.P;
    const float* p = a.pos + ((int64_t)b * a.T + t0 + t) * a.A;
    double th = 0.0;
    for (int ax = 0; ax < a.A; ++ax) th = fma((double)p[ax], (double)a.freqs[ax * a.P + i], th);
    float2 sc = sincos_turns(th * 0.15915494309189535);
    if (a.inverse) sc.x = -sc.x;
    table[e] = sc;
  }
  __syncthreads();
  const int heads = a.heads[0] + a.heads[1];
  // pieces of a head's row: rotated ones first (a half-split piece is V channels and their V partners)
  const int turned = (IL && V > 1) ? 2 * a.P / V : a.P / V;
  const int pieces = turned + (a.D - 2 * a.P) / V;
  const int per_token = heads * pieces;
  for (int e = threadIdx.x; e < nt * per_token; e += kBlock) {
    const int t = e / per_token, rest = e - t * per_token;
    int h = rest / pieces;
    const int c = rest - h * pieces;
    const int which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    const T* x = (const T*)a.x[which] + b * a.xs[which][0] + (t0 + t) * a.xs[which][1] + h * a.xs[which][2];
    T* y = (T*)a.y[which] + b * a.ys[which][0] + (t0 + t) * a.ys[which][1] + h * a.ys[which][2];
    using P = Piece<T, V>;
    if (c >= turned) {
      const int at = 2 * a.P + (c - turned) * V;
      *(P*)(y + at) = *(const P*)(x + at);
    } else if constexpr (IL && V == 1) {      // rows without alignment: a pair at a time
      const float2 sc = table[t * a.P + c];
      const float x1 = to_f32(x[2 * c]), x2 = to_f32(x[2 * c + 1]);
      y[2 * c] = (T)fmaf(x1, sc.y, -x2 * sc.x);
      y[2 * c + 1] = (T)fmaf(x2, sc.y, x1 * sc.x);
    } else if constexpr (IL) {
      P v = *(const P*)(x + c * V);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 sc = table[t * a.P + c * (V / 2) + j];
        const float x1 = to_f32(v.e[2 * j]), x2 = to_f32(v.e[2 * j + 1]);
        v.e[2 * j] = (T)fmaf(x1, sc.y, -x2 * sc.x);
        v.e[2 * j + 1] = (T)fmaf(x2, sc.y, x1 * sc.x);
      }
      *(P*)(y + c * V) = v;
    } else {
      P u = *(const P*)(x + c * V), w = *(const P*)(x + a.P + c * V);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 sc = table[t * a.P + c * V + j];
        const float x1 = to_f32(u.e[j]), x2 = to_f32(w.e[j]);
        u.e[j] = (T)fmaf(x1, sc.y, -x2 * sc.x);
        w.e[j] = (T)fmaf(x2, sc.y, x1 * sc.x);
      }
      *(P*)(y + c * V) = u;
      *(P*)(y + a.P + c * V) = w;
    }
  }
}

template <typename T, int V>
hipError_t launch(const RotaryArgs& a, hipStream_t stream) {
  const int tokens = max(1, min(kMaxTokens, kBlock / a.P));
  const int per = (a.T + tokens - 1) / tokens;
  const dim3 grid((unsigned)((int64_t)a.B * per));
  if (a.interleaved)
    rotary_kernel<T, V, true><<<grid, kBlock, 0, stream>>>(a, tokens, per);
  else
    rotary_kernel<T, V, false><<<grid, kBlock, 0, stream>>>(a, tokens, per);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream) {
  if (a.elem_bytes == 4) {
    if (a.vec == 4) return launch<float, 4>(a, stream);
    if (a.vec == 2) return launch<float, 2>(a, stream);
    return launch<float, 1>(a, stream);
  }
  if (a.vec == 8) return launch<__bf16, 8>(a, stream);
  if (a.vec == 4) return launch<__bf16, 4>(a, stream);
  if (a.vec == 2) return launch<__bf16, 2>(a, stream);
  return launch<__bf16, 1>(a, stream);
}

}  // namespace fbev
