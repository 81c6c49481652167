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
//
// Measured: bf16, 4 x 16896 tokens of ten heads of 64 (173 MB moved): 37.7 us, 4.6 TB/s of the 5.0 that a large
// copy reaches; fp32, 3 x 10007 tokens of four heads of 40, interleaved (38 MB, in the caches): 12 us; 900 tokens of
// 16 heads of 32: 3.9 us, a launch.
#include "encoder.h"
#include "pieces.h"

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

constexpr int kAhead = 4;             // items a thread loads before the angles are ready

// One item: a piece of V channels (and its V partners, half-split) of a token's head.
template <typename T, int V, bool IL>
struct Item {
  using P = Piece<T, V>;
  T* y;
  const float2* turn;                 // the piece's angles, or NULL: it is copied
  P u, w;

  __device__ __forceinline__ void load(const RotaryArgs& a, const float2* table, int b, int t0, int e, int per_token,
                                       int pieces, int turned) {
    const int t = e / per_token, rest = e - t * per_token;
    int h = rest / pieces;
    const int c = rest - h * pieces;
    const int which = h >= a.heads[0];
    if (which) h -= a.heads[0];
    const T* x = (const T*)a.x[which] + b * a.xs[which][0] + (t0 + t) * a.xs[which][1] + h * a.xs[which][2];
    y = (T*)a.y[which] + b * a.ys[which][0] + (t0 + t) * a.ys[which][1] + h * a.ys[which][2];
    turn = nullptr;
    int at = 2 * a.P + (c - turned) * V;
    if (c < turned) {
      turn = table + t * a.P + (IL ? (V > 1 ? c * (V / 2) : c) : c * V);
      at = IL && V == 1 ? 2 * c : c * V;
    }
    u = *(const P*)(x + at);
    if (c < turned) {
      if constexpr (!IL) w = *(const P*)(x + at + a.P);
      if constexpr (IL && V == 1) w = *(const P*)(x + at + 1);     // rows without alignment: a pair at a time
    }
    y += at;
  }

  __device__ __forceinline__ void store(int half) const {
    P p = u, q = w;
    if (turn != nullptr) {
      if constexpr (IL && V > 1) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 sc = turn[j];
          const float x1 = to_f32(u.e[2 * j]), x2 = to_f32(u.e[2 * j + 1]);
          p.e[2 * j] = (T)fmaf(x1, sc.y, -x2 * sc.x);
          p.e[2 * j + 1] = (T)fmaf(x2, sc.y, x1 * sc.x);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 sc = turn[j];
          const float x1 = to_f32(u.e[j]), x2 = to_f32(w.e[j]);
          p.e[j] = (T)fmaf(x1, sc.y, -x2 * sc.x);
          q.e[j] = (T)fmaf(x2, sc.y, x1 * sc.x);
        }
        *(P*)(y + (IL ? 1 : half)) = q;
      }
    }
    *(P*)y = p;
  }
};

// A workgroup takes `tokens` tokens of one sample: its threads issue the loads of their first items, form the angles
// and then turn.  In place an item's loads all come before its stores, and no other item touches its channels.
template <typename T, int V, bool IL>
__global__ __launch_bounds__(kBlock) void rotary_kernel(RotaryArgs a, int tokens, int blocks_per_sample) {
  __shared__ float2 table[kTableMax];
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  const int b = block / blocks_per_sample;
  const int t0 = (block - b * blocks_per_sample) * tokens;
  if (b >= a.B) return;
  const int nt = min(tokens, a.T - t0);
  // pieces of a head's row: rotated ones first (a half-split piece is V channels and their V partners)
  const int turned = (IL && V > 1) ? 2 * a.P / V : a.P / V;
  const int pieces = turned + (a.D - 2 * a.P) / V;
  const int per_token = (a.heads[0] + a.heads[1]) * pieces, items = nt * per_token;
  Item<T, V, IL> it[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int e = threadIdx.x + i * kBlock;
    if (e < items) it[i].load(a, table, b, t0, e, per_token, pieces, turned);
  }
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
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if ((int)threadIdx.x + i * kBlock < items) it[i].store(a.P);
  for (int e = threadIdx.x + kAhead * kBlock; e < items; e += kBlock) {
    it[0].load(a, table, b, t0, e, per_token, pieces, turned);
    it[0].store(a.P);
  }
}

template <typename T, int V>
hipError_t launch(const RotaryArgs& a, hipStream_t stream) {
  // at most one angle a thread, and no more items than the threads load ahead; few tokens are spread over the CUs
  const int turned = (a.interleaved && V > 1) ? 2 * a.P / V : a.P / V;
  const int64_t per_token = (int64_t)(a.heads[0] + a.heads[1]) * (turned + (a.D - 2 * a.P) / V);
  int64_t tokens = kBlock / a.P < kMaxTokens ? kBlock / a.P : kMaxTokens;
  if (tokens > kAhead * kBlock / per_token) tokens = kAhead * kBlock / per_token;
  if (tokens > (int64_t)a.B * a.T / 512) tokens = (int64_t)a.B * a.T / 512;
  if (tokens < 1) tokens = 1;
  const int per = (int)((a.T + tokens - 1) / tokens);
  const dim3 grid = grid_rows((int64_t)a.B * per);
  if (a.interleaved)
    rotary_kernel<T, V, true><<<grid, kBlock, 0, stream>>>(a, (int)tokens, per);
  else
    rotary_kernel<T, V, false><<<grid, kBlock, 0, stream>>>(a, (int)tokens, per);
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
