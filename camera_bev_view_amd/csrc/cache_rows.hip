// Rows of keys and values into the token cache (quantised as they are written) and back out of it.
//
//   scale = max(max_c |x_c| / most, 2^-126),  code_c = nearest(x_c / scale)        (a token and key head each)
//
// Memory bounds both: every value and code once.  A workgroup takes the call's rows of one page for up to four key heads (128
// channels: 16 lanes a token, whole lines of the tensors and of the page), or a wave where a call has a token or two.  A
// row belongs to 4, 8 or 16 lanes, eight channels each, that find its scale by lane exchanges; a row is on
// its way while the one before is at work (all eight of a team at once, at fewer waves: 37 us against 35.5 for the case below).
// Values are kept with their tokens side by side, which is how the attention's matrix products take them; they turn in LDS, four
// channels by four tokens a lane (byte permutes), on their way to or from the page.
//
// bf16 into int8 and back, 8 heads of 32, four sequences of up to 10000 rows (32500 in all): 17.9 us (52 MB) and 17.5 us (60
// MB); a copy's rate would take 10 and 12.  Neighbouring workgroups go to different XCDs, so that a short sequence leaves none idle.
// Beyond the traffic the write issues 22 vector instructions a value, 9 us over the card, and all its workgroups are on the
// card at once, so that they read, compute and write in step.
#include <hip/hip_runtime.h>

#include "codes.h"
#include "decoder.h"
#include "encoder.h"
#include "pieces.h"
#include "wave_ops.h"

namespace fbev {
namespace {

// What a workgroup's page holds of the call: tokens first .. first + n of the page are rows row .. row + n.
struct Run {
  int b, head, heads;     // heads head .. head + heads
  int page;               // -1 where there is none
  int first, n, row;
};

// The head groups of a page's tokens are neighbours.
template <int GROUP>
__device__ __forceinline__ Run find_run(const CacheArgs& c, uint32_t block, int tiles) {
  const uint32_t groups = (uint32_t)(c.Hk + GROUP - 1) / GROUP;
  const uint32_t bt = block / groups, tile = bt % (uint32_t)tiles;
  Run r;
  r.b = (int)(bt / (uint32_t)tiles);
  r.head = (int)(block - bt * groups) * GROUP;
  r.heads = min(GROUP, c.Hk - r.head);
  r.page = -1;
  const int start = c.start[r.b];
  if (start < 0) {        // no rows: readers write zeros, a page's worth a tile
    r.first = 0;
    r.row = (int)tile * kPage;
    r.n = min(kPage, c.T - r.row);
    return r;
  }
  const int64_t slot = (int64_t)(start / kPage) + tile;
  const int64_t row0 = slot * kPage - start;            // of the page's first token; negative in the first page
  r.row = (int)max(row0, (int64_t)0);
  r.first = (int)(r.row - row0);
  r.n = (int)min((int64_t)(kPage - r.first), (int64_t)c.T - r.row);
  if (slot < c.W) {
    const int p = c.table[(int64_t)r.b * c.W + slot];
    if (p >= 0 && p < c.pages) r.page = p;
  }
  return r;
}

__device__ __forceinline__ int kept_rows(const CacheArgs& c, const Run& r) {
  return c.count ? max(0, min(r.n, max(c.count[r.b], 0) - r.row)) : r.n;
}

// Four words of four bytes turned: out[i] has byte i of w[0 .. 3].
__device__ __forceinline__ void turn4(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  const auto top = [&](uint32_t y) { x = x > y ? x : y; };
  top(dpp<kQuadSwap1>(x));
  top(dpp<kQuadSwap2>(x));
  if constexpr (L >= 8) top(dpp<kHalfMirror>(x));
  if constexpr (L >= 16) top(dpp<kRowMirror>(x));
  return x;
}

// Eight channels of a row (`left` of them exist).
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, T (&e)[8]) {
  if (left >= 8) {
    __builtin_memcpy(e, p, sizeof e);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : (T)0.0f;
  }
}

constexpr int lanes_for(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : 16; }
constexpr int group_for(int L) { return 16 / L; }       // heads of a workgroup
constexpr int quads_for(int threads) { return threads == 64 ? 2 : 16; }

// L lanes a row: rows of up to 8 L channels.
template <typename T, int KIND, int L, int THREADS>
__global__ __launch_bounds__(THREADS) void cache_write(CacheMoveArgs a, int tiles, int64_t blocks) {
  using Cd = Codes<KIND>;
  constexpr int kGroup = group_for(L), kWords = 2 * L, kStride = kWords + 1, kRows = THREADS / L;
  __shared__ uint32_t turned[kGroup][kPage * kStride];  // value codes: [token][word]
  const CacheArgs& c = a.c;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const Run r = find_run<kGroup>(c, (uint32_t)block, tiles);
  if (r.page < 0) return;
  const int n = kept_rows(c, r);
  if (n <= 0) return;
  const int lane = threadIdx.x % L, ch = lane * 8;
  const int64_t at = (int64_t)r.page * c.Hk + r.head;
  uint8_t* kc = (uint8_t*)c.k + at * kPage * c.Dp;
  // a team's head and tensor stay, its token goes on by kStep; every team of a wave stays for the lane exchanges
  constexpr int kStep = kRows / (2 * kGroup);
  const int team = threadIdx.x / L, h = team % kGroup, which = team / kGroup & 1;
  const int left = h < r.heads ? c.D - ch : 0;
  int t = team / (2 * kGroup);
  const int64_t stride = which ? a.xs[1][1] : a.xs[0][1];
  const T* x = (const T*)(which ? a.x[1] : a.x[0]) + r.b * (which ? a.xs[1][0] : a.xs[0][0]) + (r.row + t) * stride +
               (r.head + h) * (which ? a.xs[1][2] : a.xs[0][2]) + ch;
  float* scales = (which ? c.v_scale : c.k_scale) + (at + h) * kPage + r.first;
  kc += (h * kPage + r.first) * c.Dp + ch;
  T next[8];                                            // a row is on its way while the one before is at work
  load8(x, t < n ? left : 0, next);
  for (int t0 = 0; t0 < n; t0 += kStep, t += kStep) {
    T e[8];
    __builtin_memcpy(e, next, sizeof e);
    x += kStep * stride;
    if (t0 + kStep < n) load8(x, t + kStep < n ? left : 0, next);
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = to_f32(e[i]);
      top = max(top, abs_bits(v[i]));
    }
    top = row_max<L>(top);
    const float scale = Cd::scale_of(top);
    const bool odd = top >= 0x7f800000u;
    const float inverse = Cd::inverse_of(scale);
    uint32_t w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float y[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      w[q] = Cd::pack(y, scale, inverse);
      if (odd) w[q] = 0;
    }
    if (t >= n || h >= r.heads) continue;
    if (lane == 0) scales[t] = scale;
    if (which == 0) {
      if (ch < c.Dp) __builtin_memcpy(__builtin_assume_aligned(kc + t * c.Dp, 8), w, 8);
    } else {
      uint32_t* to = turned[h] + (r.first + t) * kStride + 2 * lane;
      to[0] = w[0];
      to[1] = w[1];
    }
  }
  __syncthreads();
  // four tokens by four channels a lane, 16 lanes to a page's 64 tokens (two to a token or two); the page's other tokens keep
  // what they have
  uint8_t* vc = (uint8_t*)c.v + at * kPage * c.Dp;
  constexpr int kQuads = quads_for(THREADS);
  const int last = r.first + n, words = c.Dp / 4;
  const int token = 4 * ((kQuads < 16 ? r.first / 4 : 0) + (int)threadIdx.x % kQuads);
  if (token + 4 <= r.first || token >= last) return;
  for (int i = threadIdx.x / kQuads; i < kWords * r.heads; i += THREADS / kQuads) {
    const int head = i / kWords, word = i % kWords;
    if (word >= words) continue;
    uint32_t w[4], o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = turned[head][(token + j) * kStride + word];        // what no row wrote is not stored
    turn4(w, o);
    uint8_t* p = vc + (head * c.Dp + 4 * word) * kPage + token;
    if (token >= r.first && token + 4 <= last) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *(uint32_t*)(p + j * kPage) = o[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (token + t >= r.first && token + t < last) p[j * kPage + t] = (uint8_t)(o[j] >> (8 * t));
    }
  }
}

template <typename T, int KIND, int L, int THREADS>
__global__ __launch_bounds__(THREADS) void cache_read(CacheMoveArgs a, int tiles, int64_t blocks) {
  using Cd = Codes<KIND>;
  constexpr int kGroup = group_for(L), kWords = 2 * L, kStride = kWords + 1, kRows = THREADS / L;
  __shared__ uint32_t turned[kGroup][kPage * kStride];
  const CacheArgs& c = a.c;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const Run r = find_run<kGroup>(c, (uint32_t)block, tiles);
  if (r.n <= 0) return;
  const int n = r.page < 0 ? 0 : kept_rows(c, r);       // rows that hold something; the others get zeros
  const int64_t at = (int64_t)(r.page < 0 ? 0 : r.page) * c.Hk + r.head;
  const uint8_t* kc = (const uint8_t*)c.k + at * kPage * c.Dp;
  const uint8_t* vc = (const uint8_t*)c.v + at * kPage * c.Dp;
  constexpr int kQuads = quads_for(THREADS);
  const int last = r.first + n, words = c.Dp / 4;
  const int quad = 4 * ((kQuads < 16 ? r.first / 4 : 0) + (int)threadIdx.x % kQuads);
  if (a.y[1] && n > 0 && quad + 4 > r.first && quad < last) {
    for (int i = threadIdx.x / kQuads; i < kWords * r.heads; i += THREADS / kQuads) {
      const int head = i / kWords, word = i % kWords;
      if (word >= words) continue;
      const uint8_t* p = vc + (head * c.Dp + 4 * word) * kPage + quad;
      uint32_t w[4], o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *(const uint32_t*)(p + j * kPage);
      turn4(w, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) turned[head][(quad + j) * kStride + word] = o[j];
    }
  }
  // a team's head stays, its token goes on by kStep
  constexpr int kStep = kRows / kGroup;
  const int lane = threadIdx.x % L, ch = lane * 8, left = c.D - ch, team = threadIdx.x / L, h = team % kGroup;
  const bool mine = left > 0 && h < r.heads;
  const int64_t stride = (int64_t)c.Hk * c.D, out = ((int64_t)r.b * c.T + r.row) * stride + (r.head + h) * c.D + ch;
  const auto store = [&](T* y, int t, const uint32_t (&w)[2], float scale) {
    T e[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float x[4];
      Cd::unpack(w[q], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[4 * q + i] = (T)(t < n ? x[i] * scale : 0.0f);
    }
    y += out + t * stride;
    if (left >= 8) {
      __builtin_memcpy(y, e, sizeof e);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) y[i] = e[i];
    }
  };
  // keys, while the values are on their way into LDS
  if (a.y[0] && mine) {
    const uint8_t* from = kc + (h * kPage + r.first) * c.Dp + ch;
    const float* scales = c.k_scale + (at + h) * kPage + r.first;
    for (int t = team / kGroup; t < r.n; t += kStep) {
      uint32_t w[2] = {0, 0};
      float scale = 0.0f;
      if (t < n) {
        __builtin_memcpy(w, __builtin_assume_aligned(from + t * c.Dp, 8), 8);
        scale = scales[t];
      }
      store((T*)a.y[0], t, w, scale);
    }
  }
  if (a.y[1] == nullptr) return;
  __syncthreads();
  if (!mine) return;
  const float* scales = c.v_scale + (at + h) * kPage + r.first;
  for (int t = team / kGroup; t < r.n; t += kStep) {
    uint32_t w[2] = {0, 0};
    float scale = 0.0f;
    if (t < n) {
      for (int j = 0; j < 2; ++j) w[j] = turned[h][(r.first + t) * kStride + 2 * lane + j];
      scale = scales[t];
    }
    store((T*)a.y[1], t, w, scale);
  }
}

// f<T, KIND, L, THREADS>() for the call's type, codes, width and length.
template <typename T, int KIND, typename F>
hipError_t with_shape(const CacheMoveArgs& a, F f) {
  // one or two tokens are a wave's work
  const bool few = a.c.T <= 2;
  switch (lanes_for(a.c.D)) {
    case 4: return few ? f.template run<T, KIND, 4, 64>() : f.template run<T, KIND, 4, 256>();
    case 8: return few ? f.template run<T, KIND, 8, 64>() : f.template run<T, KIND, 8, 256>();
    default: return few ? f.template run<T, KIND, 16, 64>() : f.template run<T, KIND, 16, 256>();
  }
}

template <typename F>
hipError_t with_kernel(const CacheMoveArgs& a, F f) {
  const bool f32 = a.elem_bytes == 4;
  if (a.c.codes == FBEV_CODES_E4M3)
    return f32 ? with_shape<float, FBEV_CODES_E4M3>(a, f) : with_shape<__bf16, FBEV_CODES_E4M3>(a, f);
  return f32 ? with_shape<float, FBEV_CODES_INT8>(a, f) : with_shape<__bf16, FBEV_CODES_INT8>(a, f);
}

struct Work {
  const CacheMoveArgs& a;
  bool write;
  hipStream_t stream;
  template <typename T, int KIND, int L, int THREADS>
  hipError_t run() const {
    const int tiles = (a.c.T + kPage - 2) / kPage + 1;  // pages that T tokens can touch
    const int64_t blocks = (int64_t)tiles * a.c.B * ((a.c.Hk + group_for(L) - 1) / group_for(L));
    if (write)
      cache_write<T, KIND, L, THREADS><<<grid_rows(blocks), THREADS, 0, stream>>>(a, tiles, blocks);
    else
      cache_read<T, KIND, L, THREADS><<<grid_rows(blocks), THREADS, 0, stream>>>(a, tiles, blocks);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_cache_write(const CacheMoveArgs& a, hipStream_t stream) { return with_kernel(a, Work{a, true, stream}); }
hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t stream) { return with_kernel(a, Work{a, false, stream}); }

}  // namespace fbev
