// Rows of keys and values into the token cache (quantised as they are written) and back out of it.
//
//   scale = max(max_c |x_c| / most, 2^-126),  code_c = nearest(x_c / scale)        (a token and key head each)
//
// Memory bounds both: every value and code once.  A workgroup takes the call's rows of one page for one key head (the
// tokens of a page lie together, so its codes leave as whole lines), or a wave where a call has a token or two.  A row
// belongs to 4, 8 or 16 lanes, eight channels each, that find its scale by lane exchanges.  Values are kept with their
// tokens side by side, which is how the attention's matrix products take them; they turn in LDS, four channels by four
// tokens a lane (byte permutes), on their way to or from the page.
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
  int b, head, page;      // page: -1 where there is none
  int first, n, row;
};

__device__ __forceinline__ Run find_run(const CacheArgs& c, int64_t block, int tiles) {
  const uint32_t tile = (uint32_t)(block % tiles), bh = (uint32_t)(block / tiles);
  Run r;
  r.b = (int)(bh / (uint32_t)c.Hk);
  r.head = (int)(bh - (uint32_t)r.b * (uint32_t)c.Hk);
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
  return c.count ? max(0, min(r.n, c.count[r.b] - r.row)) : r.n;
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

template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
  if (left >= 8) {
    T e[8];
    __builtin_memcpy(e, p, sizeof e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
  }
}

constexpr int lanes_for(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : 16; }

// L lanes a row: rows of up to 8 L channels.
template <typename T, int KIND, int L, int THREADS>
__global__ __launch_bounds__(THREADS) void cache_write(CacheMoveArgs a, int tiles, int64_t blocks) {
  using Cd = Codes<KIND>;
  constexpr int kWords = 2 * L, kStride = kWords + 1, kRows = THREADS / L;
  __shared__ uint32_t turned[kPage * kStride];          // value codes: [token][word]
  const CacheArgs& c = a.c;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const Run r = find_run(c, block, tiles);
  if (r.page < 0) return;
  const int n = kept_rows(c, r);
  if (n <= 0) return;
  const int lane = threadIdx.x % L, ch = lane * 8;
  const int64_t at = (int64_t)r.page * c.Hk + r.head;
  uint8_t* kc = (uint8_t*)c.k + at * kPage * c.Dp;
  // both tensors' rows in one list; every team of a wave stays for the lane exchanges
  for (int base = 0; base < 2 * n; base += kRows) {
    const int item = base + (int)threadIdx.x / L;
    const bool mine = item < 2 * n;
    const int which = item & 1, t = mine ? item >> 1 : 0;
    const int64_t* s = a.xs[which];
    const T* x = (const T*)a.x[which] + r.b * s[0] + (int64_t)(r.row + t) * s[1] + r.head * s[2];
    float v[8];
    load8(x + ch, mine ? c.D - ch : 0, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
    top = row_max<L>(top);
    const float scale = Cd::scale_of(top);
    const bool odd = top >= 0x7f800000u;
    const float inverse = odd ? 0.0f : 1.0f / scale;
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = odd ? 0.0f : v[4 * j + i];
      w[j] = Cd::pack(y, scale, inverse);
    }
    if (!mine) continue;
    const int token = r.first + t;
    if (lane == 0) (which ? c.v_scale : c.k_scale)[at * kPage + token] = scale;
    if (which == 0) {
      if (ch < c.Dp) __builtin_memcpy(__builtin_assume_aligned(kc + token * c.Dp + ch, 8), w, 8);
    } else {
      turned[token * kStride + 2 * lane] = w[0];
      turned[token * kStride + 2 * lane + 1] = w[1];
    }
  }
  __syncthreads();
  // four tokens by four channels a lane, 16 lanes to a page's 64 tokens; the page's other tokens keep what they have
  uint8_t* vc = (uint8_t*)c.v + at * kPage * c.Dp;
  const int last = r.first + n, q0 = r.first / 4, quads = (last + 3) / 4 - q0, words = c.Dp / 4;
  for (int i = threadIdx.x; i < quads * words; i += THREADS) {
    const int quad = q0 + i % quads, word = i / quads, token = 4 * quad;
    uint32_t w[4], o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = turned[(token + j) * kStride + word];      // what no row wrote is not stored
    turn4(w, o);
    uint8_t* p = vc + 4 * word * kPage + token;
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
  constexpr int kWords = 2 * L, kStride = kWords + 1, kRows = THREADS / L;
  __shared__ uint32_t turned[kPage * kStride];
  const CacheArgs& c = a.c;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= blocks) return;
  const Run r = find_run(c, block, tiles);
  if (r.n <= 0) return;
  const int n = r.page < 0 ? 0 : kept_rows(c, r);       // rows that hold something; the others get zeros
  const int64_t at = (int64_t)(r.page < 0 ? 0 : r.page) * c.Hk + r.head;
  const uint8_t* kc = (const uint8_t*)c.k + at * kPage * c.Dp;
  const uint8_t* vc = (const uint8_t*)c.v + at * kPage * c.Dp;
  const int last = r.first + n, q0 = r.first / 4, quads = n > 0 ? (last + 3) / 4 - q0 : 0, words = c.Dp / 4;
  if (a.y[1]) {
    for (int i = threadIdx.x; i < quads * words; i += THREADS) {
      const int quad = q0 + i % quads, word = i / quads, token = 4 * quad;
      const uint8_t* p = vc + 4 * word * kPage + token;
      uint32_t w[4], o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *(const uint32_t*)(p + j * kPage);
      turn4(w, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) turned[(token + j) * kStride + word] = o[j];
    }
  }
  __syncthreads();
  const int lane = threadIdx.x % L, ch = lane * 8;
  if (ch >= c.D) return;
  for (int item = threadIdx.x / L; item < 2 * r.n; item += kRows) {
    const int which = item & 1, t = item >> 1, token = r.first + t;
    if (a.y[which] == nullptr) continue;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (t < n) {
      uint32_t w[2];
      if (which == 0)
        __builtin_memcpy(w, __builtin_assume_aligned(kc + token * c.Dp + ch, 8), 8);
      else
        for (int j = 0; j < 2; ++j) w[j] = turned[token * kStride + 2 * lane + j];
      const float scale = (which ? c.v_scale : c.k_scale)[at * kPage + token];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x[4];
        Cd::unpack(w[j], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = x[i] * scale;
      }
    }
    T* y = (T*)a.y[which] + (((int64_t)r.b * c.T + r.row + t) * c.Hk + r.head) * c.D + ch;
    const int left = c.D - ch;
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = (T)v[i];
    if (left >= 8) {
      __builtin_memcpy(y, e, sizeof e);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) y[i] = e[i];
    }
  }
}

// f<T, KIND, L, THREADS>() for the call's type, codes, width and length.
template <typename T, int KIND, typename F>
hipError_t with_shape(const CacheMoveArgs& a, F f) {
  // one or two tokens are at most four rows, which a wave holds
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
    const int64_t blocks = (int64_t)tiles * a.c.B * a.c.Hk;
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
