// Wave-level pieces of the attention kernels (64-lane waves, 32 x 32 MFMA tiles).
//
// A wave keeps one side of the problem in registers ("own": 32 rows, one per lane pair l, l + 32) and
// walks the other ("moving": tiles of 32 rows in LDS).  The product moving x own^T leaves lane (n, h)
// (n = lane mod 32, h = lane / 32) with own row n and the 16 moving rows 8 (i / 4) + 4 h + (i mod 4) of
// the tile, i < 16: everything a softmax row needs is in two lanes.  Those 16 values are at once the B
// operand of the next product, moving^T x values: its contraction runs over the tile's rows, whose order
// is free as long as the A operand (the transposed tile) uses the same one, so probabilities never leave
// their registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "encoder.h"
#include "wave_ops.h"

namespace fbev {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

// The moving row of accumulator register i (0 .. 15) in half-wave h.
__device__ __forceinline__ int acc_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// The same value, of which the compiler keeps no derived ones: what rare paths compute from it (or the 16 bit tests of a
// mask) does not move out of the loops and hold registers there.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Keeps a sum's additions where they are written: sunk behind the next head's work they would hold its terms' registers.
__device__ __forceinline__ void pin(float& x) { asm volatile("" : "+v"(x)); }

// Bit i: the i-th of the next 32 stages (N moving rows each, from s0 on) has a row of a document in [lo, hi].  One round of
// loads by the whole workgroup instead of one in front of every stage.
template <int N, int THREADS, typename F>
__device__ __forceinline__ uint32_t stages_with(uint32_t* shared, int s0, int end, int lo, int hi, F doc_of) {
  __syncthreads();
  if (threadIdx.x == 0) *shared = 0;
  __syncthreads();
  uint32_t bits = 0;
#pragma unroll 4
  for (int j = 0; j < 32 * N / THREADS; ++j) {
    const int r = s0 + THREADS * j + (int)threadIdx.x;
    const int d = r < end ? doc_of(r) : INT32_MIN;
    if (__any(d >= lo && d <= hi)) bits |= 1u << ((THREADS * j + ((int)threadIdx.x & ~63)) / N);
  }
  if ((threadIdx.x & 63) == 0 && bits != 0) atomicOr(shared, bits);
  __syncthreads();
  return (uint32_t)uniform((int)*shared);
}

// Over the two lanes of an own row.
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  const uint32_t a = r[0], b = r[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float pair_sum(float x) { return swap32_add(x, x); }

// Eight waves over a tile's moving rows stage 256 of them at a time, two tensors: up to 128 KB.
template <typename T>
constexpr bool eight_waves(int dp) {
  return 2 * 256 * dp * sizeof(T) <= (128 << 10);
}

// Moving rows that four row tiles share: 128, where two workgroups' tiles fit a CU's LDS.
template <typename T>
constexpr int shared_rows(int dp) {
  return 2 * 128 * dp * sizeof(T) <= (64 << 10) ? 128 : 64;
}

// A staged tile of N rows: 16-byte pieces, P to a row, piece p of row r in slot r P + (p ^ turn(r)).  There is no padding,
// so global memory moves straight into LDS (a wave's instruction fills 64 neighbouring slots, each lane fetching the piece
// that belongs there); the turn spreads the rows over the banks, both for a row's pieces read by 32 lanes (all 16 bank
// groups within 16 rows) and for the transposed reads (four rows by 64 bytes).
template <typename T, int DP>
struct Tile {
  static constexpr int P = DP * (int)sizeof(T) / 16;      // pieces of a row
  static constexpr int E = 16 / (int)sizeof(T);           // elements of a piece
  static constexpr int kRowBytes = P * 16;

  static __device__ __forceinline__ int turn(int r) {
    if constexpr (P == 4) return (r >> 2) & 3;
    if constexpr (P == 8) return ((r & 2) << 1) | ((r >> 2) & 3);
    if constexpr (P == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    return ((r & 3) << 2) | ((r >> 1) & 2);               // P == 32: a wave's chunks lie eight rows apart
  }
  static __device__ __forceinline__ int slot(int r, int p) { return r * P + (p ^ turn(r)); }
  static __device__ __forceinline__ T* at(char* tile, int r, int c) {
    return (T*)(tile + slot(r, c / E) * 16) + c % E;
  }
  static __device__ __forceinline__ const T* at(const char* tile, int r, int c) {
    return (const T*)(tile + slot(r, c / E) * 16) + c % E;
  }
};

template <typename T, int DP>
struct Mma;

// bf16: contraction in steps of 16 channels (row products) and 16 rows (transposed products).
template <int DP>
struct Mma<__bf16, DP> {
  using T = __bf16;
  using Frag = bf16x8;
  using Tl = Tile<T, DP>;
  static constexpr int kFrags = DP / 16;                 // fragments of one row's DP channels
  static constexpr int kFragElems = 8;                   // fragment f of half-wave h: piece 2 f + h

  static __device__ __forceinline__ f32x16 dot(const Frag& a, const Frag& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }

  // The B operand: values of tile rows 16 c .. 16 c + 15 (accumulator registers 8 c .. 8 c + 7), each as the sum of two bf16:
  // the first is off by up to 2^-8 of it, the second by as much of the rest, so 16 bits go into the product.
  struct Values {
    bf16x8 hi, lo;
  };
  static __device__ __forceinline__ Values split(const f32x16& p, int c) {
    Values r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = p[8 * c + 2 * j], y = p[8 * c + 2 * j + 1];
      const bf16x2 hi = {(__bf16)x, (__bf16)y};
      const uint32_t both = opaque(__builtin_bit_cast(uint32_t, hi));     // (the compiler would convert both again)
      r.hi[2 * j] = hi[0], r.hi[2 * j + 1] = hi[1];
      r.lo[2 * j] = (__bf16)(x - __builtin_bit_cast(float, both << 16));
      r.lo[2 * j + 1] = (__bf16)(y - __builtin_bit_cast(float, both & 0xFFFF0000u));
    }
    return r;
  }

  // The A operand: channels 32 blk + n of the rows above, read transposed (four rows by 16 channels for
  // every 16 lanes; lane i of the 16 addresses row i / 4, channels 4 (i mod 4)).  The turn repeats every 16 rows, so
  // the lane's addresses differ by constants between the tile's halves.
  static __device__ __forceinline__ i16x4 transposed(const char* tile, int r0, int u, int blk, int lane) {
    const int x = 4 * (lane >> 5) + ((lane >> 2) & 3), ch = 32 * blk + (lane & 16) + 4 * (lane & 3);
    const uint32_t at = (x * Tl::P + ((ch / 8) ^ Tl::turn(8 * (u & 1) + x))) * 16 + (ch & 4) * 2;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4*)((uint32_t)(uintptr_t)tile + at + (r0 + 8 * u) * Tl::kRowBytes));
  }
  static __device__ __forceinline__ bf16x8 columns(const char* tile, int r0, int c, int blk, int lane) {
    union {
      i16x4 s[2];
      bf16x8 v;
    } u;
    u.s[0] = transposed(tile, r0, 2 * c, blk, lane);
    u.s[1] = transposed(tile, r0, 2 * c + 1, blk, lane);
    return u.v;
  }

  template <int NB>
  static __device__ __forceinline__ void accumulate(f32x16 (&acc)[NB], const f32x16& p, const char* tile, int r0,
                                                    int lane) {
    const Values v[2] = {split(p, 0), split(p, 1)};
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bf16x8 x = columns(tile, r0, c, blk, lane);
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, v[c].hi, acc[blk], 0, 0, 0);
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, v[c].lo, acc[blk], 0, 0, 0);
      }
  }
};

// fp32: contraction in steps of two; a fragment is four channels (the half-waves' share of eight).
template <int DP>
struct Mma<float, DP> {
  using T = float;
  using Frag = f32x4;
  using Tl = Tile<T, DP>;
  static constexpr int kFrags = DP / 8;
  static constexpr int kFragElems = 4;

  static __device__ __forceinline__ f32x16 dot(const Frag& a, const Frag& b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }

  template <int NB>
  static __device__ __forceinline__ void accumulate(f32x16 (&acc)[NB], const f32x16& p, const char* tile, int r0,
                                                    int lane) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[blk] = __builtin_amdgcn_mfma_f32_32x32x2f32(
            *Tl::at(tile + r0 * Tl::kRowBytes, acc_row(i, lane >> 5), 32 * blk + (lane & 31)), p[i], acc[blk], 0, 0, 0);
  }
};

// One row's fragments from global memory, zero beyond its D channels.
template <typename T, int DP>
__device__ __forceinline__ void load_row(const T* row, bool vec, int D, int h,
                                         typename Mma<T, DP>::Frag (&f)[Mma<T, DP>::kFrags]) {
  using M = Mma<T, DP>;
  constexpr int E = M::kFragElems;
  if (vec) {
#pragma unroll
    for (int i = 0; i < M::kFrags; ++i) {
      const int c = (2 * i + h) * E;
      f[i] = typename M::Frag{};
      if (c < D) f[i] = *(const typename M::Frag*)(row + c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < M::kFrags; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int c = (2 * i + h) * E + j;
        f[i][j] = c < D ? row[c] : (T)0.0f;
      }
  }
}

// One wave instruction: 16 bytes a lane from the buffer's byte off + add to 64 neighbouring slots at `lds` (uniform).
__device__ __forceinline__ void move_pieces(__amdgpu_buffer_rsrc_t rs, char* lds, int off, int add) {
#ifdef __HIP_DEVICE_COMPILE__      // the host pass does not know the 16-byte form
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(uint32_t)(uintptr_t)lds, 16, off,
                                           add, 0, 0);
#endif
}

// One wave instruction: 4 bytes a lane.
__device__ __forceinline__ void move_words(__amdgpu_buffer_rsrc_t rs, void* lds, int off) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(uint32_t)(uintptr_t)lds, 4, off,
                                           0, 0, 0);
#endif
}

// `count` of the up to `room` (a multiple of 64) floats at `base` (uniform), zeros behind them, by the whole workgroup.
template <int THREADS>
__device__ __forceinline__ void stage_floats(float* lds, const float* base, int count, int room) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), 0, count * 4, 0x00020000);
  for (int at = 64 * wave; at < room; at += THREADS) move_words(rs, lds + at, (at + lane) * 4);
}

// A thread's part in staging: row and byte offset of its piece within a tile's first pieces, one a thread (an offset out of every
// buffer's bounds for channels beyond D: such pieces become zeros).
constexpr uint32_t kFarOut = 0x7FFFFF00u;

struct Stager {
  uint32_t row, byte;
};

template <typename T, int DP>
__device__ __forceinline__ Stager make_stager(int D) {
  using Tl = Tile<T, DP>;
  const uint32_t tid = threadIdx.x, p = (tid % Tl::P) ^ (uint32_t)Tl::turn((int)(tid / Tl::P));
  Stager s;
  s.row = tid / Tl::P;
  s.byte = p * Tl::E < (uint32_t)D ? p * 16 : kFarOut;
  asm volatile("" : "+v"(s.row), "+v"(s.byte));      // kept, not formed again for every tile
  return s;
}

// Stages N rows of a tensor, `stride` elements apart from `base` (uniform), zero beyond `rows` and beyond D channels, by
// the whole workgroup.  The wide path (vec: 16-byte pieces, N rows within 2^30 bytes) only issues the moves:
// wait_staged() before the barrier.
template <typename T, int DP, int N, int THREADS>
__device__ __forceinline__ void stage_rows(char* tile, const T* base, int64_t stride, int rows, bool vec, int D,
                                           const Stager& st) {
  using Tl = Tile<T, DP>;
  constexpr int WAVES = THREADS / 64, CHUNKS = N * Tl::P / 64;      // wave instructions
  static_assert(CHUNKS % WAVES == 0 && THREADS / Tl::P % (Tl::P < 32 ? 16 : 8) == 0,
                "a wave's chunks repeat the turn of their rows");
  if (vec) {
    const int wave = uniform(threadIdx.x >> 6);
    const uint32_t bytes = (uint32_t)stride * (uint32_t)sizeof(T);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<T*>(base), 0, (int)((uint32_t)(rows - 1) * bytes + (uint32_t)D * (uint32_t)sizeof(T)), 0x00020000);
    const int off = (int)(st.row * bytes + st.byte);
#pragma unroll
    for (int k = 0; k < CHUNKS / WAVES; ++k)
      move_pieces(rs, tile + (WAVES * k + wave) * 1024, off, k * (THREADS / Tl::P) * (int)bytes);
  } else {
#pragma unroll 1
    for (int e = (int)opaque(threadIdx.x); e < N * DP; e += THREADS) {
      const int r = e / DP, c = e - r * DP;
      *Tl::at(tile, r, c) = r < rows && c < D ? base[r * stride + c] : (T)0.0f;
    }
  }
}

// The same for N rows r0 .. of a key head's group of G query heads: row r is token r / G, head r mod G.
template <typename T, int DP, int N, int THREADS>
__device__ __forceinline__ void stage_group(char* tile, const T* base, int64_t token, int64_t head, int r0, int G,
                                            int rows, bool vec, int D) {
  using Tl = Tile<T, DP>;
  if (vec) {
    // offsets from the tile's first token: at most N tokens, within 2^31 bytes
    const int lane = (int)opaque(threadIdx.x) & 63, wave = uniform(threadIdx.x >> 6), t0 = r0 / G;
    const T* first = base + t0 * token;
    const int tb = (int)token * (int)sizeof(T), hb = (int)head * (int)sizeof(T);
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(first), 0, 0x7FFFFF00, 0x00020000);
#pragma unroll
    for (int k = 0; k < N * Tl::P / THREADS; ++k) {
      const int s = THREADS * k + 64 * wave + lane, r = s / Tl::P, p = (s % Tl::P) ^ Tl::turn(r);
      const int t = (r0 + r) / G, g = r0 + r - t * G;
      const int off = r < rows && p * Tl::E < D ? (t - t0) * tb + g * hb + p * 16 : (int)kFarOut;
      move_pieces(rs, tile + (THREADS / 64 * k + wave) * 1024, off, 0);
    }
  } else {
#pragma unroll 1
    for (int e = (int)opaque(threadIdx.x); e < N * DP; e += THREADS) {
      const int r = e / DP, c = e - r * DP, t = (r0 + r) / G, g = r0 + r - t * G;
      *Tl::at(tile, r, c) = r < rows && c < D ? base[t * token + g * head + c] : (T)0.0f;
    }
  }
}

__device__ __forceinline__ void wait_staged() { __builtin_amdgcn_s_waitcnt(0x0F70); }      // vmcnt(0)

// The row fragments of tile row r0 + n.
template <typename T, int DP>
__device__ __forceinline__ typename Mma<T, DP>::Frag tile_frag(const char* tile, int r0, int f, int lane) {
  const int n = lane & 31;
  return *(const typename Mma<T, DP>::Frag*)(tile + r0 * Tile<T, DP>::kRowBytes +
                                             Tile<T, DP>::slot(n, 2 * f + (lane >> 5)) * 16);
}

// Products of tile rows r0 .. r0 + 31 with the own row, added to s.
template <typename T, int DP>
__device__ __forceinline__ f32x16 tile_dot(const char* tile, int r0,
                                           const typename Mma<T, DP>::Frag (&own)[Mma<T, DP>::kFrags], int lane,
                                           f32x16 s = f32x16{}) {
  using M = Mma<T, DP>;
#pragma unroll
  for (int f = 0; f < M::kFrags; ++f) s = M::dot(tile_frag<T, DP>(tile, r0, f, lane), own[f], s);
  return s;
}

// The same with the own row's fragments in LDS ([fragment][lane], 16 bytes each) instead of registers.
template <typename T, int DP>
__device__ __forceinline__ f32x16 tile_dot(const char* tile, int r0, const char* own, int lane, f32x16 s = f32x16{}) {
  using M = Mma<T, DP>;
#pragma unroll
  for (int f = 0; f < M::kFrags; ++f)
    s = M::dot(tile_frag<T, DP>(tile, r0, f, lane), *(const typename M::Frag*)(own + (f * 64 + lane) * 16), s);
  return s;
}

// Infinities and NaN in masked places.  A transposed product multiplies every tile row with every own row, and
// 0 x inf is NaN: a non-finite element must reach only the own rows that see its tile row.  Tiles with masks are
// searched for one (holds_odd), and only when there is one the workgroup notes which sums it belongs to (find_odd),
// takes it out of the tile (clean_rows), and puts it back at the end (add_odd).
template <typename T, int DP, int N, int THREADS>
__device__ __forceinline__ bool holds_odd(const char* tile) {
  uint32_t odd = 0;
#pragma unroll 1
  for (int e = (int)opaque(threadIdx.x); e < N * Tile<T, DP>::P; e += THREADS) {
    const i32x4 w = *(const i32x4*)(tile + e * 16);
    // the exponent's ones carry into the sign bit
#pragma unroll
    for (int j = 0; j < 4; ++j)
      odd |= sizeof(T) == 2 ? ((uint32_t)w[j] & 0x7F807F80u) + 0x00800080u : ((uint32_t)w[j] & 0x7F800000u) + 0x00800000u;
  }
  return (odd & (sizeof(T) == 2 ? 0x80008000u : 0x80000000u)) != 0;
}

template <typename T, int DP, int N, int THREADS>
__device__ __forceinline__ void clean_rows(char* tile) {
#pragma unroll 1
  for (int e = (int)opaque(threadIdx.x); e < N * DP; e += THREADS) {
    T* x = (T*)tile + e;
    if (!(fabsf((float)*x) < __builtin_huge_valf())) *x = (T)0.0f;
  }
}

// Bit i of vis: the own row sees tile row r0 + acc_row(i, h).  The result's bit r: it sees tile row r0 + r.
__device__ __forceinline__ uint32_t seen_rows(uint32_t vis, int h) {
  const uint32_t other = __shfl_xor(vis, 32);
  uint32_t seen = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    seen |= (((vis >> (4 * u)) & 15) << (8 * u + 4 * h)) | (((other >> (4 * u)) & 15) << (8 * u + 4 * (1 - h)));
  return seen;
}

// Bit i: a positive infinite element (or a NaN) belongs to the lane's sum i of channels 32 blk ..; bit 16 + i: a
// negative one (or a NaN).
template <typename T, int DP>
__device__ __forceinline__ uint32_t find_odd(const char* tile, int r0, int blk, uint32_t vis, int lane) {
  const int h = (int)opaque(lane) >> 5;
  const uint32_t seen = seen_rows(vis, h);
  uint32_t odd = 0;
#pragma unroll 1
  for (int r = 0; r < 32; ++r) {
    const bool sees = (seen >> r) & 1;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const float x = (float)*Tile<T, DP>::at(tile, r0 + r, 32 * blk + acc_row(i, h));
      if (sees && !(fabsf(x) < __builtin_huge_valf()))
        odd |= (x < 0.0f ? 0u : 1u << i) | (x > 0.0f ? 0u : 1u << (16 + i));
    }
  }
  return odd;
}

// Whether the own row sees a tile row that has a non-finite element.
template <typename T, int DP>
__device__ __forceinline__ bool sees_odd(const char* tile, int r0, uint32_t vis, int lane) {
  lane = (int)opaque(lane);
  const uint32_t seen = seen_rows(vis, lane >> 5);
  bool odd = false;       // of tile row n
#pragma unroll 1
  for (int c = 0; c < DP; ++c)
    odd |= !(fabsf((float)*Tile<T, DP>::at(tile, r0 + (lane & 31), c)) < __builtin_huge_valf());
  return ((uint32_t)__ballot(odd) & seen) != 0;
}

template <int NB>
__device__ __forceinline__ void add_odd(f32x16 (&acc)[NB], const uint32_t (&odd)[NB]) {
#pragma unroll
  for (int blk = 0; blk < NB; ++blk)
    if (__builtin_expect(__any(odd[blk] != 0), 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if ((odd[blk] >> i) & 1) acc[blk][i] += __builtin_huge_valf();
        if ((odd[blk] >> (16 + i)) & 1) acc[blk][i] += kNegInf;
      }
    }
}

template <int NB>
__device__ __forceinline__ void make_nan(f32x16 (&acc)[NB], bool odd) {
  if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[blk][i] = odd ? __builtin_nanf("") : acc[blk][i];
  }
}

// tanh(u).  Through e = exp(-2 |u|) as (1 - e) / (1 + e); near zero, where 1 - e cancels, the odd Taylor series when EXACT
// (|u| < 1/4: the first term left out is below 1e-8 of the value).
template <bool EXACT>
__device__ __forceinline__ float tanh_fast(float u) {
  const float e = __builtin_amdgcn_exp2f(fabsf(u) * (-2.0f * kLog2e));
  float t = copysignf((1.0f - e) * __builtin_amdgcn_rcpf(1.0f + e), u);
  if constexpr (EXACT) {
    const float u2 = u * u;
    float s = fmaf(u2, 0.021869488f, -0.053968254f);
    s = fmaf(u2, s, 0.13333333f);
    s = fmaf(u2, s, -0.33333333f);
    s = fmaf(u2 * u, s, u);
    t = fabsf(u) < 0.25f ? s : t;
  }
  return t;
}

// What an own query row needs to know about itself.
struct Row {
  int r, t, head;       // row, token, query head
  int lim;              // last visible key by order (-1: none)
  int doc;
};

__device__ __forceinline__ int row_limit(const AttnArgs& a, int b, int t) {
  if (!a.causal) return a.Tk - 1;
  const int pre = a.prefix ? max(a.prefix[b], 0) : 0;      // (pre - 1 of the lowest int would wrap)
  return min(a.Tk - 1, max(t + a.Tk - a.Tq, pre - 1));
}

__device__ __forceinline__ Row make_row(const AttnArgs& a, int b, int hk, int r) {
  Row w;
  w.r = r;
  w.t = r / a.G;
  w.head = hk * a.G + (r - w.t * a.G);
  w.lim = row_limit(a, b, w.t);
  w.doc = a.doc_q ? a.doc_q[(int64_t)b * a.Tq + w.t] : 0;
  if (w.doc < 0) w.lim = -1;
  return w;
}

// min / max over the wave.
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = min(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = max(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}

// The outer sum moving value x own factor + moving factor x own value as one fp32 matrix instruction (contraction of
// two: the half-waves hold the two terms).  With factors of 1 it is a sum of the two values, rounded once.
__device__ __forceinline__ f32x16 outer_sum(float moving, float own) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(moving, own, f32x16{}, 0, 0, 0);
}

// Distances between the lane's own point and the 16 moving points of its accumulator registers (pos[tile row][axis] in
// LDS).  own[axis] is 1 in the lower half-wave and minus the own coordinate in the upper one: the differences come from
// the matrix cores, which the vector-bound loops leave idle, and a moving coordinate is read once a lane instead of
// four times 16 bytes.
__device__ __forceinline__ void distances(const float* pos, int at, int dims, const float (&own)[3], int lane,
                                          f32x16& d) {
  const bool low = lane < 32;
  const float* p = pos + (at + (lane & 31)) * dims;
  d = outer_sum(low ? p[0] : 1.0f, own[0]);
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i] *= d[i];
  if (dims > 1) {
    const f32x16 e = outer_sum(low ? p[1] : 1.0f, own[1]);
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = fmaf(e[i], e[i], d[i]);
  }
  if (dims > 2) {
    const f32x16 e = outer_sum(low ? p[2] : 1.0f, own[2]);
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = fmaf(e[i], e[i], d[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) d[i] = __builtin_amdgcn_sqrtf(d[i]);
}

// The own operand of distances(): a point's coordinates, negated, in the upper half-wave.
__device__ __forceinline__ void own_point(const float* p, int dims, int h, float (&own)[3]) {
#pragma unroll
  for (int ax = 0; ax < 3; ++ax) own[ax] = h == 0 ? 1.0f : (ax < dims ? -p[ax] : 0.0f);
}

// Scores are kept in a unit that costs the loop no multiplication: the raw products (a negative scale turns
// the queries' sign) or the cap's tanh.  `unit` takes them to base-2 exponents, a slope is divided by `raw`.
// Without its series near zero tanh is off by up to 2^-24, whatever its own size, and a score by that much of the cap: up
// to this cap by 4e-6, under what bf16 probabilities keep (2^-16).  fp32 tensors always take the series.
constexpr float kCoarseCap = 64.0f;

struct Unit {
  float unit, raw, inv_cap;
  bool near;            // bf16: tanh takes its series near zero
};

__device__ __forceinline__ Unit make_unit(const AttnArgs& a) {
  Unit u;
  const float sc = fabsf(a.scale);
  u.raw = a.cap > 0.0f ? a.cap : (sc > 0.0f ? sc : 1.0f);
  u.unit = u.raw * kLog2e;
  u.inv_cap = a.cap > 0.0f ? sc / a.cap : 0.0f;
  u.near = a.cap > kCoarseCap;
  return u;
}

// Queries in that unit's sign: negated for a negative scale, zero for a zero one.
template <typename T, int DP>
__device__ __forceinline__ void sign_row(const AttnArgs& a, typename Mma<T, DP>::Frag (&f)[Mma<T, DP>::kFrags]) {
  if (a.scale > 0.0f) return;
#pragma unroll
  for (int i = 0; i < Mma<T, DP>::kFrags; ++i)
#pragma unroll
    for (int j = 0; j < Mma<T, DP>::kFragElems; ++j)
      f[i][j] = a.scale < 0.0f ? (T)(-(float)f[i][j]) : (T)0.0f;
}

template <typename T>
__device__ __forceinline__ void cap_scores(f32x16& s, const Unit& un) {
  if (sizeof(T) == 4 || un.near) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = tanh_fast<true>(s[i] * un.inv_cap);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = tanh_fast<false>(s[i] * un.inv_cap);
  }
}

}  // namespace fbev
