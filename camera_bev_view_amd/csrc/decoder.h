// Internal interface between the C-ABI host layer and the decoder operators' kernels: root-mean-square norm,
// the token cache in 8 bits, attention over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fbev {

constexpr int kPage = 64;                            // tokens of a cache page
inline int padded_dim(int D) { return (D + 15) & ~15; }

// Root-mean-square norm of rows x[o][i][c] (o < outer, i < inner, c < C).  y, gy, gh, gx, h (where written) and codes
// are contiguous.
struct RmsArgs {
  const void* x;           // backward: the normalised sums
  const void* residual;    // forward, or NULL
  const float* weight;     // [C] or NULL (ones)
  void* y;                 // forward: of the type, or codes
  void* h;                 // forward: x + residual, or NULL
  float* rstd;             // [rows]; forward: may be NULL
  float* scales;           // codes: [rows, blocks]
  const void *gy, *gh;     // backward, gh may be NULL
  void* gx;                // backward
  float* gweight;          // backward, [C] or NULL
  float* part;             // workspace
  int64_t xs[2], rs[2];    // element strides of outer and inner rows
  int64_t outer, inner, rows;
  int C;
  int elem_bytes;
  int codes;               // -1: none, else fbev_codes
  int block;               // channels to a scale; C: the whole row
  float eps;
  double part_of_row;      // 1 / C
};
size_t rms_norm_workspace_bytes(const RmsArgs& a);
hipError_t launch_rms_norm_forward(const RmsArgs& a, hipStream_t stream);
hipError_t launch_rms_norm_backward(const RmsArgs& a, hipStream_t stream);

// The token cache and the rows of a call on it.
struct CacheArgs {
  void *k, *v;             // codes [pages, Hk, 64, Dp] and [pages, Hk, Dp, 64]
  float *k_scale, *v_scale;      // [pages, Hk, 64]
  int pages, Hk, D, Dp;
  int codes;               // fbev_codes
  const int32_t* table;    // [B, W]
  const int32_t* start;    // [B]
  const int32_t* count;    // [B] or NULL
  int B, T, W;
};

struct CacheMoveArgs {
  CacheArgs c;
  const void* x[2];        // write: keys, values by strides
  void* y[2];              // read: contiguous [B, T, Hk, D]
  int64_t xs[2][3];
  int elem_bytes;
};
hipError_t launch_cache_write(const CacheMoveArgs& a, hipStream_t stream);
hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t stream);

// Attention over the cache.  A key head's G = Hq / Hk query heads are rows of one problem: row r = t G + g.
struct CacheAttnArgs {
  CacheArgs c;             // T: query tokens
  const void* q;
  int64_t qs[3];           // element strides of batch, token, head
  int Hq, G;
  int R;                   // rows per (sequence, key head): T G
  int mode;                // fbev_draft
  const uint64_t* ancestors;     // [B, T, words]
  int words;
  float scale, cap;        // cap <= 0: none
  void* out;               // [B, T, Hq, D]
  int elem_bytes;
  // set by the launcher
  int row_blocks, splits;
  float down;              // of the values' scales
  float* part;             // [splits][B Hk][R][D + 2]
};
size_t cache_attention_workspace_bytes(const CacheAttnArgs& a);
hipError_t launch_cache_attention(CacheAttnArgs a, hipStream_t stream);

}  // namespace fbev
