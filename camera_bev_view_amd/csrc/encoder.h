// Internal interface between the C-ABI host layer and the encoder operators'
// kernels: group norm with an activation, rotary positions, attention.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fbev {

// A launch has at most 2^32 - 1 threads in a dimension (the runtime cuts more to 32 bits without an error): beyond kGridRow workgroups (of up to 1024 threads) they lie in rows
// of so many, the last one padded, which the kernels number through.
constexpr int64_t kGridRow = (int64_t)1 << 21;
inline dim3 grid_rows(int64_t blocks) {
  if (blocks <= kGridRow) return dim3((unsigned)blocks);
  return dim3((unsigned)kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
}

inline int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Group norm over channels-last images x[i][s][c] (i < images, s < pixels, c < C), `groups` groups of
// C / groups neighbouring channels.  y, gy and gx are contiguous.
struct NormArgs {
  const void* x;
  const float* weight;     // [C] or NULL (ones)
  const float* bias;       // [C] or NULL (zeros)
  const void* gy;          // backward
  void* y;                 // forward
  float* stats;            // [images, groups, 2]: mean, 1 / sqrt(var + eps)
  void* gx;                // backward
  float* gweight;          // backward, [C] or NULL
  float* gbias;            // backward, [C] or NULL
  float* part;             // workspace
  int64_t x_image, x_pixel;   // element strides of x
  int images, pixels, C, groups;
  int elem_bytes;          // 4 (fp32) or 2 (bf16)
  int vec;                 // channels one lane moves at a time (set by the host layer from C, strides and addresses)
  int act;                 // fbev_activation
  float eps;
};
size_t group_norm_workspace_bytes(const NormArgs& a, bool backward);
hipError_t launch_group_norm_forward(const NormArgs& a, hipStream_t stream);
hipError_t launch_group_norm_backward(const NormArgs& a, hipStream_t stream);

// Rotary positions: two tensors (queries, keys) of the same tokens, rotated by the same angles.
struct RotaryArgs {
  const void* x[2];        // [B, T, H, D] by strides, channels contiguous
  void* y[2];
  const float* pos;        // [B, T, A]
  const float* freqs;      // [A, P]
  int64_t xs[2][3], ys[2][3];   // element strides of batch, token, head
  int heads[2];            // 0: that tensor is absent
  int B, T, D, A, P;
  int elem_bytes;
  int vec;                 // channels a lane moves at a time
  bool interleaved, inverse;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);

// Attention.  A key head's G = Hq / Hk query heads are rows of one problem: row r = t G + g.
struct AttnArgs {
  const void *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];   // element strides of batch, token, head
  int B, Tq, Tk, Hq, Hk, G, D;
  int R;                   // rows per (sample, key head): Tq G
  float scale, cap;        // cap <= 0: none
  int dims;                // position axes, 0: no distance bias
  const float *pos_q, *pos_k;    // [B, T, dims]
  const float* slope;      // [B, Tq, Hq]
  const int32_t *doc_q, *doc_k;  // [B, T] or NULL
  int causal;
  const int32_t* prefix;   // [B] or NULL
  void* out;               // [B, Tq, Hq, D] (backward: read)
  float2* stats;           // [B, Hq, Tq] (backward: read): a row's maximum m (base-2 units) and sum l of 2^(s - m)
  int elem_bytes;
  bool vec;                // q, k, v rows move as 16-byte pieces
  bool vec_out;            // rows of out (and of the gradients) move as pieces of four channels
  // forward over split keys
  int splits, split_keys;  // set by the launcher
  float* part;             // [splits][B Hk][R][D + 2] partial rows (unnormalised sum, maximum, sum of weights)
  // backward
  const void* gout;        // [B, Tq, Hq, D]
  void *gq, *gk, *gv;      // contiguous
  float* gslope;           // [B, Tq, Hq] or NULL
  float* delta;            // workspace: per (sample, key head) what the keys' launch needs of the rows
};
size_t attention_forward_workspace_bytes(const AttnArgs& a);
size_t attention_backward_workspace_bytes(const AttnArgs& a);
hipError_t launch_attention_forward(AttnArgs a, hipStream_t stream);
hipError_t launch_attention_backward(AttnArgs a, hipStream_t stream);

}  // namespace fbev
