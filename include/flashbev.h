/*
 * libflashbev -- exact dense Sampling-VT camera-to-BEV view transform, fused,
 * for AMD Instinct MI355X (gfx950).  Plain C ABI: no C++ types, no exceptions,
 * no framework types cross this boundary.
 *
 * The operation (FlashBEV reading notes, "Problem Setting", "Core Idea" and
 * "Method" items 1-4): for every batch sample b, BEV cell (x, y) and channel c,
 *
 *   out[b,c,x,y] = sum_z  mean_{n valid at (b,x,y,z)}  bilinear(F[b,n,:,:,c], u, v)
 *
 * where, for height bin z, the voxel centre p = (x_x, y_y, z_z) is projected
 * through camera n as [u, v, 1]^T ~ K_n (R_n p + t_n) (SparseDriveV2 notes,
 * "Deformable Aggregation", step 2) and camera n is valid when the depth
 * d = (K_n (R_n p + t_n))_3 > 0 and the point lands in the image.  A point
 * no camera sees contributes 0.  Nothing per (camera, height, channel) is
 * stored in device memory: projection, validity test, sampling, mean and
 * height sum happen in one kernel.
 *
 * Conventions (the pages leave these open; this library fixes them):
 *   - voxel centres of the half-open ranges: x_i = x_min + (i + 1/2)(x_max - x_min)/X,
 *     likewise y_j, z_k; out[b, c, i, j] has i along ego x, j along ego y;
 *   - (R, t) maps ego to camera coordinates, p_cam = R p + t;
 *   - integer (u, v) are pixel centres, u along W (columns), v along H (rows);
 *     "in the image" means 0 <= u <= W-1 and 0 <= v <= H-1 (closed), so every
 *     valid sample is a convex combination of existing pixels;
 *   - bilinear taps x0 = floor(u), x1 = min(x0 + 1, W - 1), likewise rows;
 *   - projection and the in-image test are evaluated in double precision;
 *     interpolation weights and accumulation are fp32.
 *
 * Memory: every pointer is caller-owned *device* memory unless stated.  The
 * library allocates no device memory and keeps no state beyond the calling
 * thread's last-error text.  All work is enqueued on `stream` (a hipStream_t;
 * NULL = the null stream) and calls return before it completes.
 *
 * Errors: arguments are validated on the host before anything is enqueued;
 * on a non-OK status nothing has been written.  FBEV_ERR_DEVICE reports a
 * launch error from the HIP runtime; fbev_last_error() gives the text.
 */
#ifndef FLASHBEV_H
#define FLASHBEV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FBEV_ABI_VERSION 10
#define FBEV_MAX_CAMERAS 64
#define FBEV_MAX_GRID 65536
#define FBEV_MAX_LEVELS 4
#define FBEV_MAX_KEYPOINTS 256
#define FBEV_MAX_HEAD_DIM 128
#define FBEV_MAX_ROTARY_PAIRS 2048

typedef enum {
  FBEV_OK = 0,
  FBEV_ERR_INVALID_ARGUMENT = 1, /* negative size, NULL pointer for a non-empty buffer, bad range, N > FBEV_MAX_CAMERAS,
                                    bad feature levels */
  FBEV_ERR_UNSUPPORTED = 2,      /* unknown dtype, odd C for bf16, misaligned features, per-sample features >= 2 GiB,
                                    cameras x levels > 64 */
  FBEV_ERR_DEVICE = 3            /* the HIP runtime reported an error when enqueueing */
} fbev_status;

typedef enum { FBEV_DTYPE_F32 = 0, FBEV_DTYPE_BF16 = 1 } fbev_dtype;

/* Feature maps are channels-last [B, N, H, W, C], contiguous. */
typedef struct {
  int32_t B, N, C, H, W;
} fbev_feat_desc;

/* BEV extent in metres, ego frame; each axis is the half-open [min, max). */
typedef struct {
  float x_min, x_max, y_min, y_max, z_min, z_max;
} fbev_range;

/*
 * Forward of the fused Sampling-VT (FlashBEV notes, "Method" items 1-2).
 *
 *   features : [B,N,H,W,C] of `dtype` (fp32, or bf16 bit patterns), device, read only.
 *              Must be 4-byte aligned; 16-byte alignment with C*elem_size a
 *              multiple of 16 takes the wide-load path.
 *   K        : [B,N,3,3] fp32 intrinsics (feature-map pixels), device.
 *   R, t     : [B,N,3,3] and [B,N,3] fp32 ego->camera extrinsics, device.
 *   bev_range, X, Y, Z : the voxel grid (X, Y, Z >= 0, each <= FBEV_MAX_GRID).
 *   out      : [B,C,X,Y] fp32, device; fully overwritten (zero where no camera
 *              sees any height bin, all zeros when Z == 0).
 *   counts   : [B,X,Y,Z] uint8 valid-camera counts, device, or NULL to skip.
 *
 * Sizes of zero are allowed and give the empty / all-zero result.  The result
 * is deterministic (fixed reduction order).
 */
fbev_status fbev_forward(const void* features, fbev_dtype dtype, fbev_feat_desc fd, const float* K,
                         const float* R, const float* t, fbev_range bev_range, int32_t X, int32_t Y,
                         int32_t Z, float* out, uint8_t* counts, void* stream);

/*
 * Gradient of fbev_forward with respect to the features (FlashBEV notes,
 * "Method" item 4: the fused operator keeps the forward/backward semantics
 * of the tensorized one).  The forward is linear in the features with the
 * validity mask, bilinear weights and camera counts fixed, so
 *
 *   dF[b,n,y,x,c] = sum over (cell, z) valid for n, and taps of that sample
 *                   landing on (y, x), of grad_out[b,c,cell] * w_tap / count.
 *
 *   grad_out      : [B,C,X,Y] fp32, device, read only.
 *   grad_features : [B,N,H,W,C] fp32, device; fully overwritten (zeroed on
 *                   `stream`, then accumulated with fp32 atomics, so the
 *                   bit pattern may vary from run to run within fp32
 *                   rounding).  Returned in fp32 also for bf16 forwards.
 * Other arguments as for fbev_forward; no feature values are needed.
 */
fbev_status fbev_backward(const float* grad_out, fbev_feat_desc fd, const float* K, const float* R,
                          const float* t, fbev_range bev_range, int32_t X, int32_t Y, int32_t Z,
                          float* grad_features, void* stream);

/*
 * Gradients of fbev_forward's output with respect to the cameras.  The
 * SparseDriveV2 notes ("Deformable Aggregation", pitfalls) ask for a
 * projection-and-sampling chain that gradients flow through; for
 * L = <grad_out, out> this returns dL/dK, dL/dR and dL/dt with the validity
 * mask and the camera counts held fixed (they are piecewise constant in the
 * cameras).  Per in-view sample of camera n at voxel centre p, with
 * h = K (R p + t), u = h_1 / h_3 and v = h_2 / h_3:
 *
 *   dL/du = <grad_out[b,:,cell], d sample / du> / count   (likewise v; inside
 *           the pixel square floor() picks, the sample is bilinear in u, v),
 *   dL/dP += [dL/du; dL/dv; -(u dL/du + v dL/dv)] [p; 1]^T / h_3,  P = K [R | t],
 *   dL/dK = dL/dP [R | t]^T,   [dL/dR | dL/dt] = K^T dL/dP.
 *
 * Every entry of K, R and t gets its partial derivative (R is not constrained
 * to a rotation).
 *
 *   grad_out   : [B,C,X,Y] fp32, device, read only.
 *   features   : [B,N,H,W,C] fp32, device, read only (4-byte aligned;
 *                16-byte alignment with C a multiple of 4 takes the wide path).
 *   grad_K, grad_R : [B,N,3,3] fp32, device; fully overwritten.
 *   grad_t     : [B,N,3] fp32, device; fully overwritten.
 *   workspace  : device scratch of at least the size that
 *                fbev_backward_cameras_workspace() reports for these sizes
 *                (may be NULL when that is 0); its contents are not needed
 *                before or after the call.  Calls that share a workspace must
 *                not overlap.
 * Other arguments as for fbev_forward; features are fp32 only.  A workspace
 * smaller than required gives FBEV_ERR_INVALID_ARGUMENT.  The result is deterministic: partial sums per workgroup are added in a
 * fixed order in fp64.  Zero sizes give zero (or empty) gradients.
 */
/*
 * Temporal fused view transform.  The FlashBEV notes name a temporal fused
 * transform as future work ("Takeaway" item 4); the SparseDriveV2 notes ask
 * that history be moved into the current ego frame before use (ego-motion
 * compensation), and the Lift-Splat-Shoot tutorial stacks two BEV maps of one
 * scene in the same BEV space (the BEVFusion paragraph).  This call writes
 *
 *   out[b, 0:C]      = fbev_forward(features, ...)[b]           (current frame)
 *   out[b, C:C+Cp]   = prev_bev[b] resampled at the current cells
 *
 * where current cell (i, j), centre (x, y), maps to (x', y') = A_b [x; y; 1]
 * in the previous ego frame, i.e. to the continuous cell index
 * i' = (x' - x_min)/dx - 1/2, j' = (y' - y_min)/dy - 1/2 of the previous map,
 * which lies on the same grid (bev_range, X, Y).  Inside the closed box
 * [0, X-1] x [0, Y-1] of cell centres the previous map is sampled bilinearly
 * (the clamped tap at i' = X-1 has weight 0); outside it the value is 0.
 *
 *   prev_bev : [B,Cp,X,Y] fp32, device, read only (NULL allowed when B*Cp*X*Y == 0).
 *   ego      : [B,2,3] fp32, device: A_b, current-ego (x, y) -> previous-ego
 *              (x, y) in metres (a rigid planar motion in practice).
 *   out      : [B,C+Cp,X,Y] fp32, device, fully overwritten.
 *   counts   : as for fbev_forward.
 * Other arguments as for fbev_forward.  Deterministic.  Cp < 0 or NULL
 * pointers for non-empty buffers -> FBEV_ERR_INVALID_ARGUMENT; X*Y >= 2^31 ->
 * FBEV_ERR_UNSUPPORTED.
 */
fbev_status fbev_forward_temporal(const void* features, fbev_dtype dtype, fbev_feat_desc fd, const float* K,
                                  const float* R, const float* t, fbev_range bev_range, int32_t X, int32_t Y,
                                  int32_t Z, const float* prev_bev, int32_t Cp, const float* ego, float* out,
                                  uint8_t* counts, void* stream);

/*
 * Gradients of fbev_forward_temporal: dL/dF from grad_out[:, 0:C] exactly as
 * fbev_backward, and dL/dprev_bev [B,Cp,X,Y] (fp32, device, fully overwritten,
 * deterministic) = the adjoint of the resampling: every current cell passes
 * grad_out[b, C + c, i, j] times its bilinear weights to its four taps.  The
 * adjoint is computed as a gather over the current cells whose sample can
 * reach a previous cell, within 16 cells per axis of the inverse-mapped cell.
 * A rigid motion stays inside that window whatever its turn when the cell
 * aspect ratio dx/dy lies in (1/15, 15); other grids give
 * FBEV_ERR_UNSUPPORTED when Cp > 0.  A non-rigid motion (ego is read on the
 * device, so the host cannot check it) whose inverse stretches the grid past
 * the window leaves those previous cells' gradient at 0.  No gradient with
 * respect to the ego motion.
 *   grad_out : [B,C+Cp,X,Y] fp32, device, read only.
 */
fbev_status fbev_backward_temporal(const float* grad_out, fbev_feat_desc fd, const float* K, const float* R,
                                   const float* t, fbev_range bev_range, int32_t X, int32_t Y, int32_t Z, int32_t Cp,
                                   const float* ego, float* grad_features, float* grad_prev, void* stream);

fbev_status fbev_backward_cameras_workspace(fbev_feat_desc fd, int32_t X, int32_t Y, int32_t Z, size_t* bytes);
fbev_status fbev_backward_cameras(const float* grad_out, const float* features, fbev_feat_desc fd, const float* K,
                                  const float* R, const float* t, fbev_range bev_range, int32_t X, int32_t Y,
                                  int32_t Z, float* grad_K, float* grad_R, float* grad_t, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * fbev_backward_cameras without a workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation).  Same arguments, results and errors as
 * fbev_backward_cameras minus the workspace; this call allocates nothing.
 *
 * The partial sums live in a fixed device scratch of FBEV_NOALLOC_SCRATCH_BYTES
 * (4 MiB) that the library holds on every GPU it runs on until the process
 * ends; its address is looked up on the first call on each device.  Problems
 * that need more than that (what fbev_backward_cameras_workspace reports: at
 * most N * 172032 bytes for B <= 27, so up to 24 cameras always fit there)
 * return FBEV_ERR_UNSUPPORTED before anything is enqueued.  Every call on one GPU shares that GPU's scratch, and each
 * call overwrites all of it that it reads: calls that overlap on one GPU (on
 * different streams, or from different threads) race and must be serialized
 * by the caller.  The scratch needs no clearing between calls.
 */
#define FBEV_NOALLOC_SCRATCH_BYTES (4 << 20)
fbev_status fbev_backward_cameras_noalloc(const float* grad_out, const float* features, fbev_feat_desc fd,
                                          const float* K, const float* R, const float* t, fbev_range bev_range,
                                          int32_t X, int32_t Y, int32_t Z, float* grad_K, float* grad_R,
                                          float* grad_t, void* stream);

/*
 * Multi-level (feature-pyramid) variants.  The pages name a multi-scale fused
 * view transform as the next step (FlashBEV notes, "Limitation" item 4 and
 * "Takeaway" item 4) and describe the FPN pyramid it would read
 * (SparseDriveV2 notes, "Multi-scale features": P2-P5 at growing strides);
 * they do not define the fused operator, so this library fixes it as the
 * single-level operator with each camera's sample replaced by the mean of its
 * L level samples:
 *   - level l is (H / r_l) x (W / r_l) with integer ratios r_l, r_0 = 1; K maps
 *     to level-0 pixels; validity and the camera count are decided at level 0
 *     exactly as in fbev_forward;
 *   - level l is sampled at u_l = (u + 1/2) / r_l - 1/2 (v likewise): a level
 *     pixel centre sits at the centre of the r_l x r_l level-0 block it covers;
 *     u_l, v_l are clamped to the level's pixel-centre box (border replication);
 *   - camera sample = (1/L) sum_l bilinear_l; then the valid-camera mean and
 *     the height sum as in fbev_forward.  L = 1 is fbev_forward.
 *
 *   features : [B, N, P, C] with P = sum_l (H/r_l)(W/r_l): per camera, level 0's
 *              pixels row-major, then level 1's, ... (dtype and alignment as for
 *              fbev_forward).  fd.H, fd.W describe level 0.
 *   L        : 1..FBEV_MAX_LEVELS levels, with N * L <= 64.
 *   ratios   : host array of L ratios (ratios[0] = 1, each divides H and W), read
 *              during the call only; may be NULL when L = 1.
 * Other arguments, outputs and errors as for fbev_forward.
 */
fbev_status fbev_forward_levels(const void* features, fbev_dtype dtype, fbev_feat_desc fd, int32_t L,
                                const int32_t* ratios, const float* K, const float* R, const float* t,
                                fbev_range bev_range, int32_t X, int32_t Y, int32_t Z, float* out, uint8_t* counts,
                                void* stream);

/*
 * Gradient of fbev_forward_levels with respect to the packed level features:
 * grad_features is [B, N, P, C] fp32 in the same packing, fully overwritten
 * (zeroed on `stream`, then accumulated with fp32 atomics).  The adjoint of the
 * level mean scales each level's taps by 1/L.  Other arguments as for
 * fbev_forward_levels and fbev_backward.
 */
fbev_status fbev_backward_levels(const float* grad_out, fbev_feat_desc fd, int32_t L, const int32_t* ratios,
                                 const float* K, const float* R, const float* t, fbev_range bev_range, int32_t X,
                                 int32_t Y, int32_t Z, float* grad_features, void* stream);

/*
 * Lift-Splat, the push view transform (Lift-Splat-Shoot tutorial, sections
 * "Lift" and "Splat").  Every feature-map pixel (n, v, u) carries a depth
 * distribution alpha over D bins and a context vector c of C channels; bin k
 * puts the point alpha_k * c on the pixel's ray at camera depth
 * d_k = d_min + k * d_step (the tutorial's nuScenes setting: [4, 45) at 1 m,
 * 41 bins at 4, 5, ..., 44).  The point moves to the ego frame,
 *   p = R_n^T (d_k K_n^-1 [u, v, 1]^T - t_n)     ((R, t) maps ego to camera),
 * and lands in BEV cell (i, j) = (floor((p_x - x_min) / dx), floor((p_y - y_min) / dy)),
 * dx = (x_max - x_min) / X, dy = (y_max - y_min) / Y, when 0 <= i < X and
 * 0 <= j < Y; there is no bound on p_z (each cell is a pillar) and
 * bev_range.z_min / z_max are not used.  Each cell sums its points:
 *
 *   out[b, c, i, j] = sum over (n, k, v, u) whose point lands in (i, j) of alpha[b,n,v,u,k] * ctx[b,n,v,u,c]
 *
 * The geometry and the cell index are evaluated in double precision; the
 * products and sums are fp32.  A point within rounding of a cell edge lands in
 * one of the two cells, never in both or neither.  No point, cell index or
 * sorted order is stored in device memory.
 *
 *   depth    : alpha, [B, N, H, W, D] fp32, device, read only (any values; a
 *              softmax output in the tutorial's network).
 *   context  : c, [B, N, H, W, C] fp32 (channels-last), device, read only.
 *   fd       : B, N, C (context channels), H, W of the feature map.
 *   D, d_min, d_step : the depth bins, 0 <= D <= FBEV_MAX_GRID, d_step > 0.
 *   K, R, t  : as for fbev_forward (K in feature-map pixels).
 *   out      : [B, C, X, Y] fp32, device, fully overwritten (zero where no
 *              point lands).  Deterministic.
 * Errors as for fbev_forward; FBEV_ERR_UNSUPPORTED when one sample's depth or
 * context has 2^31 elements or more.
 */
fbev_status fbev_lss_forward(const float* depth, const float* context, fbev_feat_desc fd, int32_t D, float d_min,
                             float d_step, const float* K, const float* R, const float* t, fbev_range bev_range,
                             int32_t X, int32_t Y, float* out, void* stream);

/*
 * Gradients of fbev_lss_forward.  With the geometry fixed the forward is
 * bilinear in (alpha, c) (tutorial, "Lift": the point features are the outer
 * product of the two), so for the point of bin k of pixel q landing in cell s:
 *
 *   grad_depth[b, q, k]   = <ctx[b, q, :], grad_out[b, :, s]>     (0 for points outside the grid)
 *   grad_context[b, q, c] = sum over q's landing points of alpha[b, q, k] * grad_out[b, c, s]
 *
 *   grad_out     : [B, C, X, Y] fp32, device, read only.
 *   depth, context : the forward's inputs (read only).
 *   grad_depth   : [B, N, H, W, D] fp32, device, fully overwritten.
 *   grad_context : [B, N, H, W, C] fp32, device, fully overwritten.
 * Both outputs are zeroed on `stream` and then accumulated with fp32 atomics:
 * grad_depth is deterministic for C <= 64 (one add per element), grad_context
 * sums one add per (pixel, 4 x 8 cell tile) in run-dependent order.  Pointers
 * whose buffer has no elements may be NULL.  Other arguments and errors as
 * for fbev_lss_forward.
 */
fbev_status fbev_lss_backward(const float* grad_out, const float* depth, const float* context, fbev_feat_desc fd,
                              int32_t D, float d_min, float d_step, const float* K, const float* R, const float* t,
                              fbev_range bev_range, int32_t X, int32_t Y, float* grad_depth, float* grad_context,
                              void* stream);

/*
 * Deformable Aggregation: multi-camera deformable sampling (SparseDriveV2
 * notes, "Deformable Aggregation", steps 1-3), the operator the FlashBEV
 * notes fuse for BEVFormer's spatial cross-attention.  For query q of batch
 * sample b with anchor a_q and keypoint offsets o_{q,k} (k < Kp):
 *
 *   p_{q,k} = a_q + o_{q,k}                                   (ego frame, metres)
 *   out[b, q, c] = sum_n sum_k  weights[b,q,n,k] * bilinear(F[b,n,:,:,c], u, v)   over (n, k) in view
 *
 * with [u, v, 1]^T ~ K_n (R_n p + t_n) and the in-view rule, pixel-centre
 * convention and bilinear taps of fbev_forward (depth > 0, closed box
 * [0, W-1] x [0, H-1]).  The weights are used as given (no renormalisation
 * over the pairs in view).  Projection and the in-view test in double
 * precision, interpolation and sums in fp32.
 *
 *   features : [B, N, H, W, C] fp32 channels-last, device, read only.
 *   K, R, t  : as for fbev_forward.
 *   anchors  : [B, Q, 3] fp32; offsets : [B, Q, Kp, 3] fp32; weights : [B, Q, N, Kp] fp32; device.
 *   Q, Kp    : queries per sample and keypoints per query (Kp <= FBEV_MAX_KEYPOINTS).
 *   out      : [B, Q, C] fp32, device, fully overwritten.  Deterministic.
 * Errors as for fbev_forward.
 */
fbev_status fbev_deform_forward(const float* features, fbev_feat_desc fd, const float* K, const float* R,
                                const float* t, const float* anchors, const float* offsets, const float* weights,
                                int32_t Q, int32_t Kp, float* out, void* stream);

/*
 * Gradients of fbev_deform_forward with the in-view mask held fixed (the page
 * asks for a sampling chain that gradients pass through):
 *   grad_features : [B,N,H,W,C] fp32 — each in-view sample adds w * tap weight * g
 *                   to its four taps.  Computed as a gather: a query's taps on one
 *                   pixel are merged, each (query, pixel) pair becomes an entry in the
 *                   pixel's bucket, and every element is the sum over its bucket
 *                   (written once; the order within a bucket varies run to run, so
 *                   the last bits may too).
 *   grad_weights  : [B,Q,N,Kp] fp32 — <sample, g> for pairs in view, 0 otherwise.
 *   grad_offsets  : [B,Q,Kp,3] fp32 — sum over cameras of w (<ds/du, g> du/dp + <ds/dv, g> dv/dp),
 *                   the bilinear sample's derivative inside its pixel square times the
 *                   projection's Jacobian du/dp = (P_1 - u P_3) / h_3 (P = K [R | t]).
 *   grad_anchors  : [B,Q,3] fp32 — the sum of grad_offsets over k; may be NULL.
 *   workspace     : device scratch of at least the size that
 *                   fbev_deform_backward_workspace() reports for these sizes (may be
 *                   NULL when that is 0), 16-byte aligned; its contents are not needed
 *                   before or after the call.  Calls that share a workspace must not
 *                   overlap.  It holds per-pixel counts and offsets and up to
 *                   4 N Kp entries of 20 bytes per query.
 * All outputs are fully overwritten; grad_out is [B,Q,C]; other arguments as
 * for fbev_deform_forward.  A workspace smaller than required gives
 * FBEV_ERR_INVALID_ARGUMENT; B N H W or B Q 4 N Kp of 2^31 or more gives
 * FBEV_ERR_UNSUPPORTED.
 */
fbev_status fbev_deform_backward_workspace(fbev_feat_desc fd, int32_t Q, int32_t Kp, size_t* bytes);
fbev_status fbev_deform_backward(const float* grad_out, const float* features, fbev_feat_desc fd, const float* K,
                                 const float* R, const float* t, const float* anchors, const float* offsets,
                                 const float* weights, int32_t Q, int32_t Kp, float* grad_features,
                                 float* grad_weights, float* grad_offsets, float* grad_anchors, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * Encoder operators: what stands before and after the view transforms in a
 * camera-BEV model.  Tensors are fp32 or bf16 (`dtype`); sums, statistics and
 * softmax are fp32 and results are rounded once to the tensor's type.  All
 * three are deterministic, allocate nothing and write every element of their
 * outputs.  The work runs on `stream`, whose device must be the current one.
 *
 * Group norm with an activation on channels-last maps: x holds `images`
 * images of `pixels` pixels (image_stride and pixel_stride elements apart)
 * with C contiguous channels in `groups` groups of neighbours.  Per image and
 * group, over its pixels and channels:
 *
 *   xh = (x - mean) / sqrt(var + eps),  z = weight xh + bias,  y = act(z)
 *
 *   weight, bias : [C] fp32, device, or NULL (ones / zeros).
 *   y            : [images, pixels, C] of dtype, contiguous, not on x.
 *   stats        : [images, groups, 2] fp32: mean and 1 / sqrt(var + eps)
 *                  (without pixels: 0 and 1 / sqrt(eps)).
 *   workspace    : device scratch of the size the workspace call reports
 *                  (NULL when 0), 16-byte aligned; not needed before or after
 *                  the call.  Calls that share it must not overlap.
 *
 * The backward takes grad_y and gives grad_x (both [images, pixels, C],
 * contiguous, of dtype) and the fp32 sums grad_weight, grad_bias [C] (NULL
 * skips one).  A ReLU's derivative at 0 is 0.
 *
 * C must be a multiple of groups, and a group may hold at most 1024 pieces of
 * 16 bytes (1024 channels where C or the strides do not allow wide moves):
 * FBEV_ERR_UNSUPPORTED beyond.  Zero images or pixels are allowed.
 */
typedef enum { FBEV_ACT_NONE = 0, FBEV_ACT_RELU = 1, FBEV_ACT_SILU = 2, FBEV_ACT_GELU = 3 } fbev_activation;

typedef struct {
  int64_t images, pixels;
  int64_t image_stride, pixel_stride; /* of x, in elements */
  int32_t C, groups;
  int32_t activation; /* fbev_activation; GELU is the exact one (erf) */
  float eps;
} fbev_norm_desc;

fbev_status fbev_group_norm_workspace(const fbev_norm_desc* nd, fbev_dtype dtype, int32_t backward, size_t* bytes);
fbev_status fbev_group_norm_forward(const void* x, fbev_dtype dtype, const fbev_norm_desc* nd, const float* weight,
                                    const float* bias, void* y, float* stats, void* workspace,
                                    size_t workspace_bytes, void* stream);
fbev_status fbev_group_norm_backward(const void* grad_y, const void* x, fbev_dtype dtype, const fbev_norm_desc* nd,
                                     const float* weight, const float* bias, const float* stats, void* grad_x,
                                     float* grad_weight, float* grad_bias, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Rotary positions with several axes (time, height, width, metres ...): every
 * token's queries and keys are turned, pair of channels by pair, by
 *
 *   theta[b,t,i] = sum_a pos[b,t,a] freqs[a,i]       (i < P; formed in double)
 *   (x1, x2) -> (x1 cos theta - x2 sin theta, x2 cos theta + x1 sin theta)
 *
 * Pair i is channels (i, i + P), or (2i, 2i + 1) when `interleaved`; channels
 * from 2P on are copied.  `inverse` turns by -theta: the backward of the
 * operator, applied to the gradients.
 *
 *   q, k       : [B, T, heads, D] by element strides (batch, token, head), channels
 *                contiguous; a tensor with 0 heads may be NULL.
 *   q_out, k_out : the results, by their own strides.  q_out may be q and k_out k
 *                (same strides); apart from that no output may share memory with
 *                an input, the other output or itself: one launch turns both, and
 *                its workgroups read and write in any order.
 *   pos        : [B, T, A] fp32;  freqs : [A, P] fp32, device; 1 <= A <= 8,
 *                1 <= P <= min(D / 2, FBEV_MAX_ROTARY_PAIRS).
 */
typedef struct {
  int32_t B, T, D, axes, pairs;
  int32_t q_heads, k_heads;
  int32_t interleaved, inverse;
  int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];
} fbev_rotary_desc;

fbev_status fbev_rotary(const void* q, const void* k, fbev_dtype dtype, const fbev_rotary_desc* rd, const float* pos,
                        const float* freqs, void* q_out, void* k_out, void* stream);

/*
 * Attention between queries, BEV cells and tokens.  For query i, key j and
 * query head n (key head n / (Hq / Hk)):
 *
 *   s = scale q_i . k_j,   s = cap tanh(s / cap)  when cap > 0,
 *   s = s - slope[b,i,n] |pos_q[b,i] - pos_k[b,j]|_2  when dims > 0,
 *   o_i = sum_j softmax_j(s) v_j  over the keys i sees.
 *
 * Key j is seen when doc_q[b,i] == doc_k[b,j] >= 0 (without documents:
 * always) and, when `causal`, j <= i + Tk - Tq or j < prefix[b].  A query
 * that sees no key gets zeros; what masked keys hold, NaN and infinities among
 * it, reaches no query that does not see them.
 *
 *   q [B,Tq,Hq,D], k, v [B,Tk,Hk,D] : by element strides (batch, token, head), channels
 *       contiguous; 16-byte aligned rows take the wide-load path.  Hq a
 *       multiple of Hk, 1 <= D <= FBEV_MAX_HEAD_DIM.
 *   pos_q [B,Tq,dims], pos_k [B,Tk,dims], slope [B,Tq,Hq] : fp32, contiguous,
 *       dims 0 .. 3 (0: none of them is read).
 *   doc_q [B,Tq], doc_k [B,Tk] : int32, both or neither; in any order, but
 *       documents that lie together are skipped tile by tile.
 *   prefix : [B] int32 or NULL; needs `causal`.
 *   scale, cap : 0 or of a size within [1e-12, 1e12] (cap 0: none).
 *   out [B,Tq,Hq,D] of dtype, contiguous, on memory of its own.
 *   stats [B,Hq,Tq,2] fp32, 8-byte aligned: m and l with sum_j exp(s_j) = 2^m l (no
 *       key: -inf and 0), what the backward needs of the softmax.  m is within 8 of
 *       the row's largest s log2(e); the pair keeps what one logarithm would round.
 *   workspace : as for group norm.  Few rows over many keys are split along the
 *       keys and joined from there.
 *
 * The backward takes grad_out, out [B,Tq,Hq,D] (contiguous, of dtype) and stats
 * and gives grad_q, grad_k, grad_v (contiguous, of dtype; a key head's
 * gradient is the sum over its query heads) and grad_slope [B,Tq,Hq] fp32
 * (NULL skips it).  Positions are not differentiated.  For bf16 tensors the
 * probabilities and score gradients of forward and backward go into their
 * matrix products as two bf16 each, which keeps 16 bits of them.  An
 * infinity or a NaN reaches the gradients of what sees it and no others.
 */
typedef struct {
  int32_t B, Tq, Tk, Hq, Hk, D;
  int64_t q_stride[3], k_stride[3], v_stride[3];
  float scale, cap;
  int32_t dims, causal;
  const float *pos_q, *pos_k, *slope;
  const int32_t *doc_q, *doc_k, *prefix;
} fbev_attention_desc;

fbev_status fbev_attention_workspace(const fbev_attention_desc* ad, int32_t backward, size_t* bytes);
fbev_status fbev_attention_forward(const void* q, const void* k, const void* v, fbev_dtype dtype,
                                   const fbev_attention_desc* ad, void* out, float* stats, void* workspace,
                                   size_t workspace_bytes, void* stream);
fbev_status fbev_attention_backward(const void* grad_out, const void* q, const void* k, const void* v,
                                    fbev_dtype dtype, const fbev_attention_desc* ad, const void* out,
                                    const float* stats, void* grad_q, void* grad_k, void* grad_v, float* grad_slope,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Decoder operators: what a decoder over a scene's tokens runs around its
 * projections, from training to one drafted token at a time.  Tensors are fp32
 * or bf16 (`dtype`); sums, statistics and softmax are fp32.  All of them are
 * deterministic and allocate nothing; the work runs on `stream`, whose device
 * must be the current one.
 *
 * Numbers in 8 bits: signed integers (int8, up to 127) or e4m3 (four
 * significant bits, up to 448, no infinities).  Values that share a scale have
 *
 *   scale = max(max_j |x_j| / most, 2^-126)      (a quotient of fp32)
 *   code  = the format's number nearest to x / scale, ties to the even one,
 *
 * decided on the exact quotient.  Where an x is infinite or NaN the scale is
 * NaN and the codes are 0.  A code stands for code * scale.
 */
typedef enum { FBEV_CODES_INT8 = 0, FBEV_CODES_E4M3 = 1 } fbev_codes;

/*
 * Root-mean-square norm with the residual's addition: per row of C channels
 *
 *   h = x + residual (rounded once to dtype; without a residual h is x)
 *   y = h w / sqrt(mean_c h^2 + eps)
 *
 *   x, residual : rows o < outer, i < inner at the given element strides,
 *                 channels contiguous, any alignment; residual may be NULL.
 *   weight      : [C] fp32 or NULL (ones).
 *   y, h        : [rows, C] of dtype, contiguous, rows = outer inner; h is NULL
 *                 without a residual.  h may be x or residual itself where that
 *                 one is contiguous; no other output may share memory with the call's tensors.
 *   rstd        : [rows] fp32, 1 / sqrt(mean h^2 + eps), what the backward needs; may be NULL.
 *
 * fbev_rms_norm_codes gives y in 8 bits instead.  Nothing is rounded in front: the
 * codes are nearest to the exact y over its exact scale, which is rounded once.
 *   out    : [rows, C] codes;  scales : [rows, ceil(C / block)] fp32, one for each
 *            `block` channels (32, 64 or 128), or [rows, 1] with block 0 or >= C.
 *
 * The backward takes h (the forward's x without a residual, by x's strides),
 * rstd, grad_y and grad_h (dL/dh from elsewhere, may be NULL), both [rows, C]
 * contiguous of dtype, and gives grad_x (dL/dx and dL/dresidual are the same;
 * contiguous, may be grad_y or grad_h) and grad_weight [C] fp32 (NULL skips it).
 *   workspace : device scratch of the size the workspace call reports, 16-byte
 *               aligned; not needed before or after the call, not shared by
 *               calls that overlap; NULL is fine without grad_weight.
 *
 * C up to FBEV_MAX_RMS_CHANNELS; 0 rows are allowed (grad_weight is zero then).
 * Without codes the sum of h^2 is fp32: past 2^128 it is infinite and y zero, and
 * squares below 2^-126 lose digits (which eps hides unless it is as small).
 */
#define FBEV_MAX_RMS_CHANNELS 16384

typedef struct {
  int64_t outer, inner;
  int64_t x_stride[2], residual_stride[2]; /* of outer and of inner rows, in elements */
  int32_t C;
  float eps;
} fbev_rms_desc;

fbev_status fbev_rms_norm_forward(const void* x, const void* residual, fbev_dtype dtype, const fbev_rms_desc* rd,
                                  const float* weight, void* y, void* h, float* rstd, void* stream);
fbev_status fbev_rms_norm_codes(const void* x, const void* residual, fbev_dtype dtype, const fbev_rms_desc* rd,
                                const float* weight, fbev_codes codes, int32_t block, void* out, float* scales,
                                void* h, void* stream);
fbev_status fbev_rms_norm_workspace(const fbev_rms_desc* rd, fbev_dtype dtype, size_t* bytes);
fbev_status fbev_rms_norm_backward(const void* grad_y, const void* grad_h, const void* h, fbev_dtype dtype,
                                   const fbev_rms_desc* rd, const float* weight, const float* rstd, void* grad_x,
                                   float* grad_weight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Token cache: keys and values of many sequences in 8 bits, in pages of
 * FBEV_CACHE_PAGE tokens that any sequence may hold in any order.
 *
 *   k       : [pages, Hk, 64, Dp] codes,  v : [pages, Hk, Dp, 64] codes (tokens
 *             side by side), Dp = D rounded up to a multiple of 16, zeros behind D;
 *             both 16-byte aligned.  1 <= D <= FBEV_MAX_HEAD_DIM.
 *   k_scale, v_scale : [pages, Hk, 64] fp32, 16-byte aligned: one scale for each token and key head.
 *
 * A call's rows:
 *   table   : [B, W] int32, page of the sequence's tokens 64 w .. 64 w + 63.
 *   start   : [B] int32, the tokens the cache holds for the sequence; the call's
 *             row t < T of sequence b is its token start[b] + t.
 *   count   : [B] int32 or NULL (T for all): rows t >= count[b] are padding.
 *
 * Nothing outside the cache is touched whatever these hold: a page that is not
 * in [0, pages) and tokens beyond 64 W do not exist, and a sequence with a
 * negative start has no tokens and no rows.
 *
 * fbev_cache_write quantises the rows k, v [B, T, Hk, D] (by element strides of
 * batch, token, head, channels contiguous, any alignment) into their tokens;
 * rows that are padding or have no page are dropped, and what they would
 * have replaced stays.  Two rows of one call must not be the same token of the same page
 * (sequences may share pages that none of them writes).
 *
 * fbev_cache_read gives the values that the codes of the rows' tokens stand
 * for (code * scale in fp32, then in dtype): k_out, v_out [B, T, Hk, D],
 * contiguous, zeros for rows that are padding or have no page.  Either may be NULL.
 */
#define FBEV_CACHE_PAGE 64

typedef struct {
  int32_t pages, Hk, D;
  int32_t codes; /* fbev_codes */
  void *k, *v;
  float *k_scale, *v_scale;
} fbev_cache_desc;

typedef struct {
  int32_t B, T, W;
  const int32_t *table, *start, *count;
} fbev_cache_rows;

fbev_status fbev_cache_write(const fbev_cache_desc* cd, const fbev_cache_rows* cr, const void* k, const void* v,
                             fbev_dtype dtype, const int64_t k_stride[3], const int64_t v_stride[3], void* stream);
fbev_status fbev_cache_read(const fbev_cache_desc* cd, const fbev_cache_rows* cr, fbev_dtype dtype, void* k_out,
                            void* v_out, void* stream);

/*
 * Attention of T query tokens a sequence over the cache, for query head n of
 * key head n / (Hq / Hk), with the values that the cache's codes stand for:
 *
 *   s = scale q_i . k_j,   s = cap tanh(s / cap) when cap > 0,
 *   o_i = sum_j softmax_j(s) v_j  over the tokens i sees.
 *
 * Every query sees the start[b] tokens of its sequence, and of the call's own
 * rows, which are in the cache too (written before), `drafts` says which:
 *   FBEV_DRAFT_NONE  : none (queries that are not tokens of the cache).
 *   FBEV_DRAFT_CHAIN : those up to itself: a prompt, a single new token.
 *   FBEV_DRAFT_TREE  : row j where bit j % 64 of ancestors[b, i, j / 64] is set
 *                      (its own bit is up to the caller): several drafted continuations at once.
 * With `count`, rows t >= count[b] are padding: nobody sees them and they get
 * zeros, as does a query that sees no token.  What unseen tokens hold reaches no
 * query: NaN in the scales of any of them, and any bytes at all behind the
 * call's last row (the tokens before it hold codes as fbev_cache_write makes them).
 *
 *   q   : [B, T, Hq, D] by element strides, channels contiguous, any alignment.
 *   ancestors : [B, T, words] uint64, words >= ceil(T / 64); NULL without a tree.
 *   scale, cap : as for fbev_attention_forward.
 *   out : [B, T, Hq, D] of dtype, contiguous, on memory of its own: finite for
 *         values of up to 2^127, with all digits in sequences whose largest
 *         value is 2^-80 W or more.  Scores are fp32: past 2^128, the
 *         product of a query with a key's codes among them, they are infinite.
 *   workspace : as above; few queries over many tokens are split along the
 *               tokens and joined from there (many: 64 W, all that the host
 *               knows of them; a table far wider than the sequences need costs time).
 */
typedef enum { FBEV_DRAFT_NONE = 0, FBEV_DRAFT_CHAIN = 1, FBEV_DRAFT_TREE = 2 } fbev_drafts;

typedef struct {
  int32_t Hq;
  int32_t drafts; /* fbev_drafts */
  int32_t words;
  int64_t q_stride[3];
  const uint64_t* ancestors;
  float scale, cap;
} fbev_cache_attention_desc;

fbev_status fbev_cache_attention_workspace(const fbev_cache_desc* cd, const fbev_cache_rows* cr,
                                           const fbev_cache_attention_desc* ad, fbev_dtype dtype, size_t* bytes);
fbev_status fbev_cache_attention(const fbev_cache_desc* cd, const fbev_cache_rows* cr,
                                 const fbev_cache_attention_desc* ad, const void* q, fbev_dtype dtype, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Static text for a status code. */
const char* fbev_status_string(fbev_status s);

/* Message for the last non-OK status returned on the calling thread ("" if none). */
const char* fbev_last_error(void);

/* FBEV_ABI_VERSION of the built library. */
int32_t fbev_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FLASHBEV_H */
