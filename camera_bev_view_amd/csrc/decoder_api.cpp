// C-ABI host layer of the decoder operators (root-mean-square norm, token cache, attention over it): argument validation.
// Every check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/flashbev.h"
#include "decoder.h"
#include "host_status.h"

namespace {

using fbev::fail;

fbev_status device_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return FBEV_OK;
  return fail(FBEV_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

bool known(fbev_dtype dtype) { return dtype == FBEV_DTYPE_F32 || dtype == FBEV_DTYPE_BF16; }
bool known_codes(int codes) { return codes == FBEV_CODES_INT8 || codes == FBEV_CODES_E4M3; }
int elem_bytes(fbev_dtype dtype) { return dtype == FBEV_DTYPE_F32 ? 4 : 2; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fbev_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && (workspace == nullptr || have < need))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "workspace of %zu bytes given, %zu needed", workspace ? have : 0, need);
  if (!aligned(workspace, 16)) return fail(FBEV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  return FBEV_OK;
}

// ---- root-mean-square norm

fbev_status check_rms(const fbev_rms_desc* rd, fbev_dtype dtype, fbev::RmsArgs& a) {
  if (rd == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the norm descriptor is NULL");
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (rd->outer < 0 || rd->inner < 0 || rd->C < 1)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "outer=%lld and inner=%lld must not be negative, C=%d must be positive",
                (long long)rd->outer, (long long)rd->inner, rd->C);
  if (rd->C > FBEV_MAX_RMS_CHANNELS)
    return fail(FBEV_ERR_UNSUPPORTED, "C=%d exceeds FBEV_MAX_RMS_CHANNELS=%d", rd->C, FBEV_MAX_RMS_CHANNELS);
  if (!std::isfinite(rd->eps) || rd->eps < 0.0f)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  for (int i = 0; i < 2; ++i)
    if (rd->x_stride[i] < 0 || rd->residual_stride[i] < 0) return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
  const int64_t limit = (int64_t)1 << 31;
  if (rd->outer >= limit || rd->inner >= limit || rd->outer * rd->inner >= limit)
    return fail(FBEV_ERR_UNSUPPORTED, "%lld x %lld rows: above 2^31 - 1", (long long)rd->outer, (long long)rd->inner);
  a.outer = rd->outer;
  a.inner = rd->inner;
  a.rows = rd->outer * rd->inner;
  a.C = rd->C;
  a.eps = rd->eps;
  a.part_of_row = 1.0 / rd->C;
  a.elem_bytes = elem_bytes(dtype);
  a.codes = -1;
  for (int i = 0; i < 2; ++i) {
    a.xs[i] = rd->x_stride[i];
    a.rs[i] = rd->residual_stride[i];
  }
  return FBEV_OK;
}

// Rows of both tensors by one stride where they have one: the kernels need no division then.
void flatten_rows(fbev::RmsArgs& a, bool residual) {
  const auto one = [&](int64_t (&s)[2]) {
    if (a.inner == 1) return true;
    if (a.outer == 1 || s[0] == a.inner * s[1]) {
      s[0] = s[1];
      return true;
    }
    return false;
  };
  int64_t x[2] = {a.xs[0], a.xs[1]}, r[2] = {a.rs[0], a.rs[1]};
  if (!one(x) || (residual && !one(r))) return;
  for (int i = 0; i < 2; ++i) {
    a.xs[i] = x[i];
    a.rs[i] = r[i];
  }
  a.outer = a.rows;
  a.inner = 1;
}

fbev_status rms_forward(const void* x, const void* residual, fbev_dtype dtype, const fbev_rms_desc* rd,
                        const float* weight, void* y, void* h, fbev::RmsArgs& a) {
  const fbev_status s = check_rms(rd, dtype, a);
  if (s != FBEV_OK) return s;
  if (a.rows > 0 && (x == nullptr || y == nullptr))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "x and the output must be non-NULL");
  if (a.rows > 0 && (residual == nullptr) != (h == nullptr))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "residual and h come together");
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.y = y;
  a.h = h;
  flatten_rows(a, residual != nullptr);
  return FBEV_OK;
}

// ---- cache

fbev_status check_cache(const fbev_cache_desc* cd, const fbev_cache_rows* cr, fbev::CacheArgs& a) {
  if (cd == nullptr || cr == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the cache or its rows are NULL");
  if (cd->pages < 0 || cd->Hk < 1 || cd->D < 1 || cr->B < 0 || cr->T < 0 || cr->W < 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "bad size (pages=%d Hk=%d D=%d B=%d T=%d W=%d)", cd->pages, cd->Hk, cd->D,
                cr->B, cr->T, cr->W);
  if (!known_codes(cd->codes)) return fail(FBEV_ERR_INVALID_ARGUMENT, "unknown codes %d", cd->codes);
  if (cd->D > FBEV_MAX_HEAD_DIM)
    return fail(FBEV_ERR_UNSUPPORTED, "D=%d exceeds FBEV_MAX_HEAD_DIM=%d", cd->D, FBEV_MAX_HEAD_DIM);
  if (cr->W > (1 << 24) || cr->T > (1 << 30))
    return fail(FBEV_ERR_UNSUPPORTED, "W=%d pages a sequence (limit 2^24) or T=%d rows (limit 2^30)", cr->W, cr->T);
  if (cd->pages > 0 && (cd->k == nullptr || cd->v == nullptr || cd->k_scale == nullptr || cd->v_scale == nullptr))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "the cache's tensors must be non-NULL");
  if (!aligned(cd->k, 16) || !aligned(cd->v, 16) || !aligned(cd->k_scale, 16) || !aligned(cd->v_scale, 16))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "the cache's tensors must be 16-byte aligned");
  if (cr->B > 0 && cr->T > 0 && (cr->start == nullptr || (cr->W > 0 && cr->table == nullptr)))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "table and start must be non-NULL");
  a.k = cd->k;
  a.v = cd->v;
  a.k_scale = cd->k_scale;
  a.v_scale = cd->v_scale;
  a.pages = cd->pages;
  a.Hk = cd->Hk;
  a.D = cd->D;
  a.Dp = fbev::padded_dim(cd->D);
  a.codes = cd->codes;
  a.table = cr->table;
  a.start = cr->start;
  a.count = cr->count;
  a.B = cr->B;
  a.T = cr->T;
  a.W = cr->W;
  return FBEV_OK;
}

fbev_status check_moves(const fbev::CacheArgs& a) {
  const int64_t tiles = ((int64_t)a.T + 62) / 64 + 1, limit = (int64_t)1 << 31;
  if ((int64_t)a.B * a.Hk >= limit || (int64_t)a.B * a.Hk * tiles >= limit)
    return fail(FBEV_ERR_UNSUPPORTED, "%lld pages of rows to move: above 2^31 - 1", (long long)tiles);
  return FBEV_OK;
}

fbev_status check_cache_attention(const fbev_cache_desc* cd, const fbev_cache_rows* cr,
                                  const fbev_cache_attention_desc* ad, fbev_dtype dtype, fbev::CacheAttnArgs& a) {
  fbev_status s = check_cache(cd, cr, a.c);
  if (s != FBEV_OK) return s;
  if (ad == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the attention descriptor is NULL");
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (ad->Hq < 1 || ad->Hq % cd->Hk != 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "Hq=%d is not a positive multiple of Hk=%d", ad->Hq, cd->Hk);
  if (ad->drafts < FBEV_DRAFT_NONE || ad->drafts > FBEV_DRAFT_TREE)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "unknown drafts %d", ad->drafts);
  if (!std::isfinite(ad->scale) || !std::isfinite(ad->cap) || ad->cap < 0.0f)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "scale and cap must be finite, cap not negative");
  const auto far = [](float x) { return x != 0.0f && !(std::fabs(x) >= 1e-12f && std::fabs(x) <= 1e12f); };
  if (far(ad->scale) || far(ad->cap))
    return fail(FBEV_ERR_UNSUPPORTED, "scale=%g and cap=%g must be 0 or of a size within [1e-12, 1e12]", ad->scale,
                ad->cap);
  for (int i = 0; i < 3; ++i)
    if (ad->q_stride[i] < 0) return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
  const bool work = cr->B > 0 && cr->T > 0;
  if (ad->drafts == FBEV_DRAFT_TREE && work && ad->words < (cr->T + 63) / 64)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "%d words of ancestors for %d rows", ad->words, cr->T);
  if (!aligned(ad->ancestors, 8)) return fail(FBEV_ERR_INVALID_ARGUMENT, "ancestors must be 8-byte aligned");
  const int64_t G = ad->Hq / cd->Hk, rows = (int64_t)cr->T * G, limit = (int64_t)1 << 30;
  if (rows >= limit) return fail(FBEV_ERR_UNSUPPORTED, "T Hq / Hk = %lld rows (limit 2^30 - 1)", (long long)rows);
  // workgroups of up to 512 threads stay below a launch's 2^32
  const int64_t heads = (int64_t)cr->B * cd->Hk, tiles = (rows + 15) / 16, most = ((int64_t)1 << 23) - 1;
  if (heads > most || (tiles > 0 && heads > most / tiles))
    return fail(FBEV_ERR_UNSUPPORTED, "B Hk = %lld heads of %lld tiles of 16 rows: above 2^23 - 1", (long long)heads,
                (long long)tiles);
  a.Hq = ad->Hq;
  a.G = (int)G;
  a.R = (int)rows;
  a.mode = ad->drafts;
  a.ancestors = ad->ancestors;
  a.words = ad->words;
  a.scale = ad->scale;
  a.cap = ad->cap;
  for (int i = 0; i < 3; ++i) a.qs[i] = ad->q_stride[i];
  a.elem_bytes = elem_bytes(dtype);
  return FBEV_OK;
}

}  // namespace

extern "C" {

fbev_status fbev_rms_norm_forward(const void* x, const void* residual, fbev_dtype dtype, const fbev_rms_desc* rd,
                                  const float* weight, void* y, void* h, float* rstd, void* stream) {
  fbev::RmsArgs a{};
  const fbev_status s = rms_forward(x, residual, dtype, rd, weight, y, h, a);
  if (s != FBEV_OK || a.rows == 0) return s;
  a.rstd = rstd;
  return device_status(fbev::launch_rms_norm_forward(a, static_cast<hipStream_t>(stream)),
                       "fbev_rms_norm_forward launch");
}

fbev_status fbev_rms_norm_codes(const void* x, const void* residual, fbev_dtype dtype, const fbev_rms_desc* rd,
                                const float* weight, fbev_codes codes, int32_t block, void* out, float* scales,
                                void* h, void* stream) {
  fbev::RmsArgs a{};
  const fbev_status s = rms_forward(x, residual, dtype, rd, weight, out, h, a);
  if (s != FBEV_OK) return s;
  if (!known_codes(codes)) return fail(FBEV_ERR_INVALID_ARGUMENT, "unknown codes %d", (int)codes);
  if (block < 0 || (block > 0 && block < a.C && block != 32 && block != 64 && block != 128))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "block=%d must be 0, 32, 64, 128 or at least C=%d", block, a.C);
  if (a.rows == 0) return FBEV_OK;
  if (scales == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "scales must be non-NULL");
  a.codes = codes;
  a.block = block == 0 || block > a.C ? a.C : block;
  a.scales = scales;
  return device_status(fbev::launch_rms_norm_forward(a, static_cast<hipStream_t>(stream)),
                       "fbev_rms_norm_codes launch");
}

fbev_status fbev_rms_norm_workspace(const fbev_rms_desc* rd, fbev_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "bytes is NULL");
  fbev::RmsArgs a{};
  const fbev_status s = check_rms(rd, dtype, a);
  if (s != FBEV_OK) return s;
  *bytes = fbev::rms_norm_workspace_bytes(a);
  return FBEV_OK;
}

fbev_status fbev_rms_norm_backward(const void* grad_y, const void* grad_h, const void* h, fbev_dtype dtype,
                                   const fbev_rms_desc* rd, const float* weight, const float* rstd, void* grad_x,
                                   float* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
  fbev::RmsArgs a{};
  fbev_status s = check_rms(rd, dtype, a);
  if (s != FBEV_OK) return s;
  if (a.rows == 0 && grad_weight == nullptr) return FBEV_OK;
  if (a.rows > 0) {
    if (grad_y == nullptr || h == nullptr || rstd == nullptr || grad_x == nullptr)
      return fail(FBEV_ERR_INVALID_ARGUMENT, "grad_y, h, rstd and grad_x must be non-NULL");
    s = check_workspace(workspace, workspace_bytes, grad_weight ? fbev::rms_norm_workspace_bytes(a) : 0);
    if (s != FBEV_OK) return s;
  }
  a.gy = grad_y;
  a.gh = grad_h;
  a.x = h;
  a.weight = weight;
  a.rstd = const_cast<float*>(rstd);
  a.gx = grad_x;
  a.gweight = grad_weight;
  a.part = static_cast<float*>(workspace);
  flatten_rows(a, false);
  return device_status(fbev::launch_rms_norm_backward(a, static_cast<hipStream_t>(stream)),
                       "fbev_rms_norm_backward launch");
}

fbev_status fbev_cache_write(const fbev_cache_desc* cd, const fbev_cache_rows* cr, const void* k, const void* v,
                             fbev_dtype dtype, const int64_t k_stride[3], const int64_t v_stride[3], void* stream) {
  fbev::CacheMoveArgs a{};
  fbev_status s = check_cache(cd, cr, a.c);
  if (s == FBEV_OK) s = check_moves(a.c);
  if (s != FBEV_OK) return s;
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (k_stride == nullptr || v_stride == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the strides are NULL");
  for (int i = 0; i < 3; ++i) {
    if (k_stride[i] < 0 || v_stride[i] < 0) return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
    a.xs[0][i] = k_stride[i];
    a.xs[1][i] = v_stride[i];
  }
  if (a.c.B == 0 || a.c.T == 0 || a.c.W == 0 || a.c.pages == 0) return FBEV_OK;
  if (k == nullptr || v == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "k and v must be non-NULL");
  a.x[0] = k;
  a.x[1] = v;
  a.elem_bytes = elem_bytes(dtype);
  return device_status(fbev::launch_cache_write(a, static_cast<hipStream_t>(stream)), "fbev_cache_write launch");
}

fbev_status fbev_cache_read(const fbev_cache_desc* cd, const fbev_cache_rows* cr, fbev_dtype dtype, void* k_out,
                            void* v_out, void* stream) {
  fbev::CacheMoveArgs a{};
  fbev_status s = check_cache(cd, cr, a.c);
  if (s == FBEV_OK) s = check_moves(a.c);
  if (s != FBEV_OK) return s;
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (a.c.B == 0 || a.c.T == 0 || (k_out == nullptr && v_out == nullptr)) return FBEV_OK;
  a.y[0] = k_out;
  a.y[1] = v_out;
  a.elem_bytes = elem_bytes(dtype);
  return device_status(fbev::launch_cache_read(a, static_cast<hipStream_t>(stream)), "fbev_cache_read launch");
}

fbev_status fbev_cache_attention_workspace(const fbev_cache_desc* cd, const fbev_cache_rows* cr,
                                           const fbev_cache_attention_desc* ad, fbev_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "bytes is NULL");
  fbev::CacheAttnArgs a{};
  const fbev_status s = check_cache_attention(cd, cr, ad, dtype, a);
  if (s != FBEV_OK) return s;
  *bytes = a.c.B == 0 || a.c.T == 0 ? 0 : fbev::cache_attention_workspace_bytes(a);
  return FBEV_OK;
}

fbev_status fbev_cache_attention(const fbev_cache_desc* cd, const fbev_cache_rows* cr,
                                 const fbev_cache_attention_desc* ad, const void* q, fbev_dtype dtype, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  fbev::CacheAttnArgs a{};
  fbev_status s = check_cache_attention(cd, cr, ad, dtype, a);
  if (s != FBEV_OK) return s;
  if (a.c.B == 0 || a.c.T == 0) return FBEV_OK;
  if (q == nullptr || out == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "q and out must be non-NULL");
  if (a.mode == FBEV_DRAFT_TREE && a.ancestors == nullptr)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "a tree needs its ancestors");
  s = check_workspace(workspace, workspace_bytes, fbev::cache_attention_workspace_bytes(a));
  if (s != FBEV_OK) return s;
  a.q = q;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  return device_status(fbev::launch_cache_attention(a, static_cast<hipStream_t>(stream)),
                       "fbev_cache_attention launch");
}

}  // extern "C"
