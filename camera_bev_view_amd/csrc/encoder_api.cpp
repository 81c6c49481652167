// C-ABI host layer of the encoder operators (group norm with an activation, rotary positions, attention):
// argument validation and the choice of lane widths.  Every check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/flashbev.h"
#include "encoder.h"
#include "host_status.h"

namespace {

using fbev::fail;
using fbev::gcd;

fbev_status device_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return FBEV_OK;
  return fail(FBEV_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

bool known(fbev_dtype dtype) { return dtype == FBEV_DTYPE_F32 || dtype == FBEV_DTYPE_BF16; }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fbev_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && (workspace == nullptr || have < need))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "workspace of %zu bytes given, %zu needed", workspace ? have : 0, need);
  if (!aligned(workspace, 16)) return fail(FBEV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  return FBEV_OK;
}

// ---- group norm

fbev_status check_norm(const fbev_norm_desc* nd, fbev_dtype dtype, fbev::NormArgs& a) {
  if (nd == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the norm descriptor is NULL");
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (nd->images < 0 || nd->pixels < 0 || nd->C < 1 || nd->groups < 1 || nd->C % nd->groups != 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT,
                "images=%lld and pixels=%lld must not be negative, C=%d must be a multiple of groups=%d >= 1",
                (long long)nd->images, (long long)nd->pixels, nd->C, nd->groups);
  if (nd->activation < FBEV_ACT_NONE || nd->activation > FBEV_ACT_GELU)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "unknown activation %d", nd->activation);
  if (!std::isfinite(nd->eps) || nd->eps < 0.0f)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  if (nd->image_stride < 0 || nd->pixel_stride < 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
  if (nd->images >= (int64_t)1 << 31 || nd->pixels >= (int64_t)1 << 31 ||
      nd->images * nd->pixels >= ((int64_t)1 << 40) / nd->C)
    return fail(FBEV_ERR_UNSUPPORTED, "%lld images of %lld pixels of %d channels: above 2^40 elements",
                (long long)nd->images, (long long)nd->pixels, nd->C);
  a.images = (int)nd->images;
  a.pixels = (int)nd->pixels;
  a.x_image = nd->image_stride;
  a.x_pixel = nd->pixel_stride;
  a.C = nd->C;
  a.groups = nd->groups;
  a.act = nd->activation;
  a.eps = nd->eps;
  a.elem_bytes = dtype == FBEV_DTYPE_F32 ? 4 : 2;
  return FBEV_OK;
}

// The widest piece of 16, 8 or 4 bytes that divides the rows and suits every address.
fbev_status pick_norm_width(fbev::NormArgs& a, const void* x, const void* y, const void* z) {
  a.vec = 1;
  for (int bytes = 16; bytes >= 4; bytes /= 2) {
    const int v = bytes / a.elem_bytes;
    if (v > 1 && a.C % v == 0 && (a.images <= 1 || a.x_image % v == 0) && (a.pixels <= 1 || a.x_pixel % v == 0) &&
        aligned(x, bytes) && aligned(y, bytes) && aligned(z, bytes)) {
      a.vec = v;
      break;
    }
  }
  const int cg = a.C / a.groups;
  if (cg / gcd(cg, a.vec) > 1024)
    return fail(FBEV_ERR_UNSUPPORTED, "groups of %d channels moved %d at a time: more than 1024 pieces", cg, a.vec);
  // workgroups hold at least six pixels of a group: their numbers stay within 32 bits
  const size_t blocks = (size_t)a.images * a.groups * ((size_t)a.pixels / 8 + 1);
  if (blocks >= (size_t)1 << 31)
    return fail(FBEV_ERR_UNSUPPORTED, "%d images of %d pixels in %d groups: too many", a.images, a.pixels, a.groups);
  return FBEV_OK;
}

// ---- rotary

fbev_status check_rotary(const fbev_rotary_desc* rd, fbev_dtype dtype, fbev::RotaryArgs& a) {
  if (rd == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the rotary descriptor is NULL");
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (rd->B < 0 || rd->T < 0 || rd->q_heads < 0 || rd->k_heads < 0 || rd->D < 1)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "negative size (B=%d T=%d heads %d, %d D=%d)", rd->B, rd->T, rd->q_heads,
                rd->k_heads, rd->D);
  if (rd->axes < 1 || rd->axes > 8) return fail(FBEV_ERR_INVALID_ARGUMENT, "axes=%d outside [1, 8]", rd->axes);
  if (rd->pairs < 1 || rd->pairs > rd->D / 2)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "pairs=%d outside [1, D / 2 = %d]", rd->pairs, rd->D / 2);
  if (rd->pairs > FBEV_MAX_ROTARY_PAIRS)
    return fail(FBEV_ERR_UNSUPPORTED, "pairs=%d exceeds FBEV_MAX_ROTARY_PAIRS=%d", rd->pairs, FBEV_MAX_ROTARY_PAIRS);
  for (int i = 0; i < 3; ++i)
    if (rd->q_stride[i] < 0 || rd->k_stride[i] < 0 || rd->q_out_stride[i] < 0 || rd->k_out_stride[i] < 0)
      return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
  if ((int64_t)rd->B * rd->T >= (int64_t)1 << 31 ||
      ((int64_t)rd->q_heads + rd->k_heads) * rd->D >= (int64_t)1 << 26)
    return fail(FBEV_ERR_UNSUPPORTED, "B*T = %lld tokens (limit 2^31 - 1) or %lld channels a token (limit 2^26 - 1)",
                (long long)rd->B * rd->T, ((long long)rd->q_heads + rd->k_heads) * rd->D);
  a.B = rd->B;
  a.T = rd->T;
  a.D = rd->D;
  a.A = rd->axes;
  a.P = rd->pairs;
  a.heads[0] = rd->q_heads;
  a.heads[1] = rd->k_heads;
  a.interleaved = rd->interleaved != 0;
  a.inverse = rd->inverse != 0;
  a.elem_bytes = dtype == FBEV_DTYPE_F32 ? 4 : 2;
  for (int i = 0; i < 3; ++i) {
    a.xs[0][i] = rd->q_stride[i];
    a.xs[1][i] = rd->k_stride[i];
    a.ys[0][i] = rd->q_out_stride[i];
    a.ys[1][i] = rd->k_out_stride[i];
  }
  return FBEV_OK;
}

void pick_rotary_width(fbev::RotaryArgs& a) {
  a.vec = 1;
  for (int bytes = 16; bytes >= 4; bytes /= 2) {
    const int v = bytes / a.elem_bytes;
    const int turned = a.interleaved ? 2 * a.P : a.P;
    if (v < 2 || turned % v != 0 || (a.D - 2 * a.P) % v != 0) continue;
    bool ok = true;
    for (int w = 0; w < 2; ++w) {
      if (a.heads[w] == 0) continue;
      ok = ok && aligned(a.x[w], bytes) && aligned(a.y[w], bytes);
      const int n[3] = {a.B, a.T, a.heads[w]};
      for (int i = 0; i < 3; ++i) ok = ok && (n[i] <= 1 || (a.xs[w][i] % v == 0 && a.ys[w][i] % v == 0));
    }
    if (ok) {
      a.vec = v;
      return;
    }
  }
}

// ---- attention

fbev_status check_attention(const fbev_attention_desc* ad, fbev::AttnArgs& a) {
  if (ad == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "the attention descriptor is NULL");
  if (ad->B < 0 || ad->Tq < 0 || ad->Tk < 0 || ad->Hq < 1 || ad->Hk < 1 || ad->D < 1)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "bad size (B=%d Tq=%d Tk=%d Hq=%d Hk=%d D=%d)", ad->B, ad->Tq, ad->Tk,
                ad->Hq, ad->Hk, ad->D);
  if (ad->Hq % ad->Hk != 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "Hq=%d is not a multiple of Hk=%d", ad->Hq, ad->Hk);
  if (ad->D > FBEV_MAX_HEAD_DIM)
    return fail(FBEV_ERR_UNSUPPORTED, "D=%d exceeds FBEV_MAX_HEAD_DIM=%d", ad->D, FBEV_MAX_HEAD_DIM);
  if (!std::isfinite(ad->scale) || !std::isfinite(ad->cap) || ad->cap < 0.0f)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "scale and cap must be finite, cap not negative");
  // slopes and exponents are divided by the one or the other: their quotients stay within fp32
  const auto far = [](float x) { return x != 0.0f && !(std::fabs(x) >= 1e-12f && std::fabs(x) <= 1e12f); };
  if (far(ad->scale) || far(ad->cap))
    return fail(FBEV_ERR_UNSUPPORTED, "scale=%g and cap=%g must be 0 or of a size within [1e-12, 1e12]", ad->scale,
                ad->cap);
  if (ad->dims < 0 || ad->dims > 3) return fail(FBEV_ERR_INVALID_ARGUMENT, "dims=%d outside [0, 3]", ad->dims);
  if ((ad->doc_q == nullptr) != (ad->doc_k == nullptr) && ad->B > 0 && ad->Tq > 0 && ad->Tk > 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "doc_q and doc_k come together");
  if (ad->prefix != nullptr && !ad->causal) return fail(FBEV_ERR_INVALID_ARGUMENT, "prefix needs causal");
  for (int i = 0; i < 3; ++i)
    if (ad->q_stride[i] < 0 || ad->k_stride[i] < 0 || ad->v_stride[i] < 0)
      return fail(FBEV_ERR_INVALID_ARGUMENT, "negative stride");
  const int64_t limit = (int64_t)1 << 30;
  const int64_t rows = (int64_t)ad->Tq * (ad->Hq / ad->Hk);
  if (rows >= limit || ad->Tk >= limit)
    return fail(FBEV_ERR_UNSUPPORTED, "Tq Hq / Hk = %lld rows or Tk = %d keys (limit 2^30 - 1)", (long long)rows,
                ad->Tk);
  const int64_t longest = (rows > ad->Tk ? rows : ad->Tk) / 32 + 1;
  // (heads of the whole batch) x (tiles of 32) blocks; splits come only where these are under 128
  if ((int64_t)ad->B * ad->Hk >= limit / longest || (int64_t)ad->B * ad->Hk * longest >= (int64_t)1 << 26)
    return fail(FBEV_ERR_UNSUPPORTED, "B Hk = %lld heads of %lld tiles of 32: above 2^26",
                (long long)ad->B * ad->Hk, (long long)longest);
  a.B = ad->B;
  a.Tq = ad->Tq;
  a.Tk = ad->Tk;
  a.Hq = ad->Hq;
  a.Hk = ad->Hk;
  a.G = ad->Hq / ad->Hk;
  a.D = ad->D;
  a.R = (int)rows;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = ad->q_stride[i];
    a.ks[i] = ad->k_stride[i];
    a.vs[i] = ad->v_stride[i];
  }
  a.scale = ad->scale;
  a.cap = ad->cap;
  a.dims = ad->dims;
  a.pos_q = ad->pos_q;
  a.pos_k = ad->pos_k;
  a.slope = ad->slope;
  a.doc_q = ad->doc_q;
  a.doc_k = ad->doc_q ? ad->doc_k : nullptr;
  a.causal = ad->causal != 0;
  a.prefix = ad->prefix;
  return FBEV_OK;
}

fbev_status check_attention_data(fbev::AttnArgs& a, const void* q, const void* k, const void* v, fbev_dtype dtype) {
  if (!known(dtype)) return fail(FBEV_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  const bool rows = a.B > 0 && a.R > 0, keys = a.B > 0 && a.Tk > 0;
  if (rows && q == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "q is NULL");
  if (keys && (k == nullptr || v == nullptr)) return fail(FBEV_ERR_INVALID_ARGUMENT, "k and v must be non-NULL");
  if (a.dims > 0 && ((rows && (a.pos_q == nullptr || a.slope == nullptr)) || (keys && a.pos_k == nullptr)))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "pos_q, pos_k and slope must be non-NULL with dims=%d", a.dims);
  a.q = q;
  a.k = k;
  a.v = v;
  a.elem_bytes = dtype == FBEV_DTYPE_F32 ? 4 : 2;
  const int e = 16 / a.elem_bytes;
  a.vec = a.D % e == 0 && aligned(q, 16) && aligned(k, 16) && aligned(v, 16);
  const int nq[3] = {a.B, a.Tq, a.Hq}, nk[3] = {a.B, a.Tk, a.Hk};
  // rows behind the last are told by their offset, so staged tokens have to lie a row apart: broadcast ones (stride 0) move
  // element by element
  const auto apart = [&](int tokens, int64_t& stride) {
    if (tokens <= 1) stride = a.D;
    return stride >= a.D;
  };
  a.vec = a.vec && (a.G > 1 || apart(a.Tq, a.qs[1])) && apart(a.Tk, a.ks[1]) && apart(a.Tk, a.vs[1]);
  // a staged tile (128 tokens, all heads of a group) is addressed with 31 bits
  const int64_t far = ((int64_t)1 << 30) / (128 * a.elem_bytes);
  a.vec = a.vec && a.qs[1] < far && a.ks[1] < far && a.vs[1] < far && a.qs[2] < far / a.G * 64;
  for (int i = 0; i < 3; ++i) {
    a.vec = a.vec && (nq[i] <= 1 || a.qs[i] % e == 0);
    a.vec = a.vec && (nk[i] <= 1 || (a.ks[i] % e == 0 && a.vs[i] % e == 0));
  }
  return FBEV_OK;
}

}  // namespace

extern "C" {

fbev_status fbev_group_norm_workspace(const fbev_norm_desc* nd, fbev_dtype dtype, int32_t backward, size_t* bytes) {
  if (bytes == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "bytes is NULL");
  fbev::NormArgs a{};
  fbev_status s = check_norm(nd, dtype, a);
  if (s != FBEV_OK) return s;
  *bytes = 0;
  if ((int64_t)a.images * a.pixels == 0) return FBEV_OK;
  // addresses may force narrower pieces: the size covers every width
  size_t need = 0;
  for (int v = 16 / a.elem_bytes; v >= 1; v /= 2) {
    const int cg = a.C / a.groups;
    if (a.C % v != 0 || cg / gcd(cg, v) > 1024) continue;
    a.vec = v;
    const size_t n = fbev::group_norm_workspace_bytes(a, backward != 0);
    if (n > need) need = n;
  }
  *bytes = need;
  return FBEV_OK;
}

fbev_status fbev_group_norm_forward(const void* x, fbev_dtype dtype, const fbev_norm_desc* nd, const float* weight,
                                    const float* bias, void* y, float* stats, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  fbev::NormArgs a{};
  fbev_status s = check_norm(nd, dtype, a);
  if (s != FBEV_OK) return s;
  if (a.images == 0) return FBEV_OK;
  if (stats == nullptr || (a.pixels > 0 && (x == nullptr || y == nullptr)))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "x, y and stats must be non-NULL");
  if (a.pixels > 0) {
    s = pick_norm_width(a, x, y, y);
    if (s != FBEV_OK) return s;
    s = check_workspace(workspace, workspace_bytes, fbev::group_norm_workspace_bytes(a, false));
    if (s != FBEV_OK) return s;
  }
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.stats = stats;
  a.part = static_cast<float*>(workspace);
  return device_status(fbev::launch_group_norm_forward(a, static_cast<hipStream_t>(stream)),
                       "fbev_group_norm_forward launch");
}

fbev_status fbev_group_norm_backward(const void* grad_y, const void* x, fbev_dtype dtype, const fbev_norm_desc* nd,
                                     const float* weight, const float* bias, const float* stats, void* grad_x,
                                     float* grad_weight, float* grad_bias, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  fbev::NormArgs a{};
  fbev_status s = check_norm(nd, dtype, a);
  if (s != FBEV_OK) return s;
  const bool empty = (int64_t)a.images * a.pixels == 0;
  if (empty && grad_weight == nullptr && grad_bias == nullptr) return FBEV_OK;
  if (!empty) {
    if (grad_y == nullptr || x == nullptr || stats == nullptr || grad_x == nullptr)
      return fail(FBEV_ERR_INVALID_ARGUMENT, "grad_y, x, stats and grad_x must be non-NULL");
    s = pick_norm_width(a, x, grad_y, grad_x);
    if (s != FBEV_OK) return s;
    s = check_workspace(workspace, workspace_bytes, fbev::group_norm_workspace_bytes(a, true));
    if (s != FBEV_OK) return s;
  }
  a.x = x;
  a.gy = grad_y;
  a.weight = weight;
  a.bias = bias;
  a.stats = const_cast<float*>(stats);
  a.gx = grad_x;
  a.gweight = grad_weight;
  a.gbias = grad_bias;
  a.part = static_cast<float*>(workspace);
  return device_status(fbev::launch_group_norm_backward(a, static_cast<hipStream_t>(stream)),
                       "fbev_group_norm_backward launch");
}

fbev_status fbev_rotary(const void* q, const void* k, fbev_dtype dtype, const fbev_rotary_desc* rd, const float* pos,
                        const float* freqs, void* q_out, void* k_out, void* stream) {
  fbev::RotaryArgs a{};
  const fbev_status s = check_rotary(rd, dtype, a);
  if (s != FBEV_OK) return s;
  if ((int64_t)a.B * a.T * (a.heads[0] + a.heads[1]) == 0) return FBEV_OK;
  if ((a.heads[0] > 0 && (q == nullptr || q_out == nullptr)) || (a.heads[1] > 0 && (k == nullptr || k_out == nullptr)))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "a tensor with heads is NULL");
  if (pos == nullptr || freqs == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "pos and freqs must be non-NULL");
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k_out;
  a.pos = pos;
  a.freqs = freqs;
  pick_rotary_width(a);
  return device_status(fbev::launch_rotary(a, static_cast<hipStream_t>(stream)), "fbev_rotary launch");
}

fbev_status fbev_attention_workspace(const fbev_attention_desc* ad, int32_t backward, size_t* bytes) {
  if (bytes == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "bytes is NULL");
  fbev::AttnArgs a{};
  const fbev_status s = check_attention(ad, a);
  if (s != FBEV_OK) return s;
  *bytes = 0;
  if ((int64_t)a.B * a.R == 0) return FBEV_OK;
  a.elem_bytes = 4;      // neither size depends on the type
  if (backward) {
    *bytes = fbev::attention_backward_workspace_bytes(a);
    return FBEV_OK;
  }
  *bytes = fbev::attention_forward_workspace_bytes(a);
  return FBEV_OK;
}

fbev_status fbev_attention_forward(const void* q, const void* k, const void* v, fbev_dtype dtype,
                                   const fbev_attention_desc* ad, void* out, float* stats, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  fbev::AttnArgs a{};
  fbev_status s = check_attention(ad, a);
  if (s == FBEV_OK) s = check_attention_data(a, q, k, v, dtype);
  if (s != FBEV_OK) return s;
  if ((int64_t)a.B * a.R == 0) return FBEV_OK;
  if (out == nullptr || stats == nullptr) return fail(FBEV_ERR_INVALID_ARGUMENT, "out and stats must be non-NULL");
  if (!aligned(stats, 8)) return fail(FBEV_ERR_INVALID_ARGUMENT, "stats must be 8-byte aligned");
  s = check_workspace(workspace, workspace_bytes, fbev::attention_forward_workspace_bytes(a));
  if (s != FBEV_OK) return s;
  a.out = out;
  a.stats = reinterpret_cast<float2*>(stats);
  a.part = static_cast<float*>(workspace);
  a.vec_out = a.D % 4 == 0 && aligned(out, 4 * a.elem_bytes);
  return device_status(fbev::launch_attention_forward(a, static_cast<hipStream_t>(stream)),
                       "fbev_attention_forward launch");
}

fbev_status fbev_attention_backward(const void* grad_out, const void* q, const void* k, const void* v,
                                    fbev_dtype dtype, const fbev_attention_desc* ad, const void* out,
                                    const float* stats, void* grad_q, void* grad_k, void* grad_v, float* grad_slope,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  fbev::AttnArgs a{};
  fbev_status s = check_attention(ad, a);
  if (s == FBEV_OK) s = check_attention_data(a, q, k, v, dtype);
  if (s != FBEV_OK) return s;
  const bool rows = (int64_t)a.B * a.R > 0, keys = (int64_t)a.B * a.Tk > 0;
  if (!rows && !keys) return FBEV_OK;
  if (rows && (grad_out == nullptr || out == nullptr || stats == nullptr || grad_q == nullptr))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "grad_out, out, stats and grad_q must be non-NULL");
  if (!aligned(stats, 8)) return fail(FBEV_ERR_INVALID_ARGUMENT, "stats must be 8-byte aligned");
  if (keys && (grad_k == nullptr || grad_v == nullptr))
    return fail(FBEV_ERR_INVALID_ARGUMENT, "grad_k and grad_v must be non-NULL");
  if (grad_slope != nullptr && a.dims == 0)
    return fail(FBEV_ERR_INVALID_ARGUMENT, "grad_slope without a distance bias (dims=0)");
  s = check_workspace(workspace, workspace_bytes, rows ? fbev::attention_backward_workspace_bytes(a) : 0);
  if (s != FBEV_OK) return s;
  a.vec = a.vec && (int64_t)a.Hq * a.D < ((int64_t)1 << 30) / (128 * a.elem_bytes) && aligned(out, 16) && aligned(grad_out, 16);
  a.vec_out = a.D % 4 == 0 && aligned(grad_q, 4 * a.elem_bytes) && aligned(grad_k, 4 * a.elem_bytes) &&
              aligned(grad_v, 4 * a.elem_bytes);
  a.gout = grad_out;
  a.out = const_cast<void*>(out);
  a.stats = reinterpret_cast<float2*>(const_cast<float*>(stats));
  a.gq = grad_q;
  a.gk = grad_k;
  a.gv = grad_v;
  a.gslope = grad_slope;
  a.delta = static_cast<float*>(workspace);
  return device_status(fbev::launch_attention_backward(a, static_cast<hipStream_t>(stream)),
                       "fbev_attention_backward launch");
}

}  // extern "C"
