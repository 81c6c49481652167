// Drives the decoder operators' host layer (decoder_api.cpp) through valid, invalid and extreme arguments under
// AddressSanitizer and UndefinedBehaviorSanitizer, with host-only launcher stand-ins.  Nothing touches a GPU.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../camera_bev_view_amd/csrc/decoder.h"
#include "../../include/flashbev.h"

static int launches = 0;
static hipError_t status = hipSuccess;

namespace fbev {
static hipError_t norm(const RmsArgs& a) {
  if (a.rows < 0 || a.C < 1 || a.C > FBEV_MAX_RMS_CHANNELS || (a.codes >= 0 && (a.block < 1 || a.block > a.C))) abort();
  return ++launches, status;
}
static hipError_t cache(const CacheArgs& c) {
  if (c.D < 1 || c.D > 128 || c.Dp < c.D || c.Dp % 16 || c.B < 1 || c.T < 1 || c.W < 0 || c.W > 1 << 24) abort();
  return ++launches, status;
}
size_t rms_norm_workspace_bytes(const RmsArgs& a) { return a.rows ? (size_t)a.C * 1024 : 0; }
hipError_t launch_rms_norm_forward(const RmsArgs& a, hipStream_t) { return norm(a); }
hipError_t launch_rms_norm_backward(const RmsArgs& a, hipStream_t) { return norm(a); }
hipError_t launch_cache_write(const CacheMoveArgs& a, hipStream_t) { return cache(a.c); }
hipError_t launch_cache_read(const CacheMoveArgs& a, hipStream_t) { return cache(a.c); }
size_t cache_attention_workspace_bytes(const CacheAttnArgs& a) { return (size_t)a.c.B * a.R; }
hipError_t launch_cache_attention(CacheAttnArgs a, hipStream_t) {
  if (a.G < 1 || (int64_t)a.c.T * a.G != a.R) abort();
  return cache(a.c);
}
}  // namespace fbev

#define EXPECT(c)                                            \
  do {                                                       \
    if (!(c)) {                                              \
      printf("%s:%d: %s\n", __FILE__, __LINE__, #c);         \
      return 1;                                              \
    }                                                        \
  } while (0)

int main() {
  void* p = reinterpret_cast<void*>(0x10000);
  float* f = static_cast<float*>(p);
  const int32_t* t = static_cast<const int32_t*>(p);
  const int64_t big = INT64_MAX;
  const int32_t ibig = INT32_MAX;
  size_t n = 0;

  for (int64_t outer : {(int64_t)-1, (int64_t)0, (int64_t)3, (int64_t)1 << 31, big})
    for (int64_t inner : {(int64_t)0, (int64_t)1, (int64_t)8, big})
      for (int64_t stride : {(int64_t)-1, (int64_t)0, (int64_t)7, big})
        for (int32_t C : {-1, 0, 1, 33, FBEV_MAX_RMS_CHANNELS, ibig}) {
          const fbev_rms_desc rd = {outer, inner, {stride, 7}, {7, stride}, C, 1e-6f};
          for (fbev_dtype d : {FBEV_DTYPE_F32, FBEV_DTYPE_BF16}) {
            fbev_rms_norm_workspace(&rd, d, &n);
            fbev_rms_norm_forward(p, p, d, &rd, f, p, p, f, nullptr);
            for (int32_t block : {-1, 0, 32, 100, ibig})
              fbev_rms_norm_codes(p, nullptr, d, &rd, f, FBEV_CODES_E4M3, block, p, f, nullptr, nullptr);
            fbev_rms_norm_backward(p, p, p, d, &rd, f, f, p, f, p, 1 << 20, nullptr);
          }
        }
  const fbev_rms_desc ok = {4, 2, {66, 33}, {0, 0}, 33, 1e-6f};
  launches = 0;
  EXPECT(fbev_rms_norm_forward(p, nullptr, FBEV_DTYPE_F32, &ok, f, p, nullptr, f, nullptr) == FBEV_OK);
  status = hipErrorUnknown;
  EXPECT(fbev_rms_norm_backward(p, p, p, FBEV_DTYPE_BF16, &ok, f, f, p, f, p, 1 << 20, nullptr) == FBEV_ERR_DEVICE);
  status = hipSuccess;
  EXPECT(launches == 2);

  for (int32_t pages : {-1, 0, 4, ibig})
    for (int32_t Hk : {0, 2, ibig})
      for (int32_t D : {0, 1, 40, 128, ibig})
        for (int32_t B : {-1, 0, 3, ibig})
          for (int32_t T : {0, 1, 70, ibig})
            for (int32_t W : {0, 9, 1 << 24, ibig}) {
              const fbev_cache_desc cd = {pages, Hk, D, FBEV_CODES_INT8, p, p, f, f};
              const fbev_cache_rows cr = {B, T, W, t, t, t};
              const int64_t s[3] = {big, 2, 3};
              fbev_cache_write(&cd, &cr, p, p, FBEV_DTYPE_BF16, s, s, nullptr);
              fbev_cache_read(&cd, &cr, FBEV_DTYPE_F32, p, p, nullptr);
              for (int32_t Hq : {0, 4, ibig})
                for (int32_t drafts : {FBEV_DRAFT_NONE, FBEV_DRAFT_TREE}) {
                  const fbev_cache_attention_desc ad = {Hq, drafts, 2, {big, 1, 1}, static_cast<const uint64_t*>(p), 0.1f, 3.0f};
                  fbev_cache_attention_workspace(&cd, &cr, &ad, FBEV_DTYPE_F32, &n);
                  fbev_cache_attention(&cd, &cr, &ad, p, FBEV_DTYPE_BF16, p, p, (size_t)1 << 40, nullptr);
                }
            }
  const fbev_cache_desc cd = {4, 2, 40, FBEV_CODES_E4M3, p, p, f, f};
  const fbev_cache_rows cr = {3, 5, 2, t, t, nullptr};
  const fbev_cache_attention_desc ad = {4, FBEV_DRAFT_CHAIN, 0, {800, 160, 40}, nullptr, 0.1f, 0.0f};
  const int64_t s[3] = {400, 80, 40};
  launches = 0;
  EXPECT(fbev_cache_write(&cd, &cr, p, p, FBEV_DTYPE_F32, s, s, nullptr) == FBEV_OK);
  EXPECT(fbev_cache_attention(&cd, &cr, &ad, p, FBEV_DTYPE_F32, p, p, 1 << 20, nullptr) == FBEV_OK);
  EXPECT(fbev_cache_attention(&cd, &cr, &ad, p, FBEV_DTYPE_F32, p, p, 8, nullptr) == FBEV_ERR_INVALID_ARGUMENT);
  EXPECT(launches == 2);
  printf("ok\n");
  return 0;
}
