// Drives the encoder operators' host layer (encoder_api.cpp) through valid, invalid and extreme arguments under
// AddressSanitizer and UndefinedBehaviorSanitizer, with host-only launcher stand-ins.  Nothing touches a GPU.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../camera_bev_view_amd/csrc/encoder.h"
#include "../../include/flashbev.h"

static int launches = 0;
static hipError_t status = hipSuccess;

namespace fbev {
size_t group_norm_workspace_bytes(const NormArgs& a, bool) { return (size_t)a.images * a.C * 8; }
hipError_t launch_group_norm_forward(const NormArgs&, hipStream_t) { return ++launches, status; }
hipError_t launch_group_norm_backward(const NormArgs&, hipStream_t) { return ++launches, status; }
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t) {
  if (a.vec < 1 || a.vec > 8) abort();
  return ++launches, status;
}
size_t attention_forward_workspace_bytes(const AttnArgs& a) { return (size_t)a.B * a.R; }
size_t attention_backward_workspace_bytes(const AttnArgs& a) { return (size_t)a.B * a.R; }
hipError_t launch_attention_forward(AttnArgs, hipStream_t) { return ++launches, status; }
hipError_t launch_attention_backward(AttnArgs, hipStream_t) { return ++launches, status; }
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
  const int64_t big = INT64_MAX;
  const int32_t ibig = INT32_MAX;
  size_t n = 0;

  for (int64_t images : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)1 << 31, big})
    for (int64_t pixels : {(int64_t)0, (int64_t)5, (int64_t)1 << 30, big})
      for (int32_t C : {-1, 0, 1, 6, 4096, ibig})
        for (int32_t groups : {-1, 0, 1, 3, ibig}) {
          const fbev_norm_desc nd = {images, pixels, big, big, C, groups, FBEV_ACT_GELU, 1e-5f};
          for (fbev_dtype t : {FBEV_DTYPE_F32, FBEV_DTYPE_BF16}) {
            fbev_group_norm_workspace(&nd, t, 0, &n);
            fbev_group_norm_workspace(&nd, t, 1, &n);
            fbev_group_norm_forward(p, t, &nd, f, f, p, f, p, 1 << 20, nullptr);
            fbev_group_norm_backward(p, p, t, &nd, f, f, f, p, f, f, p, 1 << 20, nullptr);
          }
        }
  const fbev_norm_desc ok = {2, 5, 60, 12, 12, 3, FBEV_ACT_SILU, 1e-5f};
  launches = 0;
  EXPECT(fbev_group_norm_forward(p, FBEV_DTYPE_F32, &ok, f, f, p, f, p, 1 << 20, nullptr) == FBEV_OK && launches == 1);
  status = hipErrorUnknown;
  EXPECT(fbev_group_norm_backward(p, p, FBEV_DTYPE_BF16, &ok, f, f, f, p, f, f, p, 1 << 20, nullptr) ==
         FBEV_ERR_DEVICE);
  status = hipSuccess;
  EXPECT(fbev_group_norm_forward(p, FBEV_DTYPE_F32, nullptr, f, f, p, f, p, 0, nullptr) == FBEV_ERR_INVALID_ARGUMENT);
  EXPECT(launches == 2);

  for (int32_t B : {-1, 0, 1, ibig})
    for (int32_t T : {0, 3, ibig})
      for (int32_t D : {0, 1, 7, 64, ibig})
        for (int32_t P : {-1, 0, 3, 32, ibig})
          for (int32_t h : {0, 2, ibig}) {
            const fbev_rotary_desc rd = {B, T, D, 2, P, h, h, 1, 0, {big, big, big}, {1, 2, 3}, {4, 5, 6}, {0, 0, 0}};
            fbev_rotary(p, p, FBEV_DTYPE_BF16, &rd, f, f, p, p, nullptr);
          }

  for (int32_t B : {-1, 0, 2, ibig})
    for (int32_t Tq : {0, 4, ibig})
      for (int32_t Tk : {0, 9, ibig})
        for (int32_t Hq : {0, 6, ibig})
          for (int32_t Hk : {0, 1, 3, ibig})
            for (int32_t D : {0, 1, 40, 128, ibig}) {
              const fbev_attention_desc ad = {B, Tq, Tk, Hq, Hk, D, {big, big, big}, {1, 2, 3}, {4, 5, 6}, 0.1f, 5.0f,
                                              2, 1, f, f, f, nullptr, nullptr, nullptr};
              fbev_attention_workspace(&ad, 0, &n);
              fbev_attention_workspace(&ad, 1, &n);
              fbev_attention_forward(p, p, p, FBEV_DTYPE_F32, &ad, p, f, p, 1 << 20, nullptr);
              fbev_attention_backward(p, p, p, p, FBEV_DTYPE_BF16, &ad, p, f, p, p, p, f, p, 1 << 20, nullptr);
            }
  launches = 0;
  const fbev_attention_desc ad = {1, 3, 5, 4, 2, 16, {192, 64, 16}, {160, 32, 16}, {160, 32, 16}, 0.25f, 0.0f,
                                  0, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  EXPECT(fbev_attention_forward(p, p, p, FBEV_DTYPE_F32, &ad, p, f, p, 64, nullptr) == FBEV_OK && launches == 1);
  EXPECT(fbev_attention_backward(p, p, p, p, FBEV_DTYPE_F32, &ad, p, f, p, p, p, nullptr, p, 64, nullptr) == FBEV_OK);
  EXPECT(fbev_attention_forward(p, p, p, FBEV_DTYPE_F32, &ad, p, f, nullptr, 0, nullptr) == FBEV_ERR_INVALID_ARGUMENT);
  EXPECT(launches == 2);
  printf("ok\n");
  return 0;
}
