// Host-only stand-ins for the launchers of the products with an epilogue and of
// the grouped layers (see device_stubs.cpp).
#include "internal.h"

namespace svdq {

namespace {
constexpr int kNoDevice = 100;  // hipErrorNoDevice
}

int launch_gemm_epi(const uint8_t*, const uint16_t*, const float*, const svdq_layer&, int, int, const EpiArgs&, void*,
                    void*) {
  return kNoDevice;
}
int launch_gemm8_epi(const int8_t*, const uint16_t*, const float*, const svdq_w8a8_layer&, int, int, const EpiArgs&,
                     void*, void*) {
  return kNoDevice;
}
int launch_gemm_fp4_epi(const uint8_t*, const uint8_t*, const float*, const svdq_fp4_layer&, int, int, const EpiArgs&,
                        void*, void*) {
  return kNoDevice;
}
int launch_grouped_gemm(const uint8_t*, const uint16_t*, const float*, const svdq_grouped_layer&, const int32_t*, int,
                        int, const EpiArgs&, void*) {
  return kNoDevice;
}
int launch_grouped_act(const uint16_t*, int, const int32_t*, const int32_t*, const svdq_grouped_layer&, int, uint8_t*,
                       uint16_t*, float*, void*) {
  return kNoDevice;
}
int launch_combine(const void*, int, int, int, const int32_t*, const float*, int, int, const void*, void*, void*) {
  return kNoDevice;
}

}  // namespace svdq
