// Host-only stand-ins for the launchers of the 8-bit floating-point setting and of
// the routing of rows (see device_stubs.cpp).
#include "internal.h"

namespace svdq {

namespace {
constexpr int kNoDevice = 100;  // hipErrorNoDevice
}

int launch_sort_rows(const int32_t*, int, int, int, int32_t*, int32_t*, int32_t*, void*, void*) { return kNoDevice; }
int launch_scatter_rows(const void*, int, int, int, const int32_t*, const float*, int, const void*, int, void*, float*,
                        void*) {
  return kNoDevice;
}
int launch_fp8_act(const uint16_t*, int, int, uint8_t*, uint8_t*, void*) { return kNoDevice; }
int launch_fp8_weights(const void*, int, int, int, int, bool, uint8_t*, uint8_t*, void*) { return kNoDevice; }
int launch_fp8_rows_x(const Fp8Args&, const uint16_t*, int, const Fp8Plan&, int, void*) { return kNoDevice; }
int launch_fp8_gemm(const Fp8Args&, const Fp8Plan&, int, void*, void*) { return kNoDevice; }

}  // namespace svdq
