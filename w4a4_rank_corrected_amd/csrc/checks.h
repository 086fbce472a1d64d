// Argument checks and workspace layouts shared by the C-ABI sources (defined in
// api.cpp).  A check returns an svdq_status and sets the thread's message.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace svdq {

constexpr size_t kAlign = 256;
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define REQUIRE(cond, code, ...)  \
  do {                            \
    if (!(cond)) {                \
      set_error(__VA_ARGS__);     \
      return (code);              \
    }                             \
  } while (0)

struct LinearWorkspace {
  size_t qx_off, as_off, z_off, zpart_off, gemm_off, total;
};

int check_group(int m, int group);
int check_layer(const svdq_layer* L);
int check_layer8(const svdq_w8a8_layer* L);
int check_layer_fp4(const svdq_fp4_layer* L);
int check_y(void* y, int y_dtype, int b);
int check_linear(const uint16_t* x, const svdq_layer* layer, int b, void* y, int y_dtype, bool* done);
int hip_status(int err, const char* what);

size_t gemm_ws_bytes(int b, int n, int m);
LinearWorkspace linear_ws_layout(int b, int m, int n, int rank);
LinearWorkspace linear8_ws_layout(int b, int m, int n, int rank);
LinearWorkspace linear_fp4_ws_layout(int b, int m, int n, int rank);
int run_act8(const uint16_t* x, int b, int m, int rank, const float* smooth_inv, const uint16_t* l1, int8_t* qx,
             uint16_t* ascale, float* z, float* zpart, void* stream);
int run_act_fp4(const uint16_t* x, int b, int m, int rank, const float* smooth_inv, const uint16_t* l1, float t_x,
                uint8_t* qx, uint8_t* ascale, float* z, float* zpart, void* stream);

}  // namespace svdq
