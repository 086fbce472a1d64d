// Workspaces of the products and layers with an epilogue, with stubs for the
// launchers: a call that got through every check ends in the stub
// (SVDQ_ERR_HIP).  Each call is made with exactly the bytes that its size
// function names (it gets through) and with one byte less (it is refused);
// sizes of 0 go with no workspace at all.  "epi workspace ok" at the end.
#include <cstdint>
#include <cstdio>

#include "svdq.h"

static int g_bad = 0;
static void expect(bool ok, const char* what, int b, int n, int m, int rank) {
  if (ok) return;
  std::printf("FAIL: %s, b=%d n=%d m=%d rank=%d: %s\n", what, b, n, m, rank, svdq_last_error());
  ++g_bad;
}

int main() {
  uint16_t* u16 = reinterpret_cast<uint16_t*>(1 << 12);
  uint8_t* u8 = reinterpret_cast<uint8_t*>(1 << 12);
  float* f32 = reinterpret_cast<float*>(1 << 12);
  void *y = reinterpret_cast<void*>(1 << 12), *ws = reinterpret_cast<void*>(1 << 20);
  const int bs[] = {1, 16, 17, 64, 65, 128, 500, 4608}, ns[] = {1, 130, 1152, 8192}, ms[] = {64, 1152, 4608, 8192},
            ranks[] = {0, 16, 256};
  for (int b : bs)
    for (int n : ns)
      for (int m : ms)
        for (int rank : ranks) {
          const svdq_layer L4{m, n, rank, 64, nullptr, u8, u16, u16, u16, nullptr};
          const svdq_w8a8_layer L8{m, n, rank, nullptr, reinterpret_cast<int8_t*>(u8), u16, u16, u16, nullptr};
          const svdq_fp4_layer Lf{m, n, rank, 1.0f, 1.0f, nullptr, u8, u8, u16, u16, nullptr};
          auto check = [&](const char* what, size_t need, bool none, auto&& call) {
            expect(call(need ? ws : nullptr, need) == SVDQ_ERR_HIP, what, b, n, m, rank);
            if (need) {
              expect(call(ws, need - 1) == SVDQ_ERR_WORKSPACE, what, b, n, m, rank);
              expect(call(nullptr, need) == SVDQ_ERR_WORKSPACE, what, b, n, m, rank);
            }
            if (none) expect(need == 0, what, b, n, m, rank);
          };
          const bool few = b <= 64;
          const size_t g = svdq_gemm_epi_workspace_size(b, n, m);
          check("INT4 product", g, few, [&](void* w, size_t s) {
            return svdq_gemm_w4a4_lowrank_up_epi(u8, u16, f32, &L4, nullptr, b, y, 0, w, s, nullptr);
          });
          check("NVFP4 product", g, few, [&](void* w, size_t s) {
            return svdq_fp4_gemm_lowrank_up_epi(u8, u8, f32, &Lf, nullptr, b, y, 0, w, s, nullptr);
          });
          check("8-bit product", svdq_w8a8_gemm_workspace_size(b, n, m), false, [&](void* w, size_t s) {
            return svdq_w8a8_gemm_lowrank_up_epi(reinterpret_cast<int8_t*>(u8), u16, f32, &L8, nullptr, b, y, 0, w, s, nullptr);
          });
          check("INT4 layer", svdq_linear_epi_workspace_size(b, m, n, rank), false, [&](void* w, size_t s) {
            return svdq_linear_epi(u16, &L4, nullptr, b, y, 0, w, s, nullptr);
          });
          check("NVFP4 layer", svdq_fp4_linear_epi_workspace_size(b, m, n, rank), false, [&](void* w, size_t s) {
            return svdq_fp4_linear_epi(u16, &Lf, nullptr, b, y, 0, w, s, nullptr);
          });
          check("8-bit layer", svdq_w8a8_linear_workspace_size(b, m, n, rank), false, [&](void* w, size_t s) {
            return svdq_w8a8_linear_epi(u16, &L8, nullptr, b, y, 0, w, s, nullptr);
          });
          // few rows: no more than codes, scales, Z and its partial sums (at most 64 of them)
          const size_t most = (size_t)b * (m / 2 + m / 16 + 65 * 4 * (size_t)rank) + 8 * 256;
          expect(!few || svdq_linear_epi_workspace_size(b, m, n, rank) <= most, "INT4 layer's size", b, n, m, rank);
          expect(!few || svdq_fp4_linear_epi_workspace_size(b, m, n, rank) <= most, "NVFP4 layer's size", b, n, m, rank);
          expect(svdq_linear_epi_workspace_size(b, m, n, rank) <= svdq_linear_workspace_size(b, m, n, rank, 64) &&
                     svdq_fp4_linear_epi_workspace_size(b, m, n, rank) <= svdq_fp4_linear_workspace_size(b, m, n, rank),
                 "the plain layer's workspace serves too", b, n, m, rank);
        }
  expect(svdq_linear_epi_workspace_size(0, 64, 1, 0) == 0 && svdq_linear_epi_workspace_size(1, 63, 1, 0) == 0 &&
             svdq_fp4_linear_epi_workspace_size(1, 64, 0, 0) == 0 && svdq_fp4_linear_epi_workspace_size(1, 64, 1, 257) == 0,
         "sizes of no layer", 0, 0, 0, 0);
  if (g_bad) return 1;
  std::printf("epi workspace ok\n");
  return 0;
}
