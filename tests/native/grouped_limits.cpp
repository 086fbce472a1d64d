// The largest grouped products, with stubs for the launchers: a product whose
// launch has fewer than 2^32 threads gets through (SVDQ_ERR_HIP, the stub), a
// larger one is refused before anything is launched.  "grouped limits ok" at
// the end.
#include <cstdint>
#include <cstdio>

#include "internal.h"

int main() {
  uint16_t* u16 = reinterpret_cast<uint16_t*>(1 << 12);
  uint8_t* u8 = reinterpret_cast<uint8_t*>(1 << 12);
  float* f32 = reinterpret_cast<float*>(1 << 12);
  int32_t* i32 = reinterpret_cast<int32_t*>(1 << 12);
  void *y = reinterpret_cast<void*>(1 << 12), *ws = reinterpret_cast<void*>(1 << 20);
  const struct {
    int experts, b, n;
    bool fits;
  } cases[] = {
      {1024, 8192, 1 << 19, true},  {1024, 8192, 1 << 20, false},  // row kernel: 1472 row blocks, 64 columns a workgroup
      {1024, 1024, 1 << 20, false}, {1024, 1024, 1 << 19, true},   // one row an expert
      {1, 8, 1 << 22, true},        {64, 128, 1 << 22, true},     // 68 row blocks x 65536 x 256 threads
      {1024, 16384, 1 << 20, true}, {1024, 16384, 1 << 22, false},  // 64 x 128 tiles
      {8, 1 << 22, 9216, true},     {8, 1 << 22, 1 << 20, false},   // 128 x 128 tiles
      {1024, 1 << 22, 1 << 22, false},
  };
  int bad = 0;
  for (const auto& c : cases) {
    const svdq_grouped_layer L{c.experts, 64, c.n, 8, 64, nullptr, u8, u16, u16, u16, nullptr};
    const int want = c.fits ? SVDQ_ERR_HIP : SVDQ_ERR_UNSUPPORTED;
    const int st[] = {
        svdq_grouped_gemm_w4a4_lowrank_up(u8, u16, f32, i32, &L, nullptr, c.b, y, 0, nullptr),
        svdq_grouped_linear(u16, c.b, nullptr, i32, &L, nullptr, c.b, y, 0, ws, ~(size_t)0 >> 1, nullptr)};
    const svdq::GroupedPlan p = svdq::grouped_plan(c.b, c.n, 64, c.experts);
    const bool fits = p.grid * p.threads < 4294967296LL;
    if (st[0] != want || st[1] != want || fits != c.fits) {
      std::printf("FAIL: experts=%d b=%d n=%d: %d %d, %lld x %d\n", c.experts, c.b, c.n, st[0], st[1], p.grid, p.threads);
      ++bad;
    }
  }
  if (bad) return 1;
  std::printf("grouped limits ok\n");
  return 0;
}
