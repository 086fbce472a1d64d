// Drives the argument checks of the products with an epilogue, the grouped
// layers and the combination of rows over random and extreme arguments, in a
// build with the address and undefined-behaviour sanitizers and stubs for the
// launchers.  A call either is refused before the launch or reaches the stub
// (SVDQ_ERR_HIP); "epi sanitize ok" when every call did one of the two.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "svdq.h"

static uint64_t g_state = 0x9E3779B97F4A7C15ull;
static uint32_t rnd() {
  g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(g_state >> 33);
}
static int pick(std::initializer_list<int> v) { return v.begin()[rnd() % v.size()]; }
template <class T>
static T* address() {
  static const uintptr_t at[] = {0, 1 << 12, (1 << 12) + 2, (1 << 12) + 4, 1 << 20, 1 << 30, ~(uintptr_t)0 - 15};
  return reinterpret_cast<T*>(at[rnd() % 7]);
}

int main() {
  const int kMax = SVDQ_MAX_DIM;
  long reached = 0, refused = 0;
  for (int it = 0; it < 400000; ++it) {
    const int b = pick({0, 1, 2, 63, 64, 65, 4608, kMax, kMax + 1, -1, 2147483647});
    const int n = pick({1, 2, 64, 4608, kMax, kMax + 1, 0, -5, 2147483647});
    const int m = pick({64, 128, 4096, kMax, 100, 0, -64, kMax + 64});
    const int rank = pick({0, 1, 32, 256, 257, -1});
    const int dt = pick({0, 1, 1, 0, 2, -1});
    const svdq_epilogue e{pick({0, 1, 4, 5, -1}),        pick({0, 1, 64, -1, kMax, 2147483647}),
                          pick({0, 1, 7, -1, 2147483647}), pick({0, 64, 128, kMax, -1, 2147483647}),
                          pick({0, 64, 4608, kMax, -1, 2147483647}), address<const uint16_t>(), address<const void>()};
    const svdq_epilogue* epi = rnd() % 5 ? &e : nullptr;
    void *y = address<void>(), *ws = address<void>();
    const size_t wsb = rnd() % 2 ? ~(size_t)0 >> 1 : rnd();
    const svdq_layer L{m, n, rank, 64, address<const float>(), address<const uint8_t>(), address<const uint16_t>(),
                       address<const uint16_t>(), address<const uint16_t>(), address<const uint16_t>()};
    const svdq_w8a8_layer L8{m, n, rank, address<const float>(), address<const int8_t>(), address<const uint16_t>(),
                             address<const uint16_t>(), address<const uint16_t>(), address<const uint16_t>()};
    const svdq_fp4_layer L4{m, n, rank, 1.0f, rnd() % 4 ? 0.5f : 0.3f, address<const float>(), address<const uint8_t>(),
                            address<const uint8_t>(), address<const uint16_t>(), address<const uint16_t>(),
                            address<const uint16_t>()};
    const svdq_grouped_layer Lg{pick({1, 8, 1024, 1025, 0, -1}), m, n, rank, pick({64, 64, 64, 32}), address<const float>(),
                                address<const uint8_t>(), address<const uint16_t>(), address<const uint16_t>(),
                                address<const uint16_t>(), address<const uint16_t>()};
    int st = 0;
    switch (rnd() % 10) {
      case 0: st = svdq_gemm_w4a4_lowrank_up_epi(address<const uint8_t>(), address<const uint16_t>(), address<const float>(), &L, epi, b, y, dt, ws, wsb, nullptr); break;
      case 1: st = svdq_w8a8_gemm_lowrank_up_epi(address<const int8_t>(), address<const uint16_t>(), address<const float>(), &L8, epi, b, y, dt, ws, wsb, nullptr); break;
      case 2: st = svdq_fp4_gemm_lowrank_up_epi(address<const uint8_t>(), address<const uint8_t>(), address<const float>(), &L4, epi, b, y, dt, ws, wsb, nullptr); break;
      case 3: st = svdq_linear_epi(address<const uint16_t>(), &L, epi, b, y, dt, ws, wsb, nullptr); break;
      case 4: st = svdq_w8a8_linear_epi(address<const uint16_t>(), &L8, epi, b, y, dt, ws, wsb, nullptr); break;
      case 5: st = svdq_fp4_linear_epi(address<const uint16_t>(), &L4, epi, b, y, dt, ws, wsb, nullptr); break;
      case 6: st = svdq_grouped_quantize_act_lowrank_down(address<const uint16_t>(), pick({0, 1, 4608, kMax, kMax + 1, -1}), address<const int32_t>(), address<const int32_t>(), &Lg, b, address<uint8_t>(), address<uint16_t>(), address<float>(), nullptr); break;
      case 7: st = svdq_grouped_gemm_w4a4_lowrank_up(address<const uint8_t>(), address<const uint16_t>(), address<const float>(), address<const int32_t>(), &Lg, epi, b, y, dt, nullptr); break;
      case 8: st = svdq_grouped_linear(address<const uint16_t>(), pick({0, 1, 4608, kMax}), address<const int32_t>(), address<const int32_t>(), &Lg, rnd() % 2 ? epi : nullptr, b, y, dt, ws, wsb, nullptr); break;
      default: st = svdq_combine_rows(address<const void>(), pick({0, 1, 4608, kMax, -1, kMax + 1}), n, dt, address<const int32_t>(), address<const float>(), b, pick({1, 6, 1024, 1025, 0}), address<const void>(), y, nullptr); break;
    }
    if (st == SVDQ_ERR_HIP) ++reached;
    else if (st != SVDQ_OK) ++refused;
    if (st != SVDQ_OK && svdq_last_error()[0] == 0) { std::printf("FAIL: status %d without a message\n", st); return 1; }
    svdq_gemm_epi_workspace_size(b, n, m);
    svdq_grouped_linear_workspace_size(b, Lg.experts, m, n, rank);
  }
  std::printf("reached %ld, refused %ld\n", reached, refused);
  if (reached < 100 || refused < 1000) return 1;
  std::printf("epi sanitize ok\n");
  return 0;
}
