// The plans and workspaces of the 8-bit floating-point setting and of the sort, for
// shapes from the smallest to the largest, under the sanitizers: what each kernel
// assumes of its plan, and what the C ABI asks for and accepts.
#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "internal.h"

using namespace svdq;

#define CHECK(cond)                                                                               \
  do {                                                                                            \
    if (!(cond)) {                                                                                \
      std::printf("line %d: %s (b=%d n=%d m=%d experts=%d)\n", __LINE__, #cond, b, n, m, experts); \
      std::exit(1);                                                                               \
    }                                                                                             \
  } while (0)

namespace {

void plan(int b, int n, int m, int experts, int dtype) {
  const Fp8Plan p = fp8_plan(b, n, m, experts, dtype);
  const long long G = fp8_blocks(m), grid = p.split.grid;
  const long long t128 = (experts ? grouped_row_blocks(b, experts, 128) : (b + 127LL) / 128) * ((n + 127LL) / 128);
  const long long t256 = (experts ? grouped_row_blocks(b, experts, 256) : (b + 255LL) / 256) * ((n + 255LL) / 256);
  CHECK(grid >= 1 && p.threads >= 64 && p.threads <= 1024);
  if (p.rb) {
    CHECK(p.rb == 1 || p.rb == 2 || p.rb == 4);
    CHECK(!p.big && !p.small && p.pieces == 1 && p.ws_bytes == 0);
    CHECK(p.threads == 64 * p.split.nwk * p.split.nwc && p.threads <= (p.rb == 4 ? 512 : 1024));
    CHECK(p.split.nwk * p.split.nwc * p.rb <= 32);  // KB of LDS, beside the codes of few blocks
    const long long blocks = experts ? grouped_row_blocks(b, experts, 16 * p.rb) : (b + 16LL * p.rb - 1) / (16 * p.rb);
    CHECK(grid == blocks * ((n + 16LL * p.split.nwc - 1) / (16 * p.split.nwc)));
  } else if (p.big) {
    CHECK(dtype == SVDQ_OUT_BF16 && !p.small && p.threads == 512 && p.ws_bytes == 0);
    if (experts) {
      CHECK(grid == t256);
    } else {
      CHECK(p.parts == 1 || p.parts == 2 || p.parts == 4);
      CHECK(p.full >= 1 && p.full <= t256 && grid == p.full + (t256 - p.full) * p.parts);
      CHECK(p.parts > 1 || p.full == t256);
    }
  } else if (p.small) {
    CHECK(!experts && p.threads == 256 && p.pieces == 1 && p.ws_bytes == 0);
    CHECK(grid == ((b + 63LL) / 64) * ((n + 127LL) / 128));
  } else {
    CHECK(p.threads == 256 && p.pieces >= 1 && p.pieces <= G && grid == t128 * p.pieces);
    CHECK(!experts || p.pieces == 1);
    CHECK(p.ws_bytes == (p.pieces > 1 ? (size_t)grid * 65536 : 0));
    // every piece has a channel block
    for (long long i = 0; i < p.pieces; ++i) CHECK(G * (i + 1) / p.pieces > G * i / p.pieces);
  }
}

}  // namespace

int main() {
  const int sizes[] = {1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 333, 512, 1000, 1152,
                       2047, 2048, 2049, 4096, 4608, 9216, 12288, 65536, 270000, 1 << 20, SVDQ_MAX_DIM};
  const int deep[] = {1, 127, 128, 129, 640, 1000, 1152, 2048, 4608, 8192, 16384, 1 << 20, SVDQ_MAX_DIM};
  for (int b : sizes)
    for (int n : sizes)
      for (int m : deep)
        for (int experts : {0, 1, 2, 8, 64, 1000, SVDQ_MAX_EXPERTS})
          for (int dtype : {SVDQ_OUT_BF16, SVDQ_OUT_F32}) {
            plan(b, n, m, experts, dtype);
            if (experts) continue;
            const size_t G = (size_t)fp8_blocks(m), need = svdq_fp8_gemm_workspace_size(b, n, m);
            CHECK(need >= fp8_plan(b, n, m, 0, dtype).ws_bytes && need <= ((size_t)1 << 31));
            CHECK(svdq_fp8_linear_workspace_size(b, m, n) >= G * b * 129 + need);
          }
  const int experts = 7, n = 0, m = 0;
  for (int b : sizes) {
    const SortPlan p = sort_plan(b);
    CHECK(p.chunk % kSortThreads == 0 && p.chunk >= kSortChunk && p.chunks <= 256);
    CHECK((long long)p.chunk * p.chunks >= b && (long long)p.chunk * (p.chunks - 1) < b);
    CHECK(svdq_sort_rows_workspace_size(b, 1, experts) == (p.chunks > 1 ? (size_t)p.chunks * 32 : 0));
  }
  // a call that is accepted reaches the launcher, and one with a short workspace does not
  static uint8_t memory[1 << 16];
  uint8_t* at = memory + (256 - (uintptr_t)memory % 256);
  svdq_fp8_layer layer{200, 300, at, at, nullptr};
  const int b = 100;
  const size_t need = svdq_fp8_linear_workspace_size(b, 200, 300);
  CHECK(svdq_fp8_linear((uint16_t*)at, &layer, nullptr, b, at, 0, at, need, nullptr) == SVDQ_ERR_HIP);
  CHECK(svdq_fp8_linear((uint16_t*)at, &layer, nullptr, b, at, 0, at, need - 1, nullptr) == SVDQ_ERR_WORKSPACE);
  CHECK(svdq_sort_rows((int32_t*)at, 3, 2, 4, (int32_t*)(at + 64), (int32_t*)(at + 128), (int32_t*)(at + 256), nullptr, 0,
                       nullptr) == SVDQ_ERR_HIP);
  std::printf("fp8 plans ok\n");
  return 0;
}
