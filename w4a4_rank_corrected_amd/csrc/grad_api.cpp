// C-ABI entry point of the gradient of the combination of rows (declared in
// include/svdq.h).  Arguments are validated on the host before any HIP call.
#include "route_checks.h"

using namespace svdq;

extern "C" {

int svdq_combine_rows_grad(const void* dy, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                           const void* rows, int R, void* drows, float* dweight, void* stream) {
  clear_error();
  int st = check_scatter(dy, t, n, dtype, index, weight, k, R);
  if (st || t == 0 || (!drows && !dweight)) return st;
  REQUIRE(!dweight || rows || R == 0, SVDQ_ERR_INVALID_ARG, "rows must not be NULL when dweight is wanted");
  REQUIRE(element_aligned(rows, dtype) && element_aligned(drows, dtype), SVDQ_ERR_ALIGNMENT,
          "rows and drows must be element-aligned");
  REQUIRE(((uintptr_t)dweight & 3u) == 0, SVDQ_ERR_ALIGNMENT, "dweight must be 4-byte aligned");
  const size_t row = (size_t)n * (dtype == SVDQ_OUT_F32 ? 4 : 2), slots = (size_t)t * k * 4, all = (size_t)R * row;
  const void* read = dweight ? rows : nullptr;
  st = check_apart({{drows, all, "drows"}, {dweight, slots, "dweight"}},
                   {{dy, (size_t)t * row, "dy"}, {index, slots, "index"}, {weight, slots, "weight"},
                    {read == drows ? nullptr : read, all, "rows"}});
  if (!st) st = check_apart({{dweight, slots, "dweight"}}, {{read, all, "rows"}});
  if (st || (R == 0 && !dweight)) return st;
  return hip_status(launch_combine_grad(dy, t, n, dtype, index, weight, k, rows, R, drows, dweight, stream),
                    "combine_rows_grad");
}

}  // extern "C"
