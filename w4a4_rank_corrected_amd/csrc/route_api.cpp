// C-ABI entry points of the routing of rows to experts (declared in
// include/svdq.h).  Arguments are validated on the host before any HIP call.
#include "route_checks.h"

using namespace svdq;

extern "C" {

size_t svdq_sort_rows_workspace_size(int t, int k, int experts) {
  if (t < 0 || k < 1 || k > SVDQ_MAX_EXPERTS || (long long)t * k > SVDQ_MAX_DIM || experts < 1 ||
      experts > SVDQ_MAX_EXPERTS)
    return 0;
  const SortPlan p = sort_plan(t * k);
  return p.chunks > 1 ? (size_t)p.chunks * (size_t)(experts + 1) * 4 : 0;
}

int svdq_sort_rows(const int32_t* expert, int t, int k, int experts, int32_t* offsets, int32_t* row_index,
                   int32_t* index, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  int st = check_slots(t, k);
  if (st) return st;
  REQUIRE((long long)t * k <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "t k must be <= %d (got %d x %d)", SVDQ_MAX_DIM, t, k);
  REQUIRE(experts >= 1, SVDQ_ERR_INVALID_ARG, "experts must be >= 1 (got %d)", experts);
  REQUIRE(experts <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "experts must be <= %d (got %d)", SVDQ_MAX_EXPERTS, experts);
  const int b = t * k;
  REQUIRE(offsets && (b == 0 || (expert && row_index && index)), SVDQ_ERR_INVALID_ARG,
          "expert, offsets, row_index and index must not be NULL");
  REQUIRE((((uintptr_t)expert | (uintptr_t)offsets | (uintptr_t)row_index | (uintptr_t)index) & 3u) == 0,
          SVDQ_ERR_ALIGNMENT, "expert, offsets, row_index and index must be 4-byte aligned");
  const size_t need = svdq_sort_rows_workspace_size(t, k, experts), slots = (size_t)b * 4;
  st = check_workspace(workspace, workspace_bytes, need, 16);
  if (!st)
    st = check_apart({{offsets, (size_t)(experts + 1) * 4, "offsets"},
                      {row_index, slots, "row_index"},
                      {index, slots, "index"},
                      {need ? workspace : nullptr, need, "the workspace"}},
                     {{expert, slots, "expert"}});
  if (st) return st;
  return hip_status(launch_sort_rows(expert, b, k, experts, offsets, row_index, index, workspace, stream), "sort_rows");
}

int svdq_dispatch_rows(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k, int R,
                       void* rows, void* stream) {
  clear_error();
  int st = check_scatter(x, t, n, dtype, index, weight, k, R);
  if (st || t == 0 || R == 0) return st;
  REQUIRE(rows != nullptr, SVDQ_ERR_INVALID_ARG, "rows must not be NULL");
  REQUIRE(element_aligned(rows, dtype), SVDQ_ERR_ALIGNMENT, "rows must be element-aligned");
  const size_t row = (size_t)n * (dtype == SVDQ_OUT_F32 ? 4 : 2), slots = (size_t)t * k * 4;
  st = check_apart({{rows, (size_t)R * row, "rows"}},
                   {{x, (size_t)t * row, "x"}, {index, slots, "index"}, {weight, slots, "weight"}});
  if (st) return st;
  return hip_status(launch_scatter_rows(x, t, n, dtype, index, weight, k, nullptr, R, rows, nullptr, stream),
                    "dispatch_rows");
}

}  // extern "C"
