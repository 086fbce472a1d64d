// C-ABI entry points of the routing of rows to experts (declared in
// include/svdq.h).  Arguments are validated on the host before any HIP call.
#include <initializer_list>

#include "checks.h"
#include "internal.h"

using namespace svdq;

namespace {

struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};
bool apart(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return true;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  return pa + a.bytes <= pb || pb + b.bytes <= pa;
}
// Each output is apart from every input and every other output.
int check_apart(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (auto p = o + 1; p != outputs.end(); ++p)
      REQUIRE(apart(*o, *p), SVDQ_ERR_INVALID_ARG, "%s overlaps %s", o->name, p->name);
    for (const Range& i : inputs) REQUIRE(apart(*o, i), SVDQ_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
  }
  return SVDQ_OK;
}

int check_slots(int t, int k) {
  REQUIRE(t >= 0 && k >= 1, SVDQ_ERR_INVALID_ARG, "need t >= 0 and k >= 1 (got t=%d k=%d)", t, k);
  REQUIRE(k <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "k must be <= %d (got %d)", SVDQ_MAX_EXPERTS, k);
  REQUIRE(t <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "t must be <= %d (got %d)", SVDQ_MAX_DIM, t);
  return SVDQ_OK;
}

// What svdq_dispatch_rows and svdq_combine_rows_grad share.
int check_scatter(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k, int R) {
  int st = check_slots(t, k);
  if (st) return st;
  REQUIRE(n >= 1 && R >= 0, SVDQ_ERR_INVALID_ARG, "need n >= 1 and R >= 0 (got n=%d R=%d)", n, R);
  REQUIRE(n <= SVDQ_MAX_DIM && R <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "n and R must be <= %d", SVDQ_MAX_DIM);
  REQUIRE(dtype == SVDQ_OUT_BF16 || dtype == SVDQ_OUT_F32, SVDQ_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (t == 0) return SVDQ_OK;
  REQUIRE(x && index, SVDQ_ERR_INVALID_ARG, "the tokens' rows and index must not be NULL");
  REQUIRE(element_aligned(x, dtype), SVDQ_ERR_ALIGNMENT, "the tokens' rows must be element-aligned");
  REQUIRE((((uintptr_t)index | (uintptr_t)weight) & 3u) == 0, SVDQ_ERR_ALIGNMENT,
          "index and weight must be 4-byte aligned");
  return SVDQ_OK;
}

}  // namespace

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
  return hip_status(launch_scatter_rows(dy, t, n, dtype, index, weight, k, rows, R, drows, dweight, stream),
                    "combine_rows_grad");
}

}  // extern "C"
