// Argument checks that the routing's entry points share.
#pragma once

#include <initializer_list>

#include "checks.h"
#include "internal.h"

namespace svdq {

struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};
inline bool apart(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return true;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  return pa + a.bytes <= pb || pb + b.bytes <= pa;
}
// Each output is apart from every input and every other output.
inline int check_apart(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (auto p = o + 1; p != outputs.end(); ++p)
      REQUIRE(apart(*o, *p), SVDQ_ERR_INVALID_ARG, "%s overlaps %s", o->name, p->name);
    for (const Range& i : inputs) REQUIRE(apart(*o, i), SVDQ_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
  }
  return SVDQ_OK;
}

inline int check_slots(int t, int k) {
  REQUIRE(t >= 0 && k >= 1, SVDQ_ERR_INVALID_ARG, "need t >= 0 and k >= 1 (got t=%d k=%d)", t, k);
  REQUIRE(k <= SVDQ_MAX_EXPERTS, SVDQ_ERR_UNSUPPORTED, "k must be <= %d (got %d)", SVDQ_MAX_EXPERTS, k);
  REQUIRE(t <= SVDQ_MAX_DIM, SVDQ_ERR_UNSUPPORTED, "t must be <= %d (got %d)", SVDQ_MAX_DIM, t);
  return SVDQ_OK;
}

// What svdq_dispatch_rows and svdq_combine_rows_grad share.
inline int check_scatter(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k, int R) {
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

}  // namespace svdq
