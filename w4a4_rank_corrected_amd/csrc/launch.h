// Kernel launch with the scratch check, shared by the launchers (host code of
// the HIP sources).
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>
#include <unordered_map>

#include "internal.h"

namespace svdq {
namespace {

// A GEMM kernel that uses scratch memory (register spills) is refused before
// its first launch: spills cost bandwidth, and a spill around a divergent
// region once produced wrong results in a GEMM build.  The build checks the
// same; this guards a library rebuilt with another compiler.  Queried once per
// kernel and process.
int scratch_free(const void* kernel) {
  static std::mutex mu;
  static std::unordered_map<const void*, int> seen;
  std::lock_guard<std::mutex> lock(mu);
  const auto it = seen.find(kernel);
  if (it != seen.end()) return it->second;
  hipFuncAttributes attr{};
  const hipError_t e = hipFuncGetAttributes(&attr, kernel);
  const int status = e != hipSuccess ? (int)e : (attr.localSizeBytes != 0 ? kErrKernelScratch : 0);
  seen[kernel] = status;
  return status;
}

template <class K, class... Args>
int launch_checked(K kernel, long long grid, int threads, hipStream_t st, Args... args) {
  if (!launch_fits(grid, threads)) return (int)hipErrorInvalidConfiguration;
  const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
  if (ok != 0) return ok;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), 0, st, args...);
  return (int)hipGetLastError();
}

}  // namespace
}  // namespace svdq
