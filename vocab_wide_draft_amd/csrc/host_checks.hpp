// Host-side helpers of the C ABI shared by its source files: they set the
// message of dspark_last_error() (one per host thread) and return the code.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>

#include "dspark.h"

namespace dspark {
__attribute__((visibility("hidden"))) int host_fail(int code, const char* msg);
__attribute__((visibility("hidden"))) int host_check_launch();
__attribute__((visibility("hidden"))) int host_check_rows(const dspark_rows* r, const char* what);

inline int fail(int code, const char* msg) { return host_fail(code, msg); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// a grid of at least n workgroups in two dimensions (a launch takes fewer
// than 2^32 threads per dimension)
inline dim3 grid_of(int64_t n) {
  const int64_t x = std::min<int64_t>(n, 1 << 20);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}
}  // namespace dspark
