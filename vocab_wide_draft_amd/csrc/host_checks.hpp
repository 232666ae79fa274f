// Host-side helpers of the C ABI shared by its source files: they set the
// message of dspark_last_error() (one per host thread) and return the code.
#pragma once
#include "dspark.h"

namespace dspark {
__attribute__((visibility("hidden"))) int host_fail(int code, const char* msg);
__attribute__((visibility("hidden"))) int host_check_launch();
__attribute__((visibility("hidden"))) int host_check_rows(const dspark_rows* r, const char* what);
}  // namespace dspark
