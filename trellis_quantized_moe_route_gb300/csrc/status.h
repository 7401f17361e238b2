// Error reporting shared by the entry points outside api.cu.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "../../include/trellis_moe.h"
#include "launch.h"

namespace tmoe {

inline tm_status status_fail(tm_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

inline tm_status status_cuda(cudaError_t e, const char* what) {
  return status_fail(TM_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool dtype_ok(int32_t d) { return d == TM_F32 || d == TM_BF16 || d == TM_F16; }
inline int dtype_bytes(int32_t d) { return d == TM_F32 ? 4 : 2; }

}  // namespace tmoe
