// What the files holding C entry points share: the error message of the calling thread.
#pragma once

#include <hip/hip_runtime.h>

#include "sgt.h"

namespace sgt {

// Record the formatted message for sgt_last_error() and return `st`.
__attribute__((format(printf, 2, 3))) sgt_status fail(sgt_status st, const char* fmt, ...);

}  // namespace sgt

#define HIP_TRY(expr)                                                                                 \
  do {                                                                                                \
    hipError_t e_ = (expr);                                                                           \
    if (e_ != hipSuccess) return sgt::fail(SGT_EHIP, "%s: %s (%s:%d)", #expr, hipGetErrorString(e_), \
                                           __FILE__, __LINE__);                                       \
  } while (0)
