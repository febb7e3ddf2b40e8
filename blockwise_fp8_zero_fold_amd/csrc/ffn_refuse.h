// How the feed-forward and norm calls refuse: a status and its text, never an exception (a C caller
// cannot catch one).  Without host memory for the text the status stands, with a shorter text that a
// string holds in itself.
#pragma once

#include <hip/hip_runtime.h>

#include "internal.h"

namespace fp8z1 {

inline int refuse(int status, const char* what, const char* msg) noexcept {
  try {
    return set_error(status, std::string(what) + ": " + msg);
  } catch (...) {
    return set_error(status, "no host memory");
  }
}

// The status of the launches just made.
inline int launched(const char* what) noexcept {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? FP8Z1_OK : refuse(FP8Z1_EHIP, what, hipGetErrorString(e));
}

}  // namespace fp8z1
