// Checks and error mapping shared by the files of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hisparse.h"

namespace hs {

inline int log2i(int64_t x) {
  int s = 0;
  while ((int64_t(1) << s) < x) ++s;
  return s;
}

// The kernels move 16-byte pieces: pools, outputs and layer strides are
// 16-byte aligned.
inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15) == 0; }

// Checks shared by every call that reads the pool layout.
hs_status check_layout(const hs_layout* lay);

// A launch's status: HS_ERR_LAUNCH, recorded for hs_last_error, unless it
// succeeded.
hs_status from_hip(hipError_t e, const char* what);

// A HIP runtime call other than a launch; a failure is recorded.
bool hip_ok(hipError_t e, const char* what);

}  // namespace hs
