// abi_common.h -- what the host files of the C ABI share: the calling thread's error text and the
// device check.  Defined in abi.cpp.
#pragma once

#include <hip/hip_runtime.h>

namespace qmoe {

int abi_fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));  // returns code
int abi_ok();                                      // clears the error text, returns MOE_OK
int abi_check_device();                            // MOE_OK on gfx950
int abi_hip_status(hipError_t e, const char *what);

}  // namespace qmoe
