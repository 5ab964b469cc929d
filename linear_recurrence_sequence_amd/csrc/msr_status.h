// Status returns shared by the C entry points (internal): each sets the
// calling thread's msr_last_error().
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/msr.h"

namespace msr {

msr_status fail(msr_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
msr_status ok();
msr_status from_hip(hipError_t e, const char* where);

}  // namespace msr
