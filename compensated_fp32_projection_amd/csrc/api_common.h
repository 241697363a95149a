// What the C-ABI files share (defined in api.hip): the per-device
// architecture check and the calling thread's last HIP error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/cfp32.h"

namespace cfp32 {

// Every dimension and every extent stays below 2^48 elements, so size
// products formed on the host cannot overflow 64 bits.
constexpr int64_t kApiMaxDim = ((int64_t)1 << 48) - 1;

cfp32_status api_check_device();
cfp32_status api_launched(hipError_t e);

}  // namespace cfp32
