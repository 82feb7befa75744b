// What the C ABI's translation units share (defined in api.hip): the
// thread-local error text and the device's compute units.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/moe_rounds.h"

namespace moe {

// Sets the error text ("name: msg" with a name) and returns `s`.
moe_status_t api_fail(moe_status_t s, const char* msg, const char* name = nullptr);
moe_status_t api_hip_fail(hipError_t e, const char* where);
// Compute units of the current device.
moe_status_t api_num_cus(int* out);

}  // namespace moe
