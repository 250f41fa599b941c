// ew_host.h -- what the host API's files share: the current device, the
// record of a failed HIP call and the launch log (defined in ew_api.cpp).
// Not installed; not part of the C ABI.
#pragma once

#include "ew.h"

#include <hip/hip_runtime.h>

namespace ew {

// EW_OK and the current device's compute-unit count, or an error status.
ew_status_t host_device(int *cu_count);

// Keeps e for ew_last_hip_error() and returns EW_ERR_HIP.
ew_status_t host_fail(hipError_t e);

// Whether launches are logged (EW_LOG).
bool host_log_enabled();

}  // namespace ew
