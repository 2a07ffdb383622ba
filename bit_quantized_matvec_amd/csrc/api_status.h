// api_status.h -- a HIP call's result as a tq status, shared by the C-ABI files.
#pragma once
#include <hip/hip_runtime.h>

namespace tq {
// TQ_OK, or TQ_ERR_HIP with the error kept for tq_last_hip_error (tq_api.cpp).
int hip_status(hipError_t e);
}  // namespace tq
