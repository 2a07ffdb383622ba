// batch.h -- launchers of what differs from row to row in a batch that shares
// its weights: experts, adapters, sampling (k_route.hip, k_experts_pq2.hip,
// k_adapter.hip, k_sample.hip).  Arguments are validated by batch_api.cpp
// before any launcher runs; what lies in device memory (experts, adapters,
// offsets) is checked where it is read.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tq.h"

namespace tq {

hipError_t launch_route(const tq_route_args& a, hipStream_t s);
hipError_t launch_expert_lists(const int32_t* ids, int64_t pairs, int experts, int32_t* order, int32_t* offsets, hipStream_t s);
hipError_t launch_gemm_experts_pq2(const tq_gemm_experts_args& a, hipStream_t s);

int64_t adapter_workspace_bytes(int64_t tokens, int adapters, int rank, int64_t cols);
hipError_t launch_adapter_add(const tq_adapter_add_args& a, hipStream_t s);

int64_t sample_workspace_bytes(int64_t rows, int64_t vocab);
hipError_t launch_sample(const tq_sample_args& a, hipStream_t s);

}  // namespace tq
