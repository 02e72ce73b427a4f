// lse_stats_common.cuh -- what the token statistics and their gradient share: arguments,
// launch declarations, and a few device helpers (sm_103a).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"

namespace lse {

struct StatsArgs {
    const void* x;
    int64_t B, N, row_stride;
    const int64_t* target;
    int K;
    float* logprob;      // each output may be null
    float* entropy;
    float* lse;
    float* lse_low;      // what rounding took from lse
    float* top_logprob;  // [B, K]
    int64_t* top_index;
    int cluster;         // CTAs that share a row
    int chunk_shift;     // log2 of the batches of a chunk (long rows)
};

cudaError_t launch_token_stats_f32(const StatsArgs& a, int sms, cudaStream_t s);
cudaError_t launch_token_stats_bf16(const StatsArgs& a, int sms, cudaStream_t s);
cudaError_t launch_token_stats_f16(const StatsArgs& a, int sms, cudaStream_t s);

// Below this many octaves of the maximum an exponential is 0 in f32.
constexpr float kFarBelow = -16384.0f;

}  // namespace lse
