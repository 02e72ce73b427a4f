// lse_sample_common.cuh -- what the entry point of lse_sample and its kernels share.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace lse {

// Temperatures below this draw the largest element, above kSampleHottest none.  Between them
// log2 e / T and the distances it multiplies stay within the f32 range.
constexpr float kSampleGreedy = 1e-20f, kSampleHottest = 1e20f;

struct SampleArgs {
    const void* x;
    int64_t B, N, row_stride;
    const float* u;
    const float* temperature;  // one for each row, or null: the value for all
    const int64_t* top_k;
    const float* top_p;
    const float* min_p;
    float temperature_all, top_p_all, min_p_all;
    int64_t top_k_all;
    int64_t* token;
    float* logprob;  // may be null
    int bits;        // fractional bits of a weight: N of them sum to less than 2^63
    int chunk, chunks_per_warp;  // vectors of a chunk, chunks of a warp
};

cudaError_t launch_sample_f32(const SampleArgs& a, int sms, cudaStream_t s);
cudaError_t launch_sample_bf16(const SampleArgs& a, int sms, cudaStream_t s);
cudaError_t launch_sample_f16(const SampleArgs& a, int sms, cudaStream_t s);

}  // namespace lse
