// lse_sample.cu -- the C entry point of drawing tokens.  Kernels: lse_sample.cuh.
#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_internal.h"
#include "lse_sample_common.cuh"

using namespace lse;

extern "C" {

lse_status lse_sample(const void* x, lse_dtype dtype, int64_t B, int64_t N, int64_t row_stride, const float* u,
                      const lse_sampling* settings, int64_t* token, float* logprob, lse_stream_t stream) {
    const void* stand_in = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
    lse_status st = check_args(x, dtype, B, N, row_stride, stand_in);
    if (st != LSE_OK) return st;
    if (N > INT_MAX - 64 || B > INT_MAX || settings == nullptr) return LSE_ERR_INVALID_ARG;
    const lse_sampling& g = *settings;
    if (misaligned(u, 4) || misaligned(token, 8) || misaligned(logprob, 4) || misaligned(g.temperature_rows, 4) ||
        misaligned(g.top_k_rows, 8) || misaligned(g.top_p_rows, 4) || misaligned(g.min_p_rows, 4))
        return LSE_ERR_INVALID_ARG;
    // (NaN compares false.)
    if (!g.temperature_rows && !(g.temperature >= 0.0f && g.temperature <= kSampleHottest)) return LSE_ERR_INVALID_ARG;
    if (!g.top_p_rows && !(g.top_p >= 0.0f)) return LSE_ERR_INVALID_ARG;
    if (!g.min_p_rows && !(g.min_p >= 0.0f)) return LSE_ERR_INVALID_ARG;
    if (!g.top_k_rows && g.top_k < 0) return LSE_ERR_INVALID_ARG;
    if (B == 0) return LSE_OK;
    if (u == nullptr || token == nullptr) return LSE_ERR_INVALID_ARG;
    SampleArgs a = {};
    a.x = x;
    a.B = B;
    a.N = N;
    a.row_stride = row_stride;
    a.u = u;
    a.temperature = g.temperature_rows;
    a.top_k = g.top_k_rows;
    a.top_p = g.top_p_rows;
    a.min_p = g.min_p_rows;
    a.temperature_all = g.temperature;
    a.top_k_all = g.top_k;
    a.top_p_all = g.top_p;
    a.min_p_all = g.min_p;
    a.token = token;
    a.logprob = logprob;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(dtype == LSE_F32 ? launch_sample_f32(a, sms, s)
                       : dtype == LSE_BF16 ? launch_sample_bf16(a, sms, s) : launch_sample_f16(a, sms, s));
}

}  // extern "C"
