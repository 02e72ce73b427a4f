// lse_norm_common.cuh -- what the entry points of lse_residual_norm and its kernels share.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/lse.h"

namespace lse {

enum Gate : int { kNoGate = LSE_GATE_NONE, kChannelGate = LSE_GATE_CHANNEL, kElementGate = LSE_GATE_ELEMENT };

constexpr int kNormMaxColumns = 16384;


struct NormArgs {
    int64_t T;
    int D;
    const char* x;
    const char* y;     // may be null: h = x
    const char* gate;  // null, a row of columns, or T rows
    const char* post;  // null: no norm of y
    const char* weight;
    int64_t x_bytes, y_bytes, gate_bytes;  // between rows
    bool weights_f32;  // weight, post and a channel gate (else of the rows' type)
    bool weights_vec;  // they start on 16-byte boundaries
    int gate_kind;
    float scale, eps, inv_d;
    // forward
    char* h;  // null: not wanted
    char* out;
    int64_t h_bytes, out_bytes;
    float* rstd;       // may be null
    float* post_rstd;  // may be null
    // gradient
    const char* dout;
    const char* dh;  // may be null: zeros
    int64_t dout_bytes, dh_bytes;
    const float* rstd_in;
    const float* post_rstd_in;
    char* dx;     // each may be null
    char* dy;
    char* dgate;  // of an element gate
    int64_t dx_bytes, dy_bytes, dgate_bytes;
    float* part;  // [2, parts, D]; null: no sums over rows are wanted
    int parts;
};

enum Mode : int { kSingle = 0, kCover = 1, kWhole = 2 };
// CTAs of the gradient that an SM holds: a slot of 16-bit elements takes about 120 registers
// (8 columns' sums, factors and terms), one of f32 about 64.
__host__ __device__ constexpr int backward_ctas(int threads, bool f32) {
    return threads == 128 ? (f32 ? 6 : 4) : threads == 256 ? (f32 ? 3 : 2) : threads == 512 && f32 ? 2 : 1;
}

// Rows that a CTA of the gradient takes at a time, and the CTAs.
struct BackwardPlan {
    int tx, v, rows, grid;
};

struct NormFinishArgs {
    const float* part;  // [2, parts, D]
    int parts, D;
    const void* post;  // factors of the second sum
    const void* gate;
    bool weights_f32;
    float scale;  // of the second sum
    void* dweight;  // each may be null
    void* dpost;
    void* dgate;
};


#define LSE_DECLARE_NORM(SUFFIX)                                                                                       \
    cudaError_t launch_norm_##SUFFIX(const NormArgs& a, int mode, int64_t slots, bool few, cudaStream_t s);             \
    cudaError_t launch_norm_backward_##SUFFIX(const NormArgs& a, int mode, const BackwardPlan& p, cudaStream_t s);      \
    cudaError_t launch_norm_finish_##SUFFIX(const NormFinishArgs& a, cudaStream_t s);
LSE_DECLARE_NORM(f32)
LSE_DECLARE_NORM(bf16)
LSE_DECLARE_NORM(f16)

}  // namespace lse
