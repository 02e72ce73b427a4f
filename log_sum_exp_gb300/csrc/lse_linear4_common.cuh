// lse_linear4_common.cuh -- what matrices held in 4 bits and the products with them share
// (sm_103a).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"

namespace lse {

constexpr int kBlock = 128;  // columns of a block of codes
constexpr int kBlockBytes = 64;
constexpr int kBlockWords = 16;

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t K) { return (K + kBlock - 1) / kBlock; }

// Eight elements from column k on, zeros behind the row.
template <int DT> __device__ __forceinline__ void load8(const void* row, int64_t k, int64_t K, bool vec, float (&f)[8]) {
    constexpr int EB = DType<DT>::bytes;
    if (vec && k + 8 <= K) {
        const char* p = static_cast<const char*>(row) + k * EB;
        const uint4 a = ldg_stream16(p);
        if constexpr (DT == kF32) {
            const uint4 b = ldg_stream16(p + 16);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = word_lo<DT>(w[i]), f[2 * i + 1] = word_hi<DT>(w[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k + i < K ? load_elem<DT>(row, k + i) : 0.0f;
}

struct LinearArgs {
    const void* x;
    int64_t T, x_stride;
    int K, blocks, groups, group;
    const uint4* codes;
    const void* scales;
    int64_t scale_stride, N;
    int scale_dtype;
    void* out;
    int64_t out_stride;
    bool out_f32;
    bool x_vec;        // rows of x start on 16-byte boundaries
    int chunk_blocks;  // blocks of x that shared memory holds at a time
    int row_bytes;     // of a row of x there: 64 more than a multiple of 128, so that eight lanes on two rows touch every bank once
    int tokens;        // rows of x in shared memory
    int64_t tiles;     // groups of 16 RT rows
    int ks;            // warps that share the columns of a tile
};

cudaError_t launch_linear4_f32(const LinearArgs& a, int sms, cudaStream_t s);
cudaError_t launch_linear4_bf16(const LinearArgs& a, int sms, cudaStream_t s);
cudaError_t launch_linear4_f16(const LinearArgs& a, int sms, cudaStream_t s);

}  // namespace lse
