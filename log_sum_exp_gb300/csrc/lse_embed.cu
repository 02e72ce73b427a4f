// lse_embed.cu -- embedding rows for given tokens, and the table's gradient
// (sm_103a).
//
//     out[t, :]    = scale * table[ids[t], :]
//     dtable[v, :] = scale * sum_{t : ids[t] = v} grad[t, :]
//
// The gradient sorts the tokens by id, stably, so that each table row's sum runs
// over its tokens in their order: nothing is added through atomics, and equal
// inputs give equal bits.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_internal.h"

namespace lse {
namespace {

constexpr int kEmbedThreads = 256;

template <int DT>
__device__ __forceinline__ void put_elem(void* row, int64_t i, float v) {
    if constexpr (DT == kF32) {
        static_cast<float*>(row)[i] = v;
    } else {
        uint32_t r;
        if constexpr (DT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
        else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
        static_cast<unsigned short*>(row)[i] = static_cast<unsigned short>(r);
    }
}

template <int DT>
__global__ void __launch_bounds__(kEmbedThreads)
embed_kernel(const char* __restrict__ table, int64_t V, int64_t D, int64_t table_stride,
             const int64_t* __restrict__ ids, int64_t T, float scale, char* __restrict__ out,
             int64_t out_stride) {
    pdl_trigger();
    pdl_wait();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int64_t id = ids[t];
        const bool in = id >= 0 && id < V;
        for (int64_t d = threadIdx.x; d < D; d += kEmbedThreads)
            put_elem<DT>(out + t * out_stride * DType<DT>::bytes, d,
                         in ? load_elem<DT>(table + id * table_stride * DType<DT>::bytes, d) * scale
                            : __int_as_float(0x7fc00000));
    }
}

// Sorted place of every token: the tokens with a lower id, or the same id and an
// earlier place.  Tokens that add nothing sort last.
__device__ __forceinline__ uint32_t sort_id(int64_t id, int64_t V, int64_t padding) {
    return id >= 0 && id < V && id != padding ? static_cast<uint32_t>(id) : 0xffffffffu;
}

__global__ void __launch_bounds__(kEmbedThreads)
rank_kernel(const int64_t* __restrict__ ids, int64_t T, int64_t V, int64_t padding,
            uint32_t* __restrict__ sorted_id, uint32_t* __restrict__ sorted_at) {
    pdl_trigger();
    pdl_wait();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kEmbedThreads + threadIdx.x; t < T;
         t += static_cast<int64_t>(gridDim.x) * kEmbedThreads) {
        const uint32_t mine = sort_id(ids[t], V, padding);
        uint32_t place = 0;
        for (int64_t j = 0; j < T; ++j) {
            const uint32_t other = sort_id(__ldg(ids + j), V, padding);
            place += other < mine || (other == mine && j < t);
        }
        sorted_id[place] = mine;
        sorted_at[place] = static_cast<uint32_t>(t);
    }
}

__device__ __forceinline__ int64_t lower_bound(const uint32_t* a, int64_t n, uint32_t v) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <int DT, int OT>
__global__ void __launch_bounds__(kEmbedThreads)
embed_backward_kernel(const char* __restrict__ grad, int64_t T, int64_t D, int64_t grad_stride,
                      const uint32_t* __restrict__ sorted_id, const uint32_t* __restrict__ sorted_at,
                      int64_t V, float scale, char* __restrict__ dtable, int64_t dtable_stride,
                      bool accumulate) {
    pdl_trigger();
    pdl_wait();
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
        const int64_t i0 = lower_bound(sorted_id, T, static_cast<uint32_t>(v));
        const int64_t i1 = lower_bound(sorted_id, T, static_cast<uint32_t>(v) + 1);
        if (accumulate && i0 == i1) continue;
        char* row = dtable + v * dtable_stride * DType<OT>::bytes;
        for (int64_t d = threadIdx.x; d < D; d += kEmbedThreads) {
            float s = 0.0f;
            for (int64_t i = i0; i < i1; ++i)
                s += load_elem<DT>(grad + static_cast<int64_t>(sorted_at[i]) * grad_stride * DType<DT>::bytes, d);
            s *= scale;
            if (accumulate) s += load_elem<OT>(row, d);
            put_elem<OT>(row, d, s);
        }
    }
}

bool rows_ok(int64_t rows, int64_t D, int64_t stride, int64_t eb) {
    int64_t extent = 0;
    if (rows < 0 || D < 0 || stride < D) return false;
    if (rows > 0 && __builtin_mul_overflow(rows - 1, stride, &extent)) return false;
    return !__builtin_add_overflow(extent, D, &extent) && !__builtin_mul_overflow(extent, eb, &extent);
}

bool valid_dtype(int dt) { return dt == LSE_F32 || dt == LSE_BF16 || dt == LSE_F16; }
bool misaligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

unsigned capped(int64_t n, int64_t most) { return static_cast<unsigned>(n < 1 ? 1 : n < most ? n : most); }

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_embedding(const void* table, lse_dtype dtype, int64_t V, int64_t D,
                         int64_t table_stride, const int64_t* ids, int64_t T, float scale, void* out,
                         int64_t out_stride, lse_stream_t stream) {
    if (!valid_dtype(dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    if (!rows_ok(V, D, table_stride, eb) || !rows_ok(T, D, out_stride, eb)) return LSE_ERR_INVALID_ARG;
    if (misaligned(table, eb) || misaligned(out, eb) || misaligned(ids, 8)) return LSE_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return LSE_OK;
    if (ids == nullptr || out == nullptr || (V > 0 && table == nullptr)) return LSE_ERR_INVALID_ARG;
    const auto kernel = dtype == LSE_F32 ? embed_kernel<kF32>
                        : dtype == LSE_BF16 ? embed_kernel<kBF16> : embed_kernel<kF16>;
    return cuda_status(launch_pdl(kernel, dim3(capped(T, INT_MAX)), dim3(kEmbedThreads),
                                  reinterpret_cast<cudaStream_t>(stream),
                                  static_cast<const char*>(table), V, D, table_stride, ids, T, scale,
                                  static_cast<char*>(out), out_stride));
}

lse_status lse_embedding_backward(const void* grad, lse_dtype dtype, int64_t T, int64_t D,
                                  int64_t grad_stride, const int64_t* ids, int64_t V, float scale,
                                  int64_t padding, void* dtable, lse_dtype dtable_dtype,
                                  int64_t dtable_stride, int accumulate, lse_stream_t stream_) {
    if (!valid_dtype(dtype) || !valid_dtype(dtable_dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (dtable_dtype != dtype && dtable_dtype != LSE_F32) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2, ob = dtable_dtype == LSE_F32 ? 4 : 2;
    if (!rows_ok(T, D, grad_stride, eb) || !rows_ok(V, D, dtable_stride, ob)) return LSE_ERR_INVALID_ARG;
    if (T > INT32_MAX || V > INT32_MAX) return LSE_ERR_INVALID_ARG;
    if (misaligned(grad, eb) || misaligned(dtable, ob) || misaligned(ids, 8)) return LSE_ERR_INVALID_ARG;
    if (V == 0 || D == 0) return LSE_OK;
    if (dtable == nullptr || (T > 0 && (grad == nullptr || ids == nullptr))) return LSE_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    uint32_t* scratch = nullptr;
    const lse_status st = take_scratch(reinterpret_cast<void**>(&scratch), sizeof(uint32_t) * 2 * (T + 1), stream);
    if (st != LSE_OK) return st;
    cudaError_t e = cudaSuccess;
    if (T > 0)
        e = launch_pdl(rank_kernel, dim3(capped((T + kEmbedThreads - 1) / kEmbedThreads, 65536)),
                       dim3(kEmbedThreads), stream, ids, T, V, padding, scratch, scratch + T);
    const auto kernel = dtype == LSE_F32 ? embed_backward_kernel<kF32, kF32>
                        : dtype == LSE_BF16 ? (dtable_dtype == LSE_F32 ? embed_backward_kernel<kBF16, kF32>
                                                                       : embed_backward_kernel<kBF16, kBF16>)
                                            : (dtable_dtype == LSE_F32 ? embed_backward_kernel<kF16, kF32>
                                                                       : embed_backward_kernel<kF16, kF16>);
    if (e == cudaSuccess)
        e = launch_pdl(kernel, dim3(capped(V, 1 << 20)), dim3(kEmbedThreads), stream,
                       static_cast<const char*>(grad), T, D, grad_stride,
                       static_cast<const uint32_t*>(scratch), static_cast<const uint32_t*>(scratch + T), V,
                       scale, static_cast<char*>(dtable), dtable_stride, accumulate != 0);
    const cudaError_t ef = cudaFreeAsync(scratch, stream);
    return cuda_status(e == cudaSuccess ? ef : e);
}

}  // extern "C"
