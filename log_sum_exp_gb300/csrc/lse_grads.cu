// lse_grads.cu -- the global norm of many gradient tensors, and clipping by it
// (sm_103a).
//
//     norm = sqrt( sum over tensors and elements g^2 ),
//     g   <- g * min(1, max_norm / (norm + eps))
//
// The tensors are cut into chunks of kChunk elements, numbered through the
// list; CTA c takes chunks c, c + grid, ...  The list travels as a kernel
// parameter, so a call copies nothing to the device and can be captured.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_internal.h"

namespace lse {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
constexpr int64_t kChunk = 16384;  // elements
constexpr int kMaxList = 960;      // tensors per launch (32 bytes each, 32 KB of parameters)

struct GradEntry {
    const void* data;
    void* out;
    int64_t numel;
    int32_t first_chunk;
    int32_t dtype;
};

struct GradList {
    int count;
    int chunks;
    GradEntry t[kMaxList];
};

__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
    if (dtype == kF32) return static_cast<const float*>(p)[i];
    const unsigned short h = static_cast<const unsigned short*>(p)[i];
    return dtype == kBF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16)
                          : __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
    if (dtype == kF32) {
        static_cast<float*>(p)[i] = v;
        return;
    }
    uint32_t r;
    if (dtype == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
    static_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(r);
}

// The tensor that holds chunk c.
__device__ __forceinline__ int tensor_of(const GradList& list, int c) {
    int lo = 0, hi = list.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (list.t[mid].first_chunk <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// partial[c] = the sum of chunk c's squares, in 64 bits (a square of any f32 is
// a normal f64).
__global__ void __launch_bounds__(kGradThreads)
grad_square_kernel(const __grid_constant__ GradList list, double* __restrict__ partial) {
    __shared__ double part[kGradWarps];
    pdl_trigger();
    pdl_wait();
    for (int c = blockIdx.x; c < list.chunks; c += gridDim.x) {
        const GradEntry& t = list.t[tensor_of(list, c)];
        const int64_t i0 = (c - t.first_chunk) * kChunk;
        const int64_t i1 = i0 + kChunk < t.numel ? i0 + kChunk : t.numel;
        double s = 0.0;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kGradThreads) {
            const double v = load_any(t.data, t.dtype, i);
            s += v * v;
        }
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            s = 0.0;
            for (int w = 0; w < kGradWarps; ++w) s += part[w];
            partial[c] = s;
        }
        __syncthreads();
    }
}

__global__ void grad_norm_kernel(const double* __restrict__ partial, int64_t n,
                                 float* __restrict__ norm) {
    pdl_trigger();
    pdl_wait();
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 32) s += partial[i];
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(s));
}

__global__ void __launch_bounds__(kGradThreads)
grad_scale_kernel(const __grid_constant__ GradList list, const float* __restrict__ norm,
                  float max_norm, float eps) {
    pdl_trigger();
    pdl_wait();
    const float c0 = max_norm / (norm[0] + eps);
    const float coef = c0 > 1.0f ? 1.0f : c0;  // NaN stays NaN
    for (int c = blockIdx.x; c < list.chunks; c += gridDim.x) {
        const GradEntry& t = list.t[tensor_of(list, c)];
        const int64_t i0 = (c - t.first_chunk) * kChunk;
        const int64_t i1 = i0 + kChunk < t.numel ? i0 + kChunk : t.numel;
        if (coef == 1.0f && t.out == t.data) continue;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kGradThreads)
            store_any(t.out, t.dtype, i, load_any(t.data, t.dtype, i) * coef);
    }
}

lse_status check_list(const lse_tensor* tensors, int64_t count, const float* norm) {
    if (count < 0 || (count > 0 && tensors == nullptr)) return LSE_ERR_INVALID_ARG;
    if (norm == nullptr || reinterpret_cast<uintptr_t>(norm) % 4 != 0) return LSE_ERR_INVALID_ARG;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const lse_tensor& t = tensors[i];
        if (t.dtype != LSE_F32 && t.dtype != LSE_BF16 && t.dtype != LSE_F16)
            return LSE_ERR_UNSUPPORTED_DTYPE;
        const uintptr_t eb = t.dtype == LSE_F32 ? 4 : 2;
        if (t.numel < 0 || t.numel > INT64_MAX / 8) return LSE_ERR_INVALID_ARG;
        if (t.numel > 0 && t.data == nullptr) return LSE_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(t.data) % eb || reinterpret_cast<uintptr_t>(t.out) % eb)
            return LSE_ERR_INVALID_ARG;
        chunks += (t.numel + kChunk - 1) / kChunk;
        if (chunks > INT32_MAX) return LSE_ERR_INVALID_ARG;
    }
    return LSE_OK;
}

// The next tensors of the list from `at` on that fit one launch.
int64_t fill_list(const lse_tensor* tensors, int64_t count, int64_t at, GradList* list) {
    list->count = 0;
    list->chunks = 0;
    for (; at < count && list->count < kMaxList; ++at) {
        const lse_tensor& t = tensors[at];
        if (t.numel == 0) continue;
        list->t[list->count++] = GradEntry{t.data, t.out ? t.out : const_cast<void*>(t.data),
                                           t.numel, list->chunks, t.dtype};
        list->chunks += static_cast<int32_t>((t.numel + kChunk - 1) / kChunk);
    }
    return at;
}

lse_status run_grads(const lse_tensor* tensors, int64_t count, bool clip, float max_norm, float eps,
                     float* norm, cudaStream_t stream) {
    int sms = 0;
    lse_status st = device_sms(&sms);
    if (st != LSE_OK) return st;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) chunks += (tensors[i].numel + kChunk - 1) / kChunk;
    double* partial = nullptr;
    st = take_scratch(reinterpret_cast<void**>(&partial), sizeof(double) * (chunks + 1), stream);
    if (st != LSE_OK) return st;
    cudaError_t e = cudaSuccess;
    const int most = sms * 8;
    GradList list;
    int64_t done = 0;
    for (int64_t at = 0; at < count && e == cudaSuccess;) {
        at = fill_list(tensors, count, at, &list);
        if (list.chunks == 0) continue;
        e = launch_pdl(grad_square_kernel, dim3(list.chunks < most ? list.chunks : most),
                       dim3(kGradThreads), stream, list, partial + done);
        done += list.chunks;
    }
    if (e == cudaSuccess)
        e = launch_pdl(grad_norm_kernel, dim3(1), dim3(32), stream,
                       static_cast<const double*>(partial), chunks, norm);
    for (int64_t at = 0; clip && at < count && e == cudaSuccess;) {
        at = fill_list(tensors, count, at, &list);
        if (list.chunks == 0) continue;
        e = launch_pdl(grad_scale_kernel, dim3(list.chunks < most ? list.chunks : most),
                       dim3(kGradThreads), stream, list, static_cast<const float*>(norm), max_norm, eps);
    }
    const cudaError_t ef = cudaFreeAsync(partial, stream);
    return cuda_status(e == cudaSuccess ? ef : e);
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_grad_norm(const lse_tensor* tensors, int64_t count, float* norm, lse_stream_t stream) {
    const lse_status st = check_list(tensors, count, norm);
    if (st != LSE_OK) return st;
    return run_grads(tensors, count, false, 0.0f, 0.0f, norm, reinterpret_cast<cudaStream_t>(stream));
}

lse_status lse_grad_clip(const lse_tensor* tensors, int64_t count, float max_norm, float eps,
                         float* norm, lse_stream_t stream) {
    const lse_status st = check_list(tensors, count, norm);
    if (st != LSE_OK) return st;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return LSE_ERR_INVALID_ARG;
    return run_grads(tensors, count, true, max_norm, eps, norm, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
