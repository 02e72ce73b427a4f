// lse_grads.cu -- the global norm of many gradient tensors, and clipping by it
// (sm_103a).
//
//     norm = sqrt( sum over tensors and elements g^2 ),
//     g   <- g * min(1, max_norm / (norm + eps))
//
// A tensor is the 16-byte vectors that cover it (elements outside it count as 0 and
// are not written), in chunks of kChunk vectors, numbered through the list.  CTA c of
// G takes a contiguous range of chunks, so it looks its tensors up once and then
// walks.  (Walking the ranges backwards when clipping, to meet what L2 still holds,
// measured the same: 388 us for 400 M bf16 elements either way, before the loads were
// ordinary ones; 386 now.)  The list travels as a
// kernel parameter: a call copies nothing to the device and can be captured.
//
// A thread squares and adds up to 64 elements in f32 (four sums, so at most 16
// squares in a row), then goes on in 64 bits.  Squares of f32 and bf16 gradients can
// leave the f32 range although the norm does not: a batch whose sum is not finite, or
// so small that squares may have been lost, is summed again in 64 bits, where every
// square of an f32 is a normal number.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_edges.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"

namespace lse {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kGradCtas = 4;       // per SM
constexpr int kGradU = 8;          // vectors per thread and chunk
constexpr int kScaleU = 4;         // of a step of the clipping pass
constexpr int64_t kChunk = kGradU * kGradThreads;  // vectors
constexpr int kMaxList = 960;      // tensors per launch (32 bytes each, 32 KB of parameters)

struct GradEntry {
    const void* data;
    void* out;
    int64_t numel;
    int32_t first_chunk;
    int32_t dtype;
};

// N: tensors that the parameter has room for (a short list costs less to launch).
template <int N>
struct GradList {
    int count;
    int chunks;
    GradEntry t[N];
};

__host__ __device__ inline int64_t tensor_vectors(const void* p, int64_t numel, int dtype) {
    const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15u);
    return (off + numel * (dtype == kF32 ? 4 : 2) + 15) >> 4;
}

// The chunks [first, last) of this CTA, and the tensor that holds chunk c.
template <int N>
__device__ __forceinline__ void chunk_range(const GradList<N>& list, int* first, int* last) {
    *first = static_cast<int>(static_cast<int64_t>(list.chunks) * blockIdx.x / gridDim.x);
    *last = static_cast<int>(static_cast<int64_t>(list.chunks) * (blockIdx.x + 1) / gridDim.x);
}
template <int N>
__device__ __forceinline__ int tensor_of(const GradList<N>& list, int c) {
    int lo = 0, hi = list.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (list.t[mid].first_chunk <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Vector k of a tensor whose bytes are [off, end) of what its vectors cover, with 0
// for the elements outside.
__device__ __forceinline__ void mask_zero(uint32_t* w, int64_t k, int off, int64_t end) {
    if (k == 0 || (k + 1) * 16 > end) {
        const int head = k == 0 ? off : 0;
        const int tail = (k + 1) * 16 > end ? static_cast<int>(end - k * 16) : 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] &= shl_clamped(0xffffffffu, 8 * head - 32 * i) & shr_clamped(0xffffffffu, 32 * i + 32 - 8 * tail);
    }
}

// A thread's elements of a chunk, from its vector k on, squared and added in 64 bits:
// rare, so read again element by element.
__device__ __noinline__ double squares_in_f64(const GradEntry& t, int64_t k) {
    const int eb = t.dtype == kF32 ? 4 : 2;
    const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.data) & 15u);
    double d = 0.0;
    for (int j = 0; j < kGradU; ++j) {
        const int64_t b0 = (k + j * kGradThreads) * 16 - off;  // byte in the tensor (may start before it)
        for (int64_t b = b0 < 0 ? 0 : b0; b < b0 + 16 && b < t.numel * eb; b += eb) {
            const double x = t.dtype == kF32 ? load_elem<kF32>(t.data, b / eb)
                             : t.dtype == kBF16 ? load_elem<kBF16>(t.data, b / eb) : load_elem<kF16>(t.data, b / eb);
            d = fma(x, x, d);
        }
    }
    return d;
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const GradEntry& t, int64_t k0) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(t.data) & 15u);
    const char* a0 = static_cast<const char*>(t.data) - off;
    const int64_t end = off + t.numel * DType<DT>::bytes;
    const int64_t vectors = (end + 15) >> 4;
    const int64_t k = k0 + threadIdx.x;
    uint32_t w[4 * kGradU];
#pragma unroll
    for (int j = 0; j < kGradU; ++j) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k + j * kGradThreads < vectors) v = ldg_stream16(a0 + (k + j * kGradThreads) * 16);
        w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
    }
    if (k0 == 0 || k0 + kChunk >= vectors) {
#pragma unroll
        for (int j = 0; j < kGradU; ++j)
            if (k + j * kGradThreads < vectors) mask_zero(&w[4 * j], k + j * kGradThreads, off, end);
    }
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 4 * kGradU; i += DT == kF32 ? 2 : 1) {
        uint64_t x;
        if constexpr (DT == kF32) x = f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
        else x = f2_pack(word_lo<DT>(w[i]), word_hi<DT>(w[i]));
        const int q = DT == kF32 ? (i >> 1) & 1 : i & 1;
        acc[q] = f2_fma(x, x, acc[q]);
    }
    float s0, s1, s2, s3;
    f2_unpack(acc[0], s0, s1);
    f2_unpack(acc[1], s2, s3);
    const float s = (s0 + s1) + (s2 + s3);
    if (s >= 0x1.0p-100f && s < __int_as_float(0x7f800000)) return s;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4 * kGradU; ++i) bits |= w[i] & (DT == kF32 ? 0x7fffffffu : 0x7fff7fffu);
    return bits == 0 ? 0.0 : squares_in_f64(t, k);
}

// The sum of a double over the CTA, in thread 0.  64-bit adds are few per clock on this
// GPU, so only one warp takes the last steps.
__device__ __forceinline__ double cta_sum(double s, double* part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = threadIdx.x < kGradWarps ? part[threadIdx.x] : 0.0;
#pragma unroll
        for (int off = kGradWarps / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    }
    return s;
}

// sqrt(s) as f32: the mantissa's root in f32, the (even) exponent halved.  s is 0, or
// at least 2^-298 (the smallest square), or infinite or NaN.
__device__ __forceinline__ float root(double s) {
    if (!(s > 0.0) || s > 1.0e300) return static_cast<float>(s);  // 0, NaN, inf
    const int e = ((__double2hiint(s) >> 20) - 1023) & ~1;
    const double two_e = __hiloint2double((1023 - e) << 20, 0);   // 2^-e
    const float r = sqrtf(static_cast<float>(s * two_e));         // of [1, 4)
    const int h = e / 2;                                          // -149 .. 498
    // (in two factors: 2^h alone may be beyond f32)
    const int h0 = h < -64 ? -64 : h > 64 ? 64 : h;
    const int h1 = h - h0 > 127 ? 127 : h - h0;
    return r * __int_as_float((127 + h0) << 23) * __int_as_float((127 + h1) << 23);
}

// partial[c] = the sum of CTA c's squares.
//
// Bound by its one read: 400 M bf16 in 119 us, 6.7 TB/s.  Eight 16-byte loads per thread
// and four CTAs per SM keep 128 KB per SM in flight; half an instruction per element
// (packed FMA) leaves two thirds of the issue rate unused.  The 64-bit adds, which this
// GPU has few of, are one per thread and chunk of 32 to 64 elements.
template <int N>
__global__ void __launch_bounds__(kGradThreads, kGradCtas)
grad_square_kernel(const __grid_constant__ GradList<N> list, double* __restrict__ partial) {
    __shared__ double part[kGradWarps];
    pdl_trigger();
    pdl_wait();
    int c, last;
    chunk_range(list, &c, &last);
    double s = 0.0;
    int i = tensor_of(list, c);
    for (; c < last; ++c) {
        while (i + 1 < list.count && list.t[i + 1].first_chunk <= c) ++i;
        const GradEntry& t = list.t[i];
        const int64_t k0 = (c - t.first_chunk) * kChunk;
        s += t.dtype == kF32 ? chunk_squares<kF32>(t, k0)
             : t.dtype == kBF16 ? chunk_squares<kBF16>(t, k0) : chunk_squares<kF16>(t, k0);
    }
    s = cta_sum(s, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from n partial sums, the same in every thread of a CTA.
struct NormShared {
    double part[kGradWarps];
    float norm;
};
__device__ __forceinline__ float norm_of(const double* partial, int64_t n, NormShared& sh) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kGradThreads) s += partial[i];
    s = cta_sum(s, sh.part);
    if (threadIdx.x == 0) sh.norm = root(s);
    __syncthreads();
    return sh.norm;
}

__global__ void __launch_bounds__(kGradThreads)
grad_norm_kernel(const double* __restrict__ partial, int64_t n, float* __restrict__ norm) {
    __shared__ NormShared sh;
    pdl_trigger();
    pdl_wait();
    const float v = norm_of(partial, n, sh);
    if (threadIdx.x == 0) norm[0] = v;
}

// Bytes [from, to) of a vector, element by element (a tensor's ends, or an `out` at
// another offset from a 16-byte boundary).
__device__ __noinline__ void store_part(char* p, uint4 v, int from, int to, int eb) {
    for (int b = from; b < to; b += eb) {
        const uint32_t w = b < 4 ? v.x : b < 8 ? v.y : b < 12 ? v.z : v.w;
        if (eb == 4) *reinterpret_cast<uint32_t*>(p + b) = w;
        else *reinterpret_cast<unsigned short*>(p + b) = static_cast<unsigned short>((b & 2) ? w >> 16 : w);
    }
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const GradEntry& t, int64_t k0, float coef) {
    constexpr int EB = DType<DT>::bytes;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(t.data) & 15u);
    const char* a0 = static_cast<const char*>(t.data) - off;
    char* const o0 = static_cast<char*>(t.out) - off;
    const bool vec = (reinterpret_cast<uintptr_t>(o0) & 15u) == 0;  // the same offset from a boundary
    const int64_t end = off + t.numel * EB;
    const int64_t vectors = (end + 15) >> 4;
    const uint64_t c2 = f2_pack(coef, coef);
    // (four vectors at a time: eight would spill in the loop at 64 registers; four spill 48
    // bytes in the parts for a tensor's ends, none of it executed for whole vectors)
#pragma unroll 1
    for (int64_t k = k0 + threadIdx.x; k < k0 + kChunk && k < vectors; k += kScaleU * kGradThreads) {
        uint4 v[kScaleU];
#pragma unroll
        for (int j = 0; j < kScaleU; ++j)
            if (k + j * kGradThreads < vectors) v[j] = ld_stream16(a0 + (k + j * kGradThreads) * 16);
#pragma unroll
        for (int j = 0; j < kScaleU; ++j) {
            const int64_t kk = k + j * kGradThreads;
            if (kk >= vectors) continue;
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; i += DT == kF32 ? 2 : 1) {
                float x, y;
                if constexpr (DT == kF32) {
                    f2_unpack(f2_mul(f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), c2), x, y);
                    o[i] = __float_as_uint(x);
                    o[i + 1] = __float_as_uint(y);
                } else {
                    f2_unpack(f2_mul(f2_pack(word_lo<DT>(w[i]), word_hi<DT>(w[i])), c2), x, y);
                    o[i] = pack2<DT>(x, y);
                }
            }
            if (vec && (kk > 0 || off == 0) && (kk + 1) * 16 <= end) {
                *reinterpret_cast<uint4*>(o0 + kk * 16) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                const int from = kk == 0 ? off : 0;
                const int to = (kk + 1) * 16 > end ? static_cast<int>(end - kk * 16) : 16;
                store_part(o0 + kk * 16, make_uint4(o[0], o[1], o[2], o[3]), from, to, EB);
            }
        }
    }
}

// Bound by one read and one write: 400 M bf16 in 258 us, 6.2 TB/s (the copy rate measured
// on this GPU is 6.8).  Four loads per thread are in flight: eight spill in the loop (453 us), two
// measured 393 us for norm and clipping together against 388.
//
// `out` may be the tensor itself, and neighbouring tensors share vectors, so nothing here is
// read through the read-only path.
//
// out = g c for the list's tensors; every CTA forms the norm from the n partial sums
// itself (a few KB from L2), which costs less than one more launch.
template <int N>
__global__ void __launch_bounds__(kGradThreads, kGradCtas)
grad_scale_kernel(const __grid_constant__ GradList<N> list, const double* __restrict__ partial, int64_t n,
                  float max_norm, float eps, float* __restrict__ norm) {
    __shared__ NormShared sh;
    pdl_trigger();
    pdl_wait();
    const float v = norm_of(partial, n, sh);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = v;
    const float c0 = max_norm / (v + eps);
    const float coef = c0 > 1.0f || v == 0.0f ? 1.0f : c0;  // NaN stays NaN, but zeros have nothing to clip (0 / 0)
    int c, last;
    chunk_range(list, &c, &last);
    int i = tensor_of(list, c);
    for (; c < last; ++c) {
        while (i + 1 < list.count && list.t[i + 1].first_chunk <= c) ++i;
        const GradEntry& t = list.t[i];
        if (coef == 1.0f && t.out == t.data) continue;
        const int64_t k0 = (c - t.first_chunk) * kChunk;
        if (t.dtype == kF32) chunk_scale<kF32>(t, k0, coef);
        else if (t.dtype == kBF16) chunk_scale<kBF16>(t, k0, coef);
        else chunk_scale<kF16>(t, k0, coef);
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
        chunks += (tensor_vectors(t.data, t.numel, t.dtype) + kChunk - 1) / kChunk;
        if (chunks > INT32_MAX) return LSE_ERR_INVALID_ARG;
    }
    return LSE_OK;
}

// Tensors of the list from *at on, as many as one launch takes, and that launch's grid.
template <int N>
int fill_list(const lse_tensor* tensors, int64_t count, int64_t* at, int sms, GradList<N>* list) {
    list->count = 0;
    list->chunks = 0;
    for (; *at < count && list->count < N; ++*at) {
        const lse_tensor& t = tensors[*at];
        if (t.numel == 0) continue;
        list->t[list->count++] = GradEntry{t.data, t.out ? t.out : const_cast<void*>(t.data),
                                           t.numel, list->chunks, t.dtype};
        list->chunks += static_cast<int32_t>((tensor_vectors(t.data, t.numel, t.dtype) + kChunk - 1) / kChunk);
    }
    return list->chunks < sms * kGradCtas ? list->chunks : sms * kGradCtas;
}

template <int N>
lse_status run_grads(const lse_tensor* tensors, int64_t count, bool clip, float max_norm, float eps,
                     float* norm, cudaStream_t stream) {
    int sms = 0;
    lse_status st = device_sms(&sms);
    if (st != LSE_OK) return st;
    double* partial = nullptr;
    const int64_t launches = count / N + 1;
    st = take_scratch(reinterpret_cast<void**>(&partial), sizeof(double) * launches * sms * kGradCtas, stream);
    if (st != LSE_OK) return st;
    cudaError_t e = cudaSuccess;
    GradList<N> list;
    int64_t n = 0;  // partial sums
    for (int64_t at = 0; at < count && e == cudaSuccess;) {
        const int grid = fill_list(tensors, count, &at, sms, &list);
        if (grid == 0) continue;
        e = launch_pdl(grad_square_kernel<N>, dim3(grid), dim3(kGradThreads), stream, list, partial + n);
        n += grid;
    }
    if (e == cudaSuccess && (!clip || n == 0))
        e = launch_pdl(grad_norm_kernel, dim3(1), dim3(kGradThreads), stream,
                       static_cast<const double*>(partial), n, norm);
    for (int64_t at = 0; clip && at < count && e == cudaSuccess;) {
        const int grid = fill_list(tensors, count, &at, sms, &list);
        if (grid == 0) continue;
        e = launch_pdl(grad_scale_kernel<N>, dim3(grid), dim3(kGradThreads), stream, list,
                       static_cast<const double*>(partial), n, max_norm, eps, norm);
    }
    const cudaError_t ef = cudaFreeAsync(partial, stream);
    return cuda_status(e == cudaSuccess ? ef : e);
}

lse_status run_grads_list(const lse_tensor* tensors, int64_t count, bool clip, float max_norm, float eps,
                          float* norm, lse_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (count <= 48) return run_grads<48>(tensors, count, clip, max_norm, eps, norm, s);
    if (count <= 240) return run_grads<240>(tensors, count, clip, max_norm, eps, norm, s);
    return run_grads<kMaxList>(tensors, count, clip, max_norm, eps, norm, s);
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_grad_norm(const lse_tensor* tensors, int64_t count, float* norm, lse_stream_t stream) {
    const lse_status st = check_list(tensors, count, norm);
    if (st != LSE_OK) return st;
    return run_grads_list(tensors, count, false, 0.0f, 0.0f, norm, stream);
}

lse_status lse_grad_clip(const lse_tensor* tensors, int64_t count, float max_norm, float eps,
                         float* norm, lse_stream_t stream) {
    const lse_status st = check_list(tensors, count, norm);
    if (st != LSE_OK) return st;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return LSE_ERR_INVALID_ARG;
    return run_grads_list(tensors, count, true, max_norm, eps, norm, stream);
}

}  // extern "C"
