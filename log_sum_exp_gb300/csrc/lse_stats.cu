// lse_stats.cu -- token statistics of rows of logits and their gradient (sm_103a).
//
// For a row x of N logits, p = softmax(x) and lse = log sum exp x:
//
//     logprob = x[t] - lse                         (t the given token)
//     entropy = -sum_n p_n log p_n
//     top     = the K largest x_n, as (x_n - lse, n), ties by the lower n
//
// With mu the row's maximum and z_n = (x_n - mu) log2 e <= 0, the entropy is
//
//     ln 2 * ( log2 s + u / s ),   s = sum 2^z,   u = sum 2^z (-z),
//
// a sum of two non-negative terms, so nothing cancels.  (m, s, u) is kept online:
// raising the maximum by d (in units of z) turns u into (u + d s) 2^-d and s into
// s 2^-d.  A masked element (z = -inf) adds 2^z = 0 to s and, with z bounded
// below by kFarBelow, 0 to u.
#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_internal.h"
#include "lse_topk.cuh"

namespace lse {
namespace {

struct StatsArgs {
    const void* x;
    int64_t B, N, row_stride;
    const int64_t* target;
    int K;
    float* logprob;      // each output may be null
    float* entropy;
    float* lse;
    float* top_logprob;  // [B, K]
    int64_t* top_index;
};

struct StatsBackwardArgs {
    const void* x;
    int64_t B, N, row_stride;
    const float* lse;
    const float* entropy;
    const int64_t* target;
    const int64_t* top_index;
    int K;
    const float* grad_logprob;  // each gradient may be null (zero)
    const float* grad_entropy;
    const float* grad_top;
    const float* grad_lse;
    void* dx;
    int64_t dx_row_stride;
};

// Below this many octaves of the maximum an exponential is 0 in f32.
constexpr float kFarBelow = -16384.0f;

struct StatAcc {
    float m, s, u;
};

__device__ __forceinline__ StatAcc stat_identity() { return StatAcc{__int_as_float(kNegInfF32), 0.0f, 0.0f}; }

// The accumulator against another shift mu >= its own: its sums scaled by 2^-d.
__device__ __forceinline__ StatAcc stat_shift(StatAcc a, float mu) {
    const float d = fminf((mu - a.m) * kLog2e, -kFarBelow);
    const float f = ex2(-d);
    return StatAcc{a.m, a.s * f, fmaf(d, a.s, a.u) * f};
}

__device__ __forceinline__ StatAcc stat_merge(StatAcc a, StatAcc b) {
    const float m = fmaxf(a.m, b.m);
    const float mu = shift_of(m);
    a = stat_shift(a, mu);
    b = stat_shift(b, mu);
    return StatAcc{m, a.s + b.s, a.u + b.u};
}

__device__ __forceinline__ StatAcc stat_warp_merge(StatAcc a) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        StatAcc b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, off);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, off);
        b.u = __shfl_xor_sync(0xffffffffu, a.u, off);
        a = stat_merge(a, b);
    }
    return a;
}

// NaN for a row that is no distribution: a NaN or +inf in it, or nothing but -inf.
__device__ __forceinline__ float stat_entropy(StatAcc a) {
    if (!(fabsf(a.m) < __int_as_float(0x7f800000))) return __int_as_float(0x7fc00000);
    return kLn2 * (lg2(a.s) + a.u / a.s);
}

constexpr int kStatThreads = 256;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kScanElems = 4;  // elements per thread and tile of the top-K scan

// The K largest keys of a row, in row order: a running list, and per tile the
// elements above its K-th key, which warps sort and merge into it.  Equal values
// later in the row rank lower, so they are not taken up again.
template <int DT>
__device__ __forceinline__ void scan_topk(const void* rp, int64_t N, int K, uint64_t* list,
                                          uint64_t* found, int* count, uint64_t* warp_list) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid < 32) list[tid] = 0;
    __syncthreads();
    for (int64_t base = 0; base < N; base += kStatThreads * kScanElems) {
        const uint64_t bar = list[K - 1];
        if (tid == 0) *count = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kScanElems; ++j) {
            const int64_t i = base + tid + j * kStatThreads;
            if (i < N) {
                const uint64_t k = topk_key(load_elem<DT>(rp, i), static_cast<uint32_t>(i));
                if (k > bar) found[atomicAdd(count, 1)] = k;
            }
        }
        __syncthreads();
        const int n = *count;
        if (n == 0) continue;
        uint64_t best = 0;
        for (int at = wid * 32; at < n; at += kStatThreads)
            best = list_merge(best, list_sort(at + lane < n ? found[at + lane] : 0, lane), lane);
        warp_list[tid] = best;
        __syncthreads();
        if (wid == 0) {
            uint64_t k = list[lane];
            for (int w = 0; w < kStatWarps; ++w) k = list_merge(k, warp_list[w * 32 + lane], lane);
            list[lane] = k;
        }
        __syncthreads();
    }
}

// A CTA per row.
template <int DT>
__global__ void __launch_bounds__(kStatThreads)
lse_stats_kernel(const StatsArgs a) {
    __shared__ uint64_t list[32], warp_list[kStatThreads], found[kStatThreads * kScanElems];
    __shared__ float part[3][kStatWarps];
    __shared__ float row_lse;
    __shared__ int count;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    for (int64_t row = blockIdx.x; row < a.B; row += gridDim.x) {
        const char* rp = static_cast<const char*>(a.x) + row * a.row_stride * DType<DT>::bytes;
        StatAcc acc = stat_identity();
        for (int64_t i = tid; i < a.N; i += kStatThreads) {
            const float x = load_elem<DT>(rp, i);
            if (x > acc.m) {
                acc = stat_shift(acc, shift_of(x));
                acc.m = x;
            }
            const float z = (x - shift_of(acc.m)) * kLog2e;
            const float e = ex2(z);
            acc.s += e;
            acc.u = fmaf(-e, fmaxf(z, kFarBelow), acc.u);
        }
        acc = stat_warp_merge(acc);
        if (lane == 0) {
            part[0][wid] = acc.m;
            part[1][wid] = acc.s;
            part[2][wid] = acc.u;
        }
        __syncthreads();
        if (tid == 0) {
            acc = stat_identity();
            for (int w = 0; w < kStatWarps; ++w)
                acc = stat_merge(acc, StatAcc{part[0][w], part[1][w], part[2][w]});
            const float l = acc_finalize(Acc{acc.m, acc.s});
            row_lse = l;
            if (a.lse) a.lse[row] = l;
            if (a.entropy) a.entropy[row] = stat_entropy(acc);
            if (a.logprob) {
                const int64_t t = a.target[row];
                a.logprob[row] = t >= 0 && t < a.N ? load_elem<DT>(rp, t) - l : __int_as_float(0x7fc00000);
            }
        }
        __syncthreads();
        if (a.K > 0) {
            scan_topk<DT>(rp, a.N, a.K, list, found, &count, warp_list);
            if (tid < a.K) {
                const uint64_t k = list[tid];
                a.top_index[row * a.K + tid] = k ? key_column(k) : -1;
                a.top_logprob[row * a.K + tid] = k ? key_value(k) - row_lse : __int_as_float(kNegInfF32);
            }
            __syncthreads();
        }
    }
}

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

// dx_n = p_n (c - gH (log p_n + H)) + gl [n = t] + sum_k gt_k [n = i_k],
// c = g_lse - gl - sum_k gt_k.  A CTA per row.
template <int DT>
__global__ void __launch_bounds__(kStatThreads)
lse_stats_backward_kernel(const StatsBackwardArgs a) {
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < a.B; row += gridDim.x) {
        const char* xr = static_cast<const char*>(a.x) + row * a.row_stride * DType<DT>::bytes;
        char* dr = static_cast<char*>(a.dx) + row * a.dx_row_stride * DType<DT>::bytes;
        const int64_t t = a.grad_logprob ? a.target[row] : -1;
        const float gl = t >= 0 && t < a.N ? a.grad_logprob[row] : 0.0f;
        const float gh = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
        const float gs = a.grad_lse ? a.grad_lse[row] : 0.0f;
        float c = gs - gl;
        bool any = gl != 0.0f || gh != 0.0f || gs != 0.0f;
        for (int k = 0; k < a.K; ++k) {
            const int64_t i = a.top_index[row * a.K + k];
            const float g = a.grad_top[row * a.K + k];
            if (i >= 0 && i < a.N && g != 0.0f) {
                c -= g;
                any = true;
            }
        }
        const float l = a.lse[row];
        const float h = gh != 0.0f ? a.entropy[row] : 0.0f;
        for (int64_t n = tid; n < a.N; n += kStatThreads) {
            float d = 0.0f;
            if (any) {
                const float lp = load_elem<DT>(xr, n) - l;
                const float p = ex2(lp * kLog2e);
                d = p * (c - gh * (fmaxf(lp, kFarBelow) + h));
                if (n == t) d += gl;
                for (int k = 0; k < a.K; ++k)
                    if (a.top_index[row * a.K + k] == n) d += a.grad_top[row * a.K + k];
            }
            put_elem<DT>(dr, n, d);
        }
    }
}

unsigned row_grid(int64_t B) { return static_cast<unsigned>(B < INT_MAX ? B : INT_MAX); }

// The checks that the forward and the backward share beyond check_args.
bool misaligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_token_stats(const void* x, lse_dtype dtype, int64_t B, int64_t N, int64_t row_stride,
                           const int64_t* target, int64_t top_k, float* logprob, float* entropy,
                           float* lse_out, float* top_logprob, int64_t* top_index,
                           lse_stream_t stream) {
    const void* stand_in = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
    lse_status st = check_args(x, dtype, B, N, row_stride, stand_in);
    if (st != LSE_OK) return st;
    if (top_k < 0 || top_k > LSE_MAX_TOP_K) return LSE_ERR_INVALID_ARG;
    if (top_k > 0 && N > INT32_MAX) return LSE_ERR_INVALID_ARG;
    if (misaligned(target, 8) || misaligned(top_index, 8) || misaligned(logprob, 4) ||
        misaligned(entropy, 4) || misaligned(lse_out, 4) || misaligned(top_logprob, 4))
        return LSE_ERR_INVALID_ARG;
    if (B == 0) return LSE_OK;
    if ((logprob != nullptr) != (target != nullptr)) return LSE_ERR_INVALID_ARG;
    if (top_k > 0 && (top_logprob == nullptr || top_index == nullptr)) return LSE_ERR_INVALID_ARG;
    if (!logprob && !entropy && !lse_out && top_k == 0) return LSE_ERR_INVALID_ARG;
    StatsArgs a;
    a.x = x;
    a.B = B;
    a.N = N;
    a.row_stride = row_stride;
    a.target = target;
    a.K = static_cast<int>(top_k);
    a.logprob = logprob;
    a.entropy = entropy;
    a.lse = lse_out;
    a.top_logprob = top_logprob;
    a.top_index = top_index;
    const auto kernel = dtype == LSE_F32 ? lse_stats_kernel<kF32>
                        : dtype == LSE_BF16 ? lse_stats_kernel<kBF16> : lse_stats_kernel<kF16>;
    return cuda_status(launch_pdl(kernel, dim3(row_grid(B)), dim3(kStatThreads),
                                  reinterpret_cast<cudaStream_t>(stream), a));
}

lse_status lse_token_stats_backward(const void* x, lse_dtype dtype, int64_t B, int64_t N,
                                    int64_t row_stride, const float* lse_in, const float* entropy,
                                    const int64_t* target, const int64_t* top_index, int64_t top_k,
                                    const float* grad_logprob, const float* grad_entropy,
                                    const float* grad_top, const float* grad_lse, void* dx,
                                    int64_t dx_row_stride, lse_stream_t stream) {
    const void* stand_in = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
    lse_status st = check_args(x, dtype, B, N, row_stride, stand_in);
    if (st != LSE_OK) return st;
    const uintptr_t eb = dtype == LSE_F32 ? 4 : 2;
    int64_t extent = 0;
    if (dx_row_stride < N || top_k < 0 || top_k > LSE_MAX_TOP_K) return LSE_ERR_INVALID_ARG;
    if ((B > 0 && __builtin_mul_overflow(B - 1, dx_row_stride, &extent)) ||
        __builtin_add_overflow(extent, N, &extent) ||
        __builtin_mul_overflow(extent, static_cast<int64_t>(eb), &extent))
        return LSE_ERR_INVALID_ARG;
    if (misaligned(dx, eb) || misaligned(target, 8) || misaligned(top_index, 8) ||
        misaligned(lse_in, 4) || misaligned(entropy, 4) || misaligned(grad_logprob, 4) ||
        misaligned(grad_entropy, 4) || misaligned(grad_top, 4) || misaligned(grad_lse, 4))
        return LSE_ERR_INVALID_ARG;
    if (B == 0 || N == 0) return LSE_OK;
    if (dx == nullptr || lse_in == nullptr) return LSE_ERR_INVALID_ARG;
    if (grad_logprob && !target) return LSE_ERR_INVALID_ARG;
    if (grad_entropy && !entropy) return LSE_ERR_INVALID_ARG;
    if (grad_top && top_k > 0 && !top_index) return LSE_ERR_INVALID_ARG;
    StatsBackwardArgs a;
    a.x = x;
    a.B = B;
    a.N = N;
    a.row_stride = row_stride;
    a.lse = lse_in;
    a.entropy = entropy;
    a.target = target;
    a.top_index = top_index;
    a.K = grad_top ? static_cast<int>(top_k) : 0;
    a.grad_logprob = grad_logprob;
    a.grad_entropy = grad_entropy;
    a.grad_top = grad_top;
    a.grad_lse = grad_lse;
    a.dx = dx;
    a.dx_row_stride = dx_row_stride;
    const auto kernel = dtype == LSE_F32 ? lse_stats_backward_kernel<kF32>
                        : dtype == LSE_BF16 ? lse_stats_backward_kernel<kBF16>
                                            : lse_stats_backward_kernel<kF16>;
    return cuda_status(launch_pdl(kernel, dim3(row_grid(B)), dim3(kStatThreads),
                                  reinterpret_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
