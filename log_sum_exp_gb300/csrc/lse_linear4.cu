// lse_linear4.cu -- matrices held in 4 bits with a scale for each group of columns: into that
// form, back, and products of a few tokens with them (sm_103a).
//
//     s[n, g] = max |w| over the group / 7     q = round(w / s)     w ~ q s,  q in -8 .. 7
//     y[t, n] = sum_g s[n, g] sum_{k in g} x[t, k] q[n, k]
//
// Form.  A row's columns come in blocks of 128, 64 bytes each: byte 16 c + 4 w of a block
// starts the 32-bit word of columns 32 w + 8 c .. + 7, so the four lanes of a matrix
// instruction that share a row read 16 bytes each and each word of theirs lies in the same
// group of 32 columns.  Within a word, nibble i holds q + 8 of column 2 i and nibble i + 4 that
// of column 2 i + 1: one mask takes out two neighbours as the halves of a register.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"
#include "lse_linear4_common.cuh"

namespace lse {
namespace {

// Where the word of columns 8 j .. 8 j + 7 lies in its row.
__device__ __forceinline__ int64_t word_bytes(int64_t j) {
    const int r = static_cast<int>(j & 15);
    return (j >> 4) * kBlockBytes + (r & 3) * 16 + (r >> 2) * 4;
}
// Codes (0 .. 15) of eight neighbours to a word.
__device__ __forceinline__ uint32_t pack_word(const int (&c)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= static_cast<uint32_t>(c[i]) << (i / 2 * 4 + (i % 2) * 16);
    return w;
}

struct FormArgs {
    const void* in;  // matrix, or int8 values
    int64_t N, K, in_stride;
    int group;
    uint32_t* codes;
    void* scales;
    int64_t scale_stride;
    void* out;  // read back
    int64_t out_stride;
    bool vec;  // rows of the matrix start on 16-byte boundaries
};

constexpr int kFormThreads = 256;
constexpr int kFormWords = 2;  // words of a lane in flight

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// w / s to the nearest whole number, halves to even, without a division: the quotient by
// the reciprocal is off by less than 1e-5 for |w / s| <= 12, so only one next to a half needs
// the remainder w - q s, which is exact (both terms are multiples of the smaller one's last
// bit, and it is no larger than s).
__device__ __forceinline__ int nearest(float w, float s, float inv) {
    const float t = w * inv;
    float q = rintf(t);
    if (fabsf(t - q) > 0.499f) {
        const float r = fmaf(-q, s, w), h = 0.5f * s;
        if (fabsf(r) > h || (fabsf(r) == h && (static_cast<int>(q) & 1))) q += copysignf(1.0f, r);
    }
    return static_cast<int>(fminf(fmaxf(q, -8.0f), 7.0f));
}

// A warp takes 32 words of a row kFormWords times over; the lanes of a group find its largest
// magnitude with shuffles.
template <int DT> __global__ void __launch_bounds__(kFormThreads) quantize4_kernel(FormArgs a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t words = blocks_of(a.K) * kBlockWords;
    const int64_t per_row = (words + 32 * kFormWords - 1) / (32 * kFormWords);
    const int64_t units = a.N * per_row;
    const int64_t groups = (a.K + a.group - 1) / a.group;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kFormThreads + threadIdx.x) >> 5; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kFormThreads / 32)) {
        const int64_t n = u / per_row, j0 = (u - n * per_row) * 32 * kFormWords + lane;
        const char* row = static_cast<const char*>(a.in) + n * a.in_stride * DType<DT>::bytes;
        float f[kFormWords][8];
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) load8<DT>(row, (j0 + 32 * v) * 8, a.K, a.vec, f[v]);
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int64_t j = j0 + 32 * v;
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(f[v][i]));
            for (int o = a.group / 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            // A group with a NaN or an infinity has no scale: it reads back as NaN.
            float s = m <= 3.4028235e38f ? __fdiv_rn(m, 7.0f) : __int_as_float(0x7fffffff);
            if constexpr (DT != kF32) s = word_lo<DT>(pack2<DT>(s, 0.0f));
            const int64_t k = j * 8;
            if (k % a.group == 0 && k / a.group < groups) {
                const int64_t at = n * a.scale_stride + k / a.group;
                if constexpr (DT == kF32) static_cast<float*>(a.scales)[at] = s;
                else static_cast<unsigned short*>(a.scales)[at] = static_cast<unsigned short>(pack2<DT>(s, 0.0f));
            }
            if (j >= words) continue;
            int c[8];
            if (s > 0.0f) {
                const float up = s < 0x1p-60f ? 0x1p64f : 1.0f;  // the reciprocal of a small scale overflows
                const float su = s * up, inv = __fdiv_rn(1.0f, su);
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = nearest(f[v][i] * up, su, inv) + 8;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = 8;
            }
            a.codes[n * words + word_bytes(j) / 4] = pack_word(c);
        }
    }
}

// Values -8 .. 7 (larger ones are cut off) to codes.
__global__ void __launch_bounds__(kFormThreads) pack4_kernel(FormArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t words = blocks_of(a.K) * kBlockWords, all = a.N * words;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kFormThreads + threadIdx.x; u < all;
         u += static_cast<int64_t>(gridDim.x) * kFormThreads) {
        const int64_t n = u / words, j = u - n * words;
        const signed char* row = static_cast<const signed char*>(a.in) + n * a.in_stride;
        int c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int q = j * 8 + i < a.K ? row[j * 8 + i] : 0;
            c[i] = (q < -8 ? -8 : q > 7 ? 7 : q) + 8;
        }
        a.codes[n * words + word_bytes(j) / 4] = pack_word(c);
    }
}

template <int DT> __global__ void __launch_bounds__(kFormThreads) dequantize4_kernel(FormArgs a) {
    constexpr int EB = DType<DT>::bytes;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t words = blocks_of(a.K) * kBlockWords;
    const int64_t per_row = (words + 32 * kFormWords - 1) / (32 * kFormWords);
    const int64_t units = a.N * per_row;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kFormThreads + threadIdx.x) >> 5; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kFormThreads / 32)) {
        const int64_t n = u / per_row, j0 = (u - n * per_row) * 32 * kFormWords + lane;
        char* row = static_cast<char*>(a.out) + n * a.out_stride * EB;
        uint32_t w[kFormWords];
        float s[kFormWords];
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int64_t j = j0 + 32 * v, k = j * 8;
            w[v] = 0;
            s[v] = 0.0f;
            if (k >= a.K) continue;
            w[v] = __ldg(a.codes + n * words + word_bytes(j) / 4);
            s[v] = load_elem<DT>(a.scales, n * a.scale_stride + k / a.group);
        }
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int64_t k = (j0 + 32 * v) * 8;
            if (k >= a.K) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = static_cast<float>(static_cast<int>(w[v] >> (i / 2 * 4 + (i % 2) * 16) & 15) - 8) * s[v];
            if (a.vec && k + 8 <= a.K) {
                if constexpr (DT == kF32) {
                    *reinterpret_cast<float4*>(row + k * 4) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4*>(row + k * 4 + 16) = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                    *reinterpret_cast<uint4*>(row + k * 2) = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]),
                                                                        pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (k + i >= a.K) continue;
                    if constexpr (DT == kF32) reinterpret_cast<float*>(row)[k + i] = f[i];
                    else reinterpret_cast<unsigned short*>(row)[k + i] = static_cast<unsigned short>(pack2<DT>(f[i], 0.0f));
                }
            }
        }
    }
}

template <class F> cudaError_t by_type(int dtype, F&& f) {
    return dtype == LSE_F32 ? f(IntConst<kF32>{}) : dtype == LSE_BF16 ? f(IntConst<kBF16>{}) : f(IntConst<kF16>{});
}

bool extent_fits(int64_t rows, int64_t stride, int64_t bytes) {
    int64_t e = 0;
    return !__builtin_mul_overflow(rows, stride, &e) && !__builtin_mul_overflow(e, bytes, &e);
}

// The held form: sizes, group and the arrays' alignment.
lse_status check_form(int64_t N, int64_t K, int64_t group, const void* codes, const void* scales, int scale_dtype,
                      int64_t scale_stride) {
    if (!valid_dtype(scale_dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || K < 0 || K > INT32_MAX - kBlock || (group != 32 && group != 64 && group != 128)) return LSE_ERR_INVALID_ARG;
    if (!extent_fits(N, blocks_of(K) * kBlock, 4)) return LSE_ERR_INVALID_ARG;
    const uintptr_t sb = scale_dtype == LSE_F32 ? 4 : 2;
    if (misaligned(codes, 16) || misaligned(scales, sb) || !extent_fits(N, scale_stride, sb)) return LSE_ERR_INVALID_ARG;
    if (scale_stride < (K + group - 1) / group) return LSE_ERR_INVALID_ARG;
    if (N > 0 && K > 0 && (!codes || !scales)) return LSE_ERR_INVALID_ARG;
    return LSE_OK;
}

lse_status check_matrix(const void* p, int dtype, int64_t N, int64_t K, int64_t stride, int64_t eb) {
    if (dtype >= 0 && !valid_dtype(dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (stride < K || misaligned(p, static_cast<uintptr_t>(eb)) || !extent_fits(N, stride, eb)) return LSE_ERR_INVALID_ARG;
    return N > 0 && K > 0 && !p ? LSE_ERR_INVALID_ARG : LSE_OK;
}

unsigned form_grid(int64_t N, int64_t K, int sms, int64_t words_per_thread) {
    const int64_t words = blocks_of(K) * kBlockWords;
    const int64_t per_row = (words + 32 * words_per_thread - 1) / (32 * words_per_thread);
    int64_t ctas = (N * per_row + kFormThreads / 32 - 1) / (kFormThreads / 32);
    const int64_t most = static_cast<int64_t>(sms) * 8;
    return static_cast<unsigned>(ctas > most ? most : ctas);
}

FormArgs form_args(int64_t N, int64_t K, int64_t group, const void* codes, const void* scales, int64_t scale_stride) {
    FormArgs a = {};
    a.N = N;
    a.K = K;
    a.group = static_cast<int>(group);
    a.codes = static_cast<uint32_t*>(const_cast<void*>(codes));
    a.scales = const_cast<void*>(scales);
    a.scale_stride = scale_stride;
    return a;
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_quantize4(const void* w, lse_dtype dtype, int64_t N, int64_t K, int64_t w_stride, int64_t group,
                         void* codes, void* scales, int64_t scale_stride, lse_stream_t stream) {
    if (!valid_dtype(dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    lse_status st = check_form(N, K, group, codes, scales, dtype, scale_stride);
    if (st == LSE_OK) st = check_matrix(w, dtype, N, K, w_stride, eb);
    if (st != LSE_OK || N == 0 || K == 0) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    FormArgs a = form_args(N, K, group, codes, scales, scale_stride);
    a.in = w;
    a.in_stride = w_stride;
    a.vec = !misaligned(w, 16) && w_stride * eb % 16 == 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(by_type(dtype, [&](auto dt) {
        return launch_pdl(quantize4_kernel<decltype(dt)::value>, dim3(form_grid(N, K, sms, kFormWords)), dim3(kFormThreads), s, a);
    }));
}

lse_status lse_pack4(const signed char* values, int64_t N, int64_t K, int64_t values_stride, void* codes, lse_stream_t stream) {
    lse_status st = check_form(N, K, 128, codes, codes, LSE_F32, blocks_of(K < 0 ? 0 : K));
    if (st == LSE_OK) st = check_matrix(values, -1, N, K, values_stride, 1);
    if (st != LSE_OK || N == 0 || K == 0) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    FormArgs a = form_args(N, K, 128, codes, nullptr, 0);
    a.in = values;
    a.in_stride = values_stride;
    return cuda_status(launch_pdl(pack4_kernel, dim3(form_grid(N, K, sms, 1)), dim3(kFormThreads),
                                  reinterpret_cast<cudaStream_t>(stream), a));
}

lse_status lse_dequantize4(const void* codes, const void* scales, lse_dtype dtype, int64_t scale_stride, int64_t N,
                           int64_t K, int64_t group, void* out, int64_t out_stride, lse_stream_t stream) {
    if (!valid_dtype(dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    lse_status st = check_form(N, K, group, codes, scales, dtype, scale_stride);
    if (st == LSE_OK) st = check_matrix(out, dtype, N, K, out_stride, eb);
    if (st != LSE_OK || N == 0 || K == 0) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    FormArgs a = form_args(N, K, group, codes, scales, scale_stride);
    a.out = out;
    a.out_stride = out_stride;
    a.vec = !misaligned(out, 16) && out_stride * eb % 16 == 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(by_type(dtype, [&](auto dt) {
        return launch_pdl(dequantize4_kernel<decltype(dt)::value>, dim3(form_grid(N, K, sms, kFormWords)), dim3(kFormThreads), s, a);
    }));
}

lse_status lse_linear4(const void* x, lse_dtype dtype, int64_t T, int64_t K, int64_t x_stride, const void* codes,
                       const void* scales, lse_dtype scale_dtype, int64_t scale_stride, int64_t N, int64_t group,
                       void* out, lse_dtype out_dtype, int64_t out_stride, lse_stream_t stream) {
    if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (out_dtype != dtype && out_dtype != LSE_F32) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    lse_status st = check_form(N, K, group, codes, scales, scale_dtype, scale_stride);
    if (T < 0 || T > 65535 * 8LL) return LSE_ERR_INVALID_ARG;
    if (st == LSE_OK) st = check_matrix(x, dtype, T, K, x_stride, eb);
    if (st == LSE_OK) st = check_matrix(out, out_dtype, T, N, out_stride, out_dtype == LSE_F32 ? 4 : 2);
    if (st != LSE_OK || T == 0 || N == 0) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    LinearArgs a = {};
    a.x = x;
    a.T = T;
    a.x_stride = x_stride;
    a.K = static_cast<int>(K);
    a.blocks = static_cast<int>(blocks_of(K));
    a.groups = static_cast<int>((K + group - 1) / group);
    a.codes = static_cast<const uint4*>(codes);
    a.scales = scales;
    a.scale_dtype = scale_dtype;
    a.scale_stride = scale_stride;
    a.N = N;
    a.out = out;
    a.out_stride = out_stride;
    a.out_f32 = out_dtype == LSE_F32;
    a.x_vec = !misaligned(x, 16) && x_stride * eb % 16 == 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.group = static_cast<int>(group);
    return cuda_status(dtype == LSE_F32 ? launch_linear4_f32(a, sms, s)
                       : dtype == LSE_BF16 ? launch_linear4_bf16(a, sms, s) : launch_linear4_f16(a, sms, s));
}

}  // extern "C"
