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
//
// Into the form and back are bound by memory in f32 on 16-byte boundaries (32000 x 4096: 96 us, 5.9
// TB/s of 0.59 GB), by single-element loads through shared memory off them (50257 x 1001: 73 us, 44 %
// of the memory's rate) and by instructions in 16 bits (128256 x 2048 bf16: 228 us, 2.9 TB/s of 0.66
// GB); back 143 us, mostly writes.  Products: lse_linear4.cuh.
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
    int group_log2;
    uint32_t* codes;
    void* scales;
    int64_t scale_stride;
    void* out;  // read back
    int64_t out_stride;
    bool vec;  // rows of the matrix start on 16-byte boundaries
};

constexpr int kFormThreads = 256;
constexpr int kFormWords = 4;  // words of a lane in flight
constexpr int kWarpColumns = 256;  // of 32 words

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// w / s to the nearest whole number, halves to even, with the remainder of a first guess, which
// is exact (both terms are multiples of the smaller one's last bit, and it is no larger than s).
// (By value: through a pointer the words would live in memory.)
__device__ __noinline__ uint32_t nearest_codes(float4 fa, float4 fb, float s) {
    const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
    const float up = s < 0x1p-60f ? 0x1p64f : 1.0f;  // the reciprocal of a small scale overflows
    const float su = s * up, inv = __fdiv_rn(1.0f, su);
    int c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float w = f[i] * up;
        float q = rintf(fminf(fmaxf(w * inv, -16.0f), 16.0f));
        const float r = fmaf(-q, su, w), h = 0.5f * su;
        if (fabsf(r) > h || (fabsf(r) == h && (static_cast<int>(q) & 1))) q += copysignf(1.0f, r);
        c[i] = static_cast<int>(fminf(fmaxf(q, -8.0f), 7.0f)) + 8;
    }
    return pack_word(c);
}

// Rows off a 16-byte boundary pass through shared memory, so that a warp's accesses to them are
// next to each other: `columns` elements from column k on to or from 32 lanes of eight.
template <int DT> __device__ __forceinline__ void load_row_part(const void* row, int64_t k, int64_t K, bool vec, float* stage, float (&f)[8]) {
    const int lane = threadIdx.x & 31;
    if (vec) {
        load8<DT>(row, k + lane * 8, K, true, f);
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t at = k + i * 32 + lane;
        stage[i * 32 + lane] = at < K ? load_elem<DT>(row, at) : 0.0f;
    }
    __syncwarp();
    const float4 a = *reinterpret_cast<const float4*>(stage + lane * 8), b = *reinterpret_cast<const float4*>(stage + lane * 8 + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <int DT> __device__ __forceinline__ void store_row_part(void* row, int64_t k, int64_t K, bool vec, float* stage, const float (&f)[8]) {
    const int lane = threadIdx.x & 31;
    if (vec && k + lane * 8 + 8 <= K) {
        char* p = static_cast<char*>(row) + (k + lane * 8) * DType<DT>::bytes;
        if constexpr (DT == kF32) {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(p + 16) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
        }
        return;
    }
    const auto put = [&](int64_t at, float v) {
        if (at >= K) return;
        if constexpr (DT == kF32) static_cast<float*>(row)[at] = v;
        else static_cast<unsigned short*>(row)[at] = static_cast<unsigned short>(pack2<DT>(v, 0.0f));
    };
    if (vec) {  // the row's end
#pragma unroll
        for (int i = 0; i < 8; ++i) put(k + lane * 8 + i, f[i]);
        return;
    }
    __syncwarp();
    *reinterpret_cast<float4*>(stage + lane * 8) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(stage + lane * 8 + 4) = make_float4(f[4], f[5], f[6], f[7]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) put(k + i * 32 + lane, stage[i * 32 + lane]);
}

// A warp takes 256 columns of a row kFormWords times over; the lanes of a group find its largest
// magnitude with shuffles.  About 14 instructions per element and lane, where the memory's rate
// leaves about six for 16-bit weights (39 % of it is reached): a quotient is rounded by adding it to a number whose
// last bit counts 1 (its low bits are then the code).  Quotients of 16-bit numbers are often exact
// halves, and 2^-13 away from one otherwise (2 w - (2 k + 1) s is a multiple of half the last bit of
// an 11-bit s): one correction by the remainder brings them to 2^-22 and exact halves out exactly.
// Of f32, words with a quotient within 4e-6 of a half, where the reciprocal's error could matter, are
// done again with exact remainders, and so are those of scales below the type's normal range, whose
// rounding may leave quotients beyond 7.
template <int DT> __global__ void __launch_bounds__(kFormThreads) quantize4_kernel(FormArgs a) {
    __shared__ __align__(16) float stage[kFormThreads / 32][kWarpColumns];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = static_cast<int>(blocks_of(a.K) * kBlockWords);
    const int per_row = (words + 32 * kFormWords - 1) / (32 * kFormWords);
    const int64_t units = a.N * per_row;
    const int groups = static_cast<int>((a.K + (1 << a.group_log2) - 1) >> a.group_log2);
    const int span = 1 << (a.group_log2 - 3);  // lanes of a group
    constexpr float least = DT == kF16 ? 0x1p-14f : 0x1p-100f;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kFormThreads / 32) + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kFormThreads / 32)) {
        const int64_t n = u / per_row;
        const int j0 = static_cast<int>(u - n * per_row) * 32 * kFormWords + lane;
        const char* row = static_cast<const char*>(a.in) + n * a.in_stride * DType<DT>::bytes;
        float f[kFormWords][8];
#pragma unroll
        for (int v = 0; v < kFormWords; ++v)
            load_row_part<DT>(row, static_cast<int64_t>(j0 - lane + 32 * v) * 8, a.K, a.vec, stage[warp], f[v]);
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int j = j0 + 32 * v;
            float m = fabsf(f[v][0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[v][i]));
            for (int o = span / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            // A group with a NaN or an infinity has no scale: it reads back as NaN.
            float s = m <= 3.4028235e38f ? __fdiv_rn(m, 7.0f) : __int_as_float(0x7fffffff);
            if constexpr (DT != kF32) s = word_lo<DT>(pack2<DT>(s, 0.0f));
            const int grp = j >> (a.group_log2 - 3);
            if ((j & (span - 1)) == 0 && grp < groups) {
                const int64_t at = n * a.scale_stride + grp;
                if constexpr (DT == kF32) static_cast<float*>(a.scales)[at] = s;
                else static_cast<unsigned short*>(a.scales)[at] = static_cast<unsigned short>(pack2<DT>(s, 0.0f));
            }
            if (j >= words) continue;
            uint32_t w = 0x88888888u;
            if (s > 0.0f) {
                const float inv = __fdividef(1.0f, s), magic = 12582920.0f;  // 1.5 2^23 + 8
                float far = 0.0f;
                w = 0;
                const uint64_t inv2 = f2_pack(inv, inv), minus_s2 = f2_pack(-s, -s), magic2 = f2_pack(magic, magic);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint64_t x = f2_pack(f[v][i], f[v][i + 1]);
                    uint64_t t = f2_mul(x, inv2);
                    if constexpr (DT != kF32) {
                        t = f2_fma(f2_fma(t, minus_s2, x), inv2, t);
                    }
                    const uint64_t k = f2_add(t, magic2);
                    float k0, k1;
                    f2_unpack(k, k0, k1);
                    if constexpr (DT == kF32) {
                        float d0, d1;
                        f2_unpack(f2_sub(t, f2_sub(k, magic2)), d0, d1);
                        far = fmaxf(far, fmaxf(fabsf(d0), fabsf(d1)));
                    }
                    const uint32_t p = __byte_perm(__float_as_uint(k0), __float_as_uint(k1), 0x5410);
                    w |= (p & 0x000f000fu) << (2 * i);
                }
                if (far > 0.499996f || s < least) 
                    w = nearest_codes(make_float4(f[v][0], f[v][1], f[v][2], f[v][3]), make_float4(f[v][4], f[v][5], f[v][6], f[v][7]), s);
            }
            a.codes[n * words + word_bytes(j) / 4] = w;
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
    __shared__ __align__(16) float stage[kFormThreads / 32][kWarpColumns];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = static_cast<int>(blocks_of(a.K) * kBlockWords);
    const int per_row = (words + 32 * kFormWords - 1) / (32 * kFormWords);
    const int64_t units = a.N * per_row;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kFormThreads / 32) + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kFormThreads / 32)) {
        const int64_t n = u / per_row;
        const int j0 = static_cast<int>(u - n * per_row) * 32 * kFormWords + lane;
        char* row = static_cast<char*>(a.out) + n * a.out_stride * DType<DT>::bytes;
        uint32_t w[kFormWords];
        float s[kFormWords];
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int j = j0 + 32 * v;
            w[v] = 0;
            s[v] = 0.0f;
            if (static_cast<int64_t>(j) * 8 >= a.K) continue;
            w[v] = __ldg(a.codes + n * words + word_bytes(j) / 4);
            s[v] = load_elem<DT>(a.scales, n * a.scale_stride + (j >> (a.group_log2 - 3)));
        }
#pragma unroll
        for (int v = 0; v < kFormWords; ++v) {
            const int64_t k = static_cast<int64_t>(j0 - lane + 32 * v) * 8;  // of the warp
            if (k >= a.K) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // 2^23 + q + 8, less 2^23 + 8
                const uint32_t c = w[v] >> (i / 2 * 4 + (i % 2) * 16) & 15u;
                f[i] = (__uint_as_float(c | 0x4b000000u) - 8388616.0f) * s[v];
            }
            store_row_part<DT>(row, k, a.K, a.vec, stage[warp], f);
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
    a.group_log2 = group == 32 ? 5 : group == 64 ? 6 : 7;
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
