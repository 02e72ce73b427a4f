// lse_stats.cu -- token statistics: the C entry points, and the gradient's kernels
// (sm_103a).  The statistics' own kernels are in lse_stats.cuh.
#include <climits>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_internal.h"
#include "lse_stats_common.cuh"

namespace lse {
namespace {

struct StatsBackwardArgs {
    const void* x;
    int64_t B, N, row_stride;
    const float* lse;
    const float* lse_low;  // may be null (zero)
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
    int64_t seg_slots;  // vectors or elements of a segment
    int64_t segments;   // per row
};

// ---------------------------------------------------------------------------
// Gradient.
//
//     dx_n = p_n (A - gH log p_n) + gl [n = t] + sum_k gt_k [n = i_k],
//     A = g_lse - gl - sum_k gt_k - gH H,   log p_n = (x_n - lse) - lse_low
//
// lse + lse_low is the row value before it was rounded: at an lse of 30000 the rounding
// alone is 1e-3 of every p, and next to the type's lowest value all of log N.  x - lse is
// exact near the maximum, and lse_low enters through the FMA that forms the exponent, so
// both cost no more instructions than lse alone.
//
// TX threads take a segment of a row, two or four vectors each at a time, every load
// issued before the stores.  The few elements with a unit term are read before
// anything is stored and written once more, whole, at the end, so the loop compares no
// columns.  dx may be x, so x is not read through the read-only path: what is loaded
// before a store must not be loaded again after it.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void put_elem(void* row, int64_t i, float v) {
    if constexpr (DT == kF32) static_cast<float*>(row)[i] = v;
    else static_cast<unsigned short*>(row)[i] = static_cast<unsigned short>(pack2<DT>(v, 0.0f));
}

// (in octaves: low = -lse_low log2 e, gh = gH ln 2)
struct RowGrad {
    float lse, low, A, gh;
};

// One pair of elements.  An element with p = 0 adds nothing: log p is bounded from
// below, so that it stays 0 * finite.
template <bool ENT>
__device__ __forceinline__ uint64_t grad_pair(uint64_t x, const RowGrad& g) {
    const uint64_t lp = f2_fma(f2_sub(x, f2_pack(g.lse, g.lse)), f2_pack(kLog2e, kLog2e), f2_pack(g.low, g.low));
    const uint64_t e = f2_ex2(lp);
    if constexpr (!ENT) {
        return f2_mul(e, f2_pack(g.A, g.A));
    } else {
        float l0, l1;
        f2_unpack(lp, l0, l1);
        const uint64_t low = f2_pack(fmaxf(l0, kFarBelow), fmaxf(l1, kFarBelow));
        return f2_mul(e, f2_fma(f2_pack(-g.gh, -g.gh), low, f2_pack(g.A, g.A)));
    }
}

// The same for one element, with what is added to it.
__device__ __forceinline__ float grad_elem(float x, const RowGrad& g, float unit) {
    const float lp = fmaf(x - g.lse, kLog2e, g.low);
    const float e = ex2(lp);
    return (g.gh != 0.0f ? e * fmaf(-g.gh, fmaxf(lp, kFarBelow), g.A) : e * g.A) + unit;
}

template <int DT, bool ENT>
__device__ __forceinline__ uint4 grad_vector(uint4 v, const RowGrad& g) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
    if constexpr (DT == kF32) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float a, b;
            f2_unpack(grad_pair<ENT>(f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1])), g), a, b);
            o[i] = __float_as_uint(a);
            o[i + 1] = __float_as_uint(b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(grad_pair<ENT>(f2_pack(word_lo<DT>(w[i]), word_hi<DT>(w[i])), g), a, b);
            o[i] = pack2<DT>(a, b);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Vectors (or elements) per thread and step.
__host__ __device__ constexpr int grad_u(int TX) { return TX < 32 ? 2 : 4; }
constexpr int kGradCta = 256;    // threads of a CTA whose rows take a warp or less
// Positions in a row: rows that take a warp or less have at most 512 slots.
template <int TX> using GradIndex = typename std::conditional<(TX <= 32), int, int64_t>::type;

// Slots [k0, k1) of a row: the 16-byte vectors that cover it (VEC; x and dx rows at
// the same offset from a boundary), the outer ones stored element by element, or
// single elements.
template <int DT, int TX, bool VEC, bool ENT>
__device__ __forceinline__ void grad_slots(const char* xr, char* dr, int off, GradIndex<TX> end, GradIndex<TX> k0,
                                           GradIndex<TX> k1, int tid, const RowGrad& g) {
    using I = GradIndex<TX>;
    constexpr int EB = DType<DT>::bytes, EPV = 16 / EB;
    constexpr int U = grad_u(TX);
    for (I k = k0 + tid; k < k1; k += U * TX) {
        if constexpr (VEC) {
            const char* x0 = xr - off;
            char* d0 = dr - off;
            uint4 v[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k + j * TX < k1) v[j] = ld_stream16(x0 + (k + j * TX) * 16);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const I kk = k + j * TX;
                if (kk >= k1) continue;
                const uint4 o = grad_vector<DT, ENT>(v[j], g);
                if ((kk > 0 || off == 0) && kk * 16 + 16 <= end) {
                    *reinterpret_cast<uint4*>(d0 + kk * 16) = o;
                } else {
                    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int i = 0; i < EPV; ++i) {
                        const I at = kk * 16 + i * EB;
                        if (at < off || at >= end) continue;
                        if constexpr (DT == kF32) *reinterpret_cast<uint32_t*>(d0 + at) = w[i];
                        else *reinterpret_cast<unsigned short*>(d0 + at) = static_cast<unsigned short>((i & 1) ? w[i / 2] >> 16 : w[i / 2]);
                    }
                }
            }
        } else {
            float v[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k + j * TX < k1) v[j] = load_own_elem<DT>(xr, k + j * TX);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k + j * TX < k1) put_elem<DT>(dr, k + j * TX, grad_elem(v[j], g, 0.0f));
        }
    }
}

// Zeros for the same slots of a row that carries no gradient.
template <int DT, int TX, bool VEC>
__device__ __forceinline__ void zero_slots(char* dr, int off, GradIndex<TX> end, GradIndex<TX> k0, GradIndex<TX> k1, int tid) {
    using I = GradIndex<TX>;
    constexpr int EB = DType<DT>::bytes;
    for (I k = k0 + tid; k < k1; k += TX) {
        if constexpr (!VEC) {
            put_elem<DT>(dr, k, 0.0f);
        } else if ((k > 0 || off == 0) && k * 16 + 16 <= end) {
            *reinterpret_cast<uint4*>(dr - off + k * 16) = make_uint4(0, 0, 0, 0);
        } else {
            for (I at = k * 16; at < k * 16 + 16; at += EB)
                if (at >= off && at < end) put_elem<DT>(dr, (at - off) / EB, 0.0f);
        }
    }
}

// Bound by one read of x and one write of dx: 4096 rows of 32000 bf16 in 72 us, 7.3 TB/s
// (a part of it in L2); 599 of 200003 f32 in 147, 6.5.  Short rows pay for their own gradients, loaded
// in a chain of two trips before the first store (468750 rows of 256 bf16: 103 us, 4.6
// TB/s), which is why several of them share a warp; with 64-bit positions in the row these
// mappings spilled about 110 bytes and took 10 % longer (at most 28 now, none in f32's 8
// and 16 lanes).
template <int DT, int TX, bool VEC>
__global__ void __launch_bounds__(TX <= 32 ? kGradCta : TX, TX < 32 ? 5 : TX == 32 ? 4 : 1024 / TX)
lse_stats_backward_kernel(const __grid_constant__ StatsBackwardArgs a) {
    using I = GradIndex<TX>;
    constexpr int EB = DType<DT>::bytes, UNITS = TX <= 32 ? kGradCta / TX : 1;
    constexpr int W = TX < 32 ? TX : 32;  // lanes that share a row's gradients
    const int tid = threadIdx.x % TX, lane = threadIdx.x & (W - 1);
    const uint32_t group = W == 32 ? 0xffffffffu : ((1u << (W & 31)) - 1) << (threadIdx.x & 31 & ~(W - 1));
    const auto sync = [group] {
        if (TX <= 32) __syncwarp(group);
        else __syncthreads();
    };
    pdl_trigger();
    pdl_wait();
    const int64_t units = a.B * a.segments;
    for (int64_t unit = static_cast<int64_t>(blockIdx.x) * UNITS + threadIdx.x / TX; unit < units;
         unit += static_cast<int64_t>(gridDim.x) * UNITS) {
        const int64_t row = TX <= 32 ? unit : unit / a.segments;  // (a row of up to a warp is one segment)
        const int64_t seg = TX <= 32 ? 0 : unit - row * a.segments;
        const char* xr = static_cast<const char*>(a.x) + row * a.row_stride * EB;
        char* dr = static_cast<char*>(a.dx) + row * a.dx_row_stride * EB;
        const int off = VEC ? static_cast<int>(reinterpret_cast<uintptr_t>(xr) & 15u) : 0;
        const I N = static_cast<I>(a.N);
        const I end = off + N * EB;  // (VEC) bytes from the first vector
        const I slots = VEC ? (end + 15) >> 4 : N;
        const I seg_slots = static_cast<I>(a.seg_slots);
        const I k0 = static_cast<I>(seg) * seg_slots;
        const I k1 = TX <= 32 || k0 + seg_slots >= slots ? slots : k0 + seg_slots;
        if (k0 >= k1) continue;
        // The segment's columns.
        const I n0 = VEC ? (k0 == 0 ? 0 : (k0 * 16 - off) / EB) : k0;
        const I n1 = VEC ? (k1 == slots ? N : (k1 * 16 - off) / EB) : k1;

        // The row's gradients (every group of W lanes for itself; K <= W), all loaded at once.
        RowGrad g;
        g.lse = __ldg(a.lse + row);
        g.low = a.lse_low ? -kLog2e * __ldg(a.lse_low + row) : 0.0f;
        const int64_t given = a.grad_logprob ? __ldg(a.target + row) : -1;
        float gl = a.grad_logprob ? __ldg(a.grad_logprob + row) : 0.0f;
        const float gs = a.grad_lse ? __ldg(a.grad_lse + row) : 0.0f;
        g.gh = a.grad_entropy ? __ldg(a.grad_entropy + row) : 0.0f;
        const float h = a.grad_entropy ? __ldg(a.entropy + row) : 0.0f;
        I ti = -1;  // lane k: alternative k
        float gt = 0.0f;
        if (lane < a.K) {
            const int64_t column = __ldg(a.top_index + row * a.K + lane);
            const bool in = column >= 0 && column < a.N;
            ti = in ? static_cast<I>(column) : -1;
            gt = in ? __ldg(a.grad_top + row * a.K + lane) : 0.0f;
        }
        const bool in_row = given >= 0 && given < a.N;
        const I t = in_row ? static_cast<I>(given) : -1;
        if (!in_row) gl = 0.0f;
        float sum = gt;
        if (a.K > 0) {
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o, W);
        }
        const bool any = gl != 0.0f || gs != 0.0f || g.gh != 0.0f || __any_sync(group, gt != 0.0f);
        if (!any) {
            zero_slots<DT, TX, VEC>(dr, off, end, k0, k1, tid);
            continue;  // (the same for the whole unit)
        }
        g.A = gs - gl - sum;
        if (g.gh != 0.0f) g.A = fmaf(-g.gh, h, g.A);
        g.gh *= kLn2;

        // The first warp keeps the elements with a unit term.
        const bool first = tid < 32;
        const bool mine = first && ti >= n0 && ti < n1;
        float unit_term = 0.0f, x_mine = 0.0f, x_target = 0.0f;
        bool target_alone = false;
        if (first && a.K > 0) {
            for (int k = 0; k < a.K; ++k) {
                const I ok = __shfl_sync(group, ti, k, W);
                const float gk = __shfl_sync(group, gt, k, W);
                if (ok == ti) unit_term += gk;
            }
            if (ti == t && in_row) unit_term += gl;
            if (mine) x_mine = load_own_elem<DT>(xr, ti);
        }
        if (first && in_row && t >= n0 && t < n1) {
            target_alone = !__any_sync(group, ti == t);
            if (target_alone && lane == 0) x_target = load_own_elem<DT>(xr, t);
        }
        sync();
        if (g.gh != 0.0f) grad_slots<DT, TX, VEC, true>(xr, dr, off, end, k0, k1, tid, g);
        else grad_slots<DT, TX, VEC, false>(xr, dr, off, end, k0, k1, tid, g);
        sync();
        if (mine) put_elem<DT>(dr, ti, grad_elem(x_mine, g, unit_term));
        if (target_alone && lane == 0) put_elem<DT>(dr, t, grad_elem(x_target, g, gl));
    }
}

template <int DT, int TX>
cudaError_t launch_stats_backward_tx(const StatsBackwardArgs& a, bool vec, cudaStream_t stream) {
    constexpr int64_t units_per_cta = TX <= 32 ? kGradCta / TX : 1;
    const int64_t ctas = (a.B * a.segments + units_per_cta - 1) / units_per_cta;
    const dim3 grid(static_cast<unsigned>(ctas < INT_MAX ? ctas : INT_MAX)), block(TX <= 32 ? kGradCta : TX);
    return vec ? launch_pdl(lse_stats_backward_kernel<DT, TX, true>, grid, block, stream, a)
               : launch_pdl(lse_stats_backward_kernel<DT, TX, false>, grid, block, stream, a);
}

// Vectors where each x row and its dx row sit at the same offset from a 16-byte
// boundary, elements otherwise.  8, 16 or 32 lanes per row of up to 64, 256 or 512 slots
// (and no more alternatives than lanes), which waste fewer lanes and keep more rows in
// flight (us; 468750 bf16 rows of 256: 8 lanes 103, 16 136, 32 266; 80000 bf16 rows of
// 1500: 16 lanes 98, 32 lanes 100; 39986 bf16 rows of 3001: 16 lanes 100, 32 88, 128
// threads 121; 5000 bf16 rows of 6000: 32 lanes 27, 128 threads 22.4); 128 threads up to 1024
// slots, 256 beyond.  Few rows of more than 256 slots take 128 threads too.  Longer rows
// go in segments of up to 16 slots per thread, shorter ones while the segments would not
// fill the GPU.
template <int DT>
cudaError_t launch_stats_backward(StatsBackwardArgs a, int sms, cudaStream_t stream) {
    const int64_t eb = DType<DT>::bytes;
    const uintptr_t xa = reinterpret_cast<uintptr_t>(a.x), da = reinterpret_cast<uintptr_t>(a.dx);
    const bool vec = (xa - da) % 16 == 0 && ((a.row_stride - a.dx_row_stride) * eb) % 16 == 0;
    const bool aligned = xa % 16 == 0 && (a.row_stride * eb) % 16 == 0;
    const int64_t slots = vec ? (a.N * eb + 15) / 16 + (aligned ? 0 : 1) : a.N;  // at most
    const int TX = slots <= 64 && a.K <= 8                   ? 8
                   : slots <= 256 && a.K <= 16               ? 16
                   : slots <= (a.B >= 8LL * sms ? 512 : 256) ? 32
                   : slots <= 1024                           ? 128
                                                             : 256;
    int64_t steps = 4;
    while (TX > 32 && steps > 1 && a.B * ((slots + steps * grad_u(TX) * TX - 1) / (steps * grad_u(TX) * TX)) * TX < 1024LL * sms)
        --steps;
    a.seg_slots = TX <= 32 ? slots : steps * grad_u(TX) * TX;
    a.segments = (slots + a.seg_slots - 1) / a.seg_slots;
    if (a.B > INT64_MAX / a.segments) return cudaErrorInvalidValue;
    switch (TX) {
    case 8: return launch_stats_backward_tx<DT, 8>(a, vec, stream);
    case 16: return launch_stats_backward_tx<DT, 16>(a, vec, stream);
    case 32: return launch_stats_backward_tx<DT, 32>(a, vec, stream);
    case 128: return launch_stats_backward_tx<DT, 128>(a, vec, stream);
    default: return launch_stats_backward_tx<DT, 256>(a, vec, stream);
    }
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_token_stats(const void* x, lse_dtype dtype, int64_t B, int64_t N, int64_t row_stride,
                           const int64_t* target, int64_t top_k, float* logprob, float* entropy,
                           float* lse_out, float* top_logprob, int64_t* top_index,
                           lse_stream_t stream) {
    return lse_token_stats_pair(x, dtype, B, N, row_stride, target, top_k, logprob, entropy, lse_out, nullptr,
                                top_logprob, top_index, stream);
}

lse_status lse_token_stats_pair(const void* x, lse_dtype dtype, int64_t B, int64_t N, int64_t row_stride,
                                const int64_t* target, int64_t top_k, float* logprob, float* entropy,
                                float* lse_out, float* lse_low, float* top_logprob, int64_t* top_index,
                                lse_stream_t stream) {
    const void* stand_in = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
    lse_status st = check_args(x, dtype, B, N, row_stride, stand_in);
    if (st != LSE_OK) return st;
    if (top_k < 0 || top_k > LSE_MAX_TOP_K) return LSE_ERR_INVALID_ARG;
    if (top_k > 0 && N > INT32_MAX) return LSE_ERR_INVALID_ARG;
    if (misaligned(target, 8) || misaligned(top_index, 8) || misaligned(logprob, 4) ||
        misaligned(entropy, 4) || misaligned(lse_out, 4) || misaligned(lse_low, 4) || misaligned(top_logprob, 4))
        return LSE_ERR_INVALID_ARG;
    if (B == 0) return LSE_OK;
    if ((logprob != nullptr) != (target != nullptr)) return LSE_ERR_INVALID_ARG;
    if (top_k > 0 && (top_logprob == nullptr || top_index == nullptr)) return LSE_ERR_INVALID_ARG;
    if (!logprob && !entropy && !lse_out && !lse_low && top_k == 0) return LSE_ERR_INVALID_ARG;
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
    a.lse_low = lse_low;
    a.top_logprob = top_logprob;
    a.top_index = top_index;
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N > 1024 && B > INT_MAX) return LSE_ERR_INVALID_ARG;  // a CTA per row
    return cuda_status(dtype == LSE_F32 ? launch_token_stats_f32(a, sms, s)
                       : dtype == LSE_BF16 ? launch_token_stats_bf16(a, sms, s) : launch_token_stats_f16(a, sms, s));
}

lse_status lse_token_stats_backward(const void* x, lse_dtype dtype, int64_t B, int64_t N,
                                    int64_t row_stride, const float* lse_in, const float* entropy,
                                    const int64_t* target, const int64_t* top_index, int64_t top_k,
                                    const float* grad_logprob, const float* grad_entropy,
                                    const float* grad_top, const float* grad_lse, void* dx,
                                    int64_t dx_row_stride, lse_stream_t stream) {
    return lse_token_stats_backward_pair(x, dtype, B, N, row_stride, lse_in, nullptr, entropy, target, top_index, top_k,
                                         grad_logprob, grad_entropy, grad_top, grad_lse, dx, dx_row_stride, stream);
}

lse_status lse_token_stats_backward_pair(const void* x, lse_dtype dtype, int64_t B, int64_t N,
                                         int64_t row_stride, const float* lse_in, const float* lse_low,
                                         const float* entropy, const int64_t* target,
                                         const int64_t* top_index, int64_t top_k,
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
        misaligned(lse_in, 4) || misaligned(lse_low, 4) || misaligned(entropy, 4) || misaligned(grad_logprob, 4) ||
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
    a.lse_low = lse_low;
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
    int sms = 0;
    if ((st = device_sms(&sms)) != LSE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(dtype == LSE_F32 ? launch_stats_backward<kF32>(a, sms, s)
                       : dtype == LSE_BF16 ? launch_stats_backward<kBF16>(a, sms, s)
                                           : launch_stats_backward<kF16>(a, sms, s));
}

}  // extern "C"
