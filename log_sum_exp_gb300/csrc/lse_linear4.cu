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
// Products.  Bound by reading the codes: half a byte per weight leaves about three
// instructions per weight and lane at the memory's rate, so the weights do not go through
// scalar arithmetic.  A pair of nibbles becomes a pair of 16-bit floats, exactly q, by an or
// with the bits of 1024 (bf16: 128) and a subtraction, and mma.sync multiplies 16 rows x 16
// columns with 8 tokens, summing in f32.  The scale multiplies a group's f32 sum, so nothing
// but the result is rounded to 16 bits.  f32 tokens are cut into three bf16 parts (8 + 8 + 8
// bits, exact) that are three more columns of the product.  tcgen05 would need the
// weights' floats in shared memory, four times the codes' bytes through it and back, to win
// a product that takes less than a tenth of the time here; the tokens are few.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"

namespace lse {
namespace {

constexpr int kBlock = 128;       // columns of a block of codes
constexpr int kBlockBytes = 64;
constexpr int kBlockWords = 16;

__host__ __device__ __forceinline__ int64_t blocks_of(int64_t K) { return (K + kBlock - 1) / kBlock; }
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

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
struct LinearArgs {
    const void* x;
    int64_t T, x_stride;
    int K, blocks, groups;
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
};

template <bool F16> __device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (F16) asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The eight values of a word as four pairs of columns.
template <bool F16> __device__ __forceinline__ void word_pairs(uint32_t w, uint32_t (&p)[4]) {
    if constexpr (F16) {
        // 1024 + q + 8 has its last bit at 1; in the second nibble the code counts 16 times,
        // and (1024 + 16 (q + 8)) / 16 - 72 = q without a shift.
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t v = i ? w >> 8 : w;
            p[i] = sub2<true>((v & 0x000f000fu) | 0x64006400u, 0x64086408u);
            asm("fma.rn.f16x2 %0, %1, %2, %3;"
                : "=r"(p[i + 1])
                : "r"((v & 0x00f000f0u) | 0x64006400u), "r"(0x2c002c00u), "r"(0xd480d480u));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = sub2<false>((w >> (4 * i) & 0x000f000fu) | 0x43004300u, 0x43084308u);
    }
}

// c += a (16 x 16) b (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float scale_at(const LinearArgs& a, int64_t i) {
    if (a.scale_dtype == kF32) return __ldg(static_cast<const float*>(a.scales) + i);
    return a.scale_dtype == kBF16 ? load_elem<kBF16>(a.scales, i) : load_elem<kF16>(a.scales, i);
}

// The part of x that a chunk needs, as 16-bit floats: PL planes of `tokens` rows.
template <int DT>
__device__ __forceinline__ void stage_tokens(const LinearArgs& a, int64_t t0, int b0, int nb, unsigned char* smem) {
    const int cols = nb * kBlock, k0 = b0 * kBlock;
    const int plane = a.tokens * a.row_bytes;
    const int per_row = cols / 8;
    for (int i = threadIdx.x; i < a.tokens * per_row; i += blockDim.x) {
        const int t = i / per_row, v = i - t * per_row;
        const int k = k0 + v * 8;
        unsigned char* to = smem + t * a.row_bytes + v * 16;
        const char* row = static_cast<const char*>(a.x) + (t0 + t) * a.x_stride * DType<DT>::bytes;
        const bool live = t0 + t < a.T;
        if constexpr (DT == kF32) {
            float f[8];
            load8<kF32>(row, k, live ? a.K : 0, a.x_vec, f);
            uint32_t h[4], m[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t part[3][2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    // Cut off, not rounded, so that no part overflows; nothing is left of an
                    // infinity or a NaN.
                    float r = f[2 * e + s];
                    const bool finite = fabsf(r) <= 3.4028235e38f;
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        const uint32_t top = __float_as_uint(r) & 0xffff0000u;
                        part[q][s] = (q == 0 && r != r) ? 0x7fc00000u : top;
                        r = finite ? r - __uint_as_float(top) : 0.0f;
                    }
                }
                h[e] = part[0][0] >> 16 | part[0][1];
                m[e] = part[1][0] >> 16 | part[1][1];
                l[e] = part[2][0] >> 16 | part[2][1];
            }
            *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(to + plane) = make_uint4(m[0], m[1], m[2], m[3]);
            *reinterpret_cast<uint4*>(to + 2 * plane) = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
            uint4 v4 = make_uint4(0, 0, 0, 0);
            if (live && a.x_vec && k + 8 <= a.K) {
                v4 = __ldg(reinterpret_cast<const uint4*>(row + static_cast<int64_t>(k) * 2));
            } else if (live) {
                const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = (k + 2 * e < a.K ? __ldg(r + k + 2 * e) : 0u) |
                           (k + 2 * e + 1 < a.K ? static_cast<uint32_t>(__ldg(r + k + 2 * e + 1)) << 16 : 0u);
                v4 = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4*>(to) = v4;
        }
    }
}

// NT groups of 8 tokens; NS groups of columns in a block; RT tiles of 16 rows per warp; KS
// warps share the columns of a tile; W warps in a CTA; U blocks of codes in flight.
template <int DT, int NT, int NS, int RT, int KS, int W, int U>
__global__ void __launch_bounds__(32 * W) linear4_kernel(LinearArgs a) {
    constexpr bool F16 = DT == kF16;
    constexpr int PL = DT == kF32 ? 3 : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int ks = warp % KS;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 8 * NT;
    const int plane = a.tokens * a.row_bytes;
    float* red = reinterpret_cast<float*>(smem + PL * plane);
    bool staged = false;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (W / KS); first < a.tiles;
         first += static_cast<int64_t>(gridDim.x) * (W / KS)) {
        const int64_t tile = first + warp / KS;
        int64_t row[RT][2];
        const uint4* codes[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                row[r][h] = (tile * RT + r) * 16 + h * 8 + g;
                const int64_t in = row[r][h] < a.N ? row[r][h] : a.N - 1;  // rows behind the last are computed and not stored
                codes[r][h] = a.codes + in * a.blocks * 4 + c;
            }
        float acc[RT][NT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.0f;
        for (int b0 = 0; b0 < a.blocks; b0 += a.chunk_blocks) {
            const int nb = min(a.chunk_blocks, a.blocks - b0);
            if (!staged || a.chunk_blocks < a.blocks) {
                __syncthreads();
                stage_tokens<DT>(a, t0, b0, nb, smem);
                __syncthreads();
                staged = true;
            }
            for (int b = ks; b < nb; b += KS * U) {
                uint4 q[U][RT][2];
                float s[U][RT][2][NS];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int bb = b + u * KS;
                    if (bb >= nb) continue;
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            q[u][r][h] = ldg_stream16(codes[r][h] + static_cast<int64_t>(b0 + bb) * 4);
                            const int64_t in = row[r][h] < a.N ? row[r][h] : a.N - 1;
#pragma unroll
                            for (int i = 0; i < NS; ++i) {
                                const int grp = (b0 + bb) * NS + i;
                                s[u][r][h][i] = grp < a.groups ? scale_at(a, in * a.scale_stride + grp) : 0.0f;
                            }
                        }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int bb = b + u * KS;
                    if (bb >= nb) continue;
                    float part[RT][NT][4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        if (w % (4 / NS) == 0) {
#pragma unroll
                            for (int r = 0; r < RT; ++r)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) part[r][n][i] = 0.0f;
                        }
                        uint32_t p[RT][2][4];
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 v = q[u][r][h];
                                word_pairs<F16>(w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w, p[r][h]);
                            }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
#pragma unroll
                            for (int l = 0; l < PL; ++l) {
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (n * 8 + g < a.tokens)
                                    x = *reinterpret_cast<const uint4*>(smem + l * plane + (n * 8 + g) * a.row_bytes +
                                                                        bb * (kBlock * 2) + w * 64 + c * 16);
#pragma unroll
                                for (int r = 0; r < RT; ++r) {
                                    mma<F16>(part[r][n], p[r][0][0], p[r][1][0], p[r][0][1], p[r][1][1], x.x, x.y);
                                    mma<F16>(part[r][n], p[r][0][2], p[r][1][2], p[r][0][3], p[r][1][3], x.z, x.w);
                                }
                            }
                        }
                        if (w % (4 / NS) == 4 / NS - 1) {
#pragma unroll
                            for (int r = 0; r < RT; ++r)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        acc[r][n][i] = fmaf(s[u][r][i / 2][w / (4 / NS)], part[r][n][i], acc[r][n][i]);
                        }
                    }
                }
            }
        }
        if constexpr (KS > 1) {  // the warps' sums in their order
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float4*>(red + (((warp * RT + r) * NT + n) * 32 + lane) * 4) =
                        make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int k = 1; k < KS; ++k)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float4 v = *reinterpret_cast<const float4*>(red + ((((warp + k) * RT + r) * NT + n) * 32 + lane) * 4);
                            acc[r][n][0] += v.x;
                            acc[r][n][1] += v.y;
                            acc[r][n][2] += v.z;
                            acc[r][n][3] += v.w;
                        }
            }
        }
        if (KS == 1 || ks == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t t = t0 + n * 8 + c * 2 + (i & 1), at = row[r][i / 2];
                        if (t >= a.T || at >= a.N) continue;
                        const int64_t o = t * a.out_stride + at;
                        if (DT == kF32 || a.out_f32) static_cast<float*>(a.out)[o] = acc[r][n][i];
                        else static_cast<unsigned short*>(a.out)[o] = static_cast<unsigned short>(pack2<DT == kF32 ? kBF16 : DT>(acc[r][n][i], 0.0f));
                    }
        }
    }
}

constexpr int kLinearSmem = 220 * 1024;  // of the 227 KB that a CTA may have

template <int DT, int NT, int NS, int RT, int KS>
cudaError_t launch_linear(LinearArgs a, int sms, cudaStream_t s) {
    constexpr int W = 8, U = RT > 1 ? 2 : 4;
    constexpr int PL = DT == kF32 ? 3 : 1;
    constexpr size_t red = KS > 1 ? sizeof(float) * W * RT * NT * 128 : 0;
    auto kernel = linear4_kernel<DT, NT, NS, RT, KS, W, U>;
    a.tokens = static_cast<int>(a.T < 8 * NT ? a.T : 8 * NT);
    int most = ((kLinearSmem - static_cast<int>(red)) / (PL * a.tokens) - 64) / (kBlock * 2);
    if (most > a.blocks) most = a.blocks;
    a.chunk_blocks = most < 1 ? 1 : most;
    a.row_bytes = a.chunk_blocks * kBlock * 2 + 64;
    a.tiles = (a.N + 16 * RT - 1) / (16 * RT);
    const size_t smem = static_cast<size_t>(PL) * a.tokens * a.row_bytes + red;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int resident = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, 32 * W, smem);
    if (e != cudaSuccess) return e;
    int64_t grid = (a.tiles + W / KS - 1) / (W / KS);
    const int64_t most_ctas = static_cast<int64_t>(sms) * (resident < 1 ? 1 : resident);
    if (grid > most_ctas) grid = most_ctas;
    const int64_t gy = (a.T + 8 * NT - 1) / (8 * NT);
    return launch_pdl_smem(kernel, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(gy)), dim3(32 * W), smem, s, a);
}

template <int DT, int NT, int NS> cudaError_t launch_linear_split(const LinearArgs& a, int sms, cudaStream_t s) {
    constexpr int RT = NT * (DT == kF32 ? 3 : 1) > 1 ? 2 : 1;
    // Warps that read at the same time: about 16 per SM hide a load's latency.  Where rows are
    // too few for that, several warps share a tile's columns.
    const int64_t tiles = (a.N + 16 * RT - 1) / (16 * RT);
    const int64_t want = static_cast<int64_t>(sms) * 16;
    if (tiles >= want || a.blocks < 2) return launch_linear<DT, NT, NS, RT, 1>(a, sms, s);
    if (tiles * 2 >= want || a.blocks < 8) return launch_linear<DT, NT, NS, RT, 2>(a, sms, s);
    return launch_linear<DT, NT, NS, RT, 8>(a, sms, s);
}

template <int DT, int NT> cudaError_t launch_linear_groups(const LinearArgs& a, int group, int sms, cudaStream_t s) {
    return group == 128 ? launch_linear_split<DT, NT, 1>(a, sms, s)
           : group == 64 ? launch_linear_split<DT, NT, 2>(a, sms, s) : launch_linear_split<DT, NT, 4>(a, sms, s);
}

template <int DT> cudaError_t launch_linear_tokens(const LinearArgs& a, int group, int sms, cudaStream_t s) {
    if (a.T <= 8) return launch_linear_groups<DT, 1>(a, group, sms, s);
    if (a.T <= 16) return launch_linear_groups<DT, 2>(a, group, sms, s);
    return launch_linear_groups<DT, 4>(a, group, sms, s);
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
    return cuda_status(by_type(dtype, [&](auto dt) {
        return launch_linear_tokens<decltype(dt)::value>(a, static_cast<int>(group), sms, s);
    }));
}

}  // extern "C"
