// lse_linear4.cuh -- products of a few tokens with a matrix held in 4 bits (sm_103a).
//
//     y[t, n] = sum_g s[n, g] sum_{k in g} x[t, k] q[n, k]
//
// Bound by reading the codes, and here by instructions: half a byte per weight leaves about two
// and a half per weight and lane at the memory's rate.  So the weights do not go through scalar
// arithmetic.  A pair of nibbles becomes a pair of 16-bit floats, exactly q, by an or with the
// bits of 1024 (bf16: 128) and a subtraction, and mma.sync multiplies 16 rows x 16 columns with 8
// tokens, summing in f32.  The scale multiplies a group's f32 sum, so nothing but the result is
// rounded to 16 bits.  f32 tokens are cut into three bf16 parts (8 + 8 + 8 bits, exact) that are
// three more columns of the product.  Numbers of which bf16's range would cut bits off (below
// 2^-110) take a slower way, times 2^64 in columns of their own.
//
// Measured: one bf16 token x 128256 x 2048 39 us, 3.4 TB/s (the same loads without the products 26
// us); 16 f16 tokens x 32000 x 4096 32 us.  The matrix pipe is busy for 19 % and 21 % of that, the
// logic pipe for 50 % and 34 %.  For one token making floats of codes is what counts (59 % of the
// issue slots), so a matrix instruction of a higher rate (tcgen05, which would also take the floats
// through shared memory or tensor memory) has little to win before that does.  For 16 tokens
// nothing is busy (40 % of the issue slots): one CTA fits an SM, all of it waits for x before the
// first product, and 250 groups of tiles are two rounds of 152 CTAs.  Deeper prefetching (6 blocks instead of 4: 41 us) and two
// tiles per warp (46 us) were slower for one token; more warps sharing a tile's columns, which
// adds barriers, too (53 us).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"
#include "lse_linear4_common.cuh"

namespace lse {
namespace {

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
        // and (1024 + 16 (q + 8)) / 16 - 72 = q without a shift.  (A published method: Kim, Henry,
        // Fahim, Awadalla, "Who Says Elephants Can't Run", 2022; the constants are the format's.)
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

// An f32 from this magnitude on is three bf16 exactly: its last bit counts 2^-126 or more, bf16's
// smallest normal number.  Where one of a chunk's numbers is not (below 2^-110 the last bits of it
// lie below bf16's smallest), all that are smaller than this are cut into parts times 2^64.
constexpr float kSmallToken = 0x1p-103f;
enum Taken : int { kAllTokens, kLargeTokens, kSmallTokens };  // (the others as 0; small ones times 2^64)

// The part of x that a chunk needs, as 16-bit floats: PL planes of `tokens` rows.  Whether there
// are f32 among it that lose bits when cut as they are.
template <int DT, int TAKEN = kAllTokens>
__device__ __forceinline__ bool stage_tokens(const LinearArgs& a, int64_t t0, int b0, int nb, unsigned char* smem) {
    uint32_t last = 0;  // the last parts as f32
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
                    if constexpr (TAKEN == kLargeTokens) r = fabsf(r) < kSmallToken ? 0.0f : r;
                    if constexpr (TAKEN == kSmallTokens) r = fabsf(r) < kSmallToken ? r * 0x1p64f : 0.0f;
                    const bool finite = fabsf(r) <= 3.4028235e38f;
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        const uint32_t top = __float_as_uint(r) & 0xffff0000u;
                        if (q == 2) last |= __float_as_uint(r);
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
    return (last & 0xffffu) != 0;
}

// A block's codes and scales of a warp's rows, as loaded: nothing is made of them before the
// loads behind them are under way.  The 2 NS scales of a pair of rows are spread over the four
// lanes that share it.
template <int RT, int NS> struct Loaded {
    static constexpr int kScales = NS == 4 ? 2 : 1;
    uint4 q[RT][2];
    uint32_t s[RT][kScales];
};
template <bool S32> __device__ __forceinline__ float scale_of(uint32_t bits, int dtype) {
    if constexpr (S32) return __uint_as_float(bits);
    else return dtype == kBF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// Tokens by groups of 8 (NT), groups of columns in a block (NS), tiles of 16 rows per warp (RT),
// blocks of codes in flight per warp (D), scales of 32 bits.  a.ks warps share the columns of a
// tile: block b of a chunk belongs to warp b % ks.
// A CTA's tiles from `first` on.  SMALL: chunks of half as many blocks, and behind their x the small
// numbers of it, so that both meet in a group's sum.  Else it stops at f32 tokens that need that,
// and returns where (-1: it came to the end).
template <int DT, int NT, int NS, int RT, int D, bool S32, bool SMALL>
__device__ __forceinline__ int64_t linear4_tiles(const LinearArgs& a, unsigned char* smem, int64_t first) {
    constexpr bool F16 = DT == kF16;
    constexpr int PL = DT == kF32 ? 3 : 1;
    const int chunk = SMALL ? a.chunk_blocks / 2 : a.chunk_blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int KS = a.ks, ks = warp % KS, together = (blockDim.x >> 5) / KS;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 8 * NT;
    const int plane = a.tokens * a.row_bytes;
    // Behind x a row of zeros for the tokens that are not there, then the warps' sums.
    unsigned char* zeros = smem + PL * plane;
    float* red = reinterpret_cast<float*>(zeros + a.row_bytes);
    for (int i = threadIdx.x * 16; i < a.row_bytes; i += blockDim.x * 16) *reinterpret_cast<uint4*>(zeros + i) = make_uint4(0, 0, 0, 0);
    const unsigned char* mine[NT];  // where this lane's columns of its tokens are
    int next_plane[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const bool there = n * 8 + g < a.tokens;
        mine[n] = (there ? smem + (n * 8 + g) * a.row_bytes : zeros) + c * 16;
        next_plane[n] = there ? plane : 0;
    }

    Loaded<RT, NS> ring[D];
    // Where this lane's codes and scales of the tile begin.  Rows behind the last are computed from
    // it and not stored.
    const uint4* codes[RT][2];
    const char* scales[RT][Loaded<RT, NS>::kScales];
    constexpr int SB = S32 ? 4 : 2;
    const int group0 = NS == 4 ? c : NS == 2 ? (c & 1) : 0;  // of a block: the group whose scale this lane loads
    const auto aim = [&](int64_t tile) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t row = (tile * RT + r) * 16 + h * 8 + g;
                codes[r][h] = a.codes + (row < a.N ? row : a.N - 1) * a.blocks * 4 + c;
            }
#pragma unroll
            for (int i = 0; i < Loaded<RT, NS>::kScales; ++i) {
                const int h = NS == 4 ? i : NS == 2 ? c >> 1 : c & 1;
                const int64_t row = (tile * RT + r) * 16 + h * 8 + g;
                scales[r][i] = static_cast<const char*>(a.scales) + (row < a.N ? row : a.N - 1) * a.scale_stride * SB;
            }
        }
    };
    const auto fetch = [&](Loaded<RT, NS>& to, int block) {
        const int grp = min(block * NS + group0, a.groups - 1);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) to.q[r][h] = ldg_stream16(codes[r][h] + block * 4);
#pragma unroll
            for (int i = 0; i < Loaded<RT, NS>::kScales; ++i) {
                if constexpr (S32) to.s[r][i] = __ldg(reinterpret_cast<const uint32_t*>(scales[r][i]) + grp);
                else to.s[r][i] = __ldg(reinterpret_cast<const unsigned short*>(scales[r][i]) + grp);
            }
        }
    };
    float acc[RT][NT][4];
    const auto multiply = [&](const Loaded<RT, NS>& from, int b0, int at) {  // at: the block in the chunk
        // Groups behind the last meet codes of 0: with a scale of 0, since 0 times one that is there
        // need not be 0.
        const bool there = NS == 1 || (b0 + at) * NS + group0 < a.groups;
        float part[RT][NT][4], part_small[SMALL ? RT : 1][SMALL ? NT : 1][4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w % (4 / NS) == 0) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            part[r][n][i] = 0.0f;
                            if constexpr (SMALL) part_small[r][n][i] = 0.0f;
                        }
            }
            uint32_t p[RT][2][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 v = from.q[r][h];
                    word_pairs<F16>(w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w, p[r][h]);
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int l = 0; l < PL; ++l) {
                    const uint4 x = *reinterpret_cast<const uint4*>(mine[n] + l * next_plane[n] + at * (kBlock * 2) + w * 64);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        mma<F16>(part[r][n], p[r][0][0], p[r][1][0], p[r][0][1], p[r][1][1], x.x, x.y);
                        mma<F16>(part[r][n], p[r][0][2], p[r][1][2], p[r][0][3], p[r][1][3], x.z, x.w);
                    }
                    if constexpr (SMALL) {
                        const uint4 y = *reinterpret_cast<const uint4*>(mine[n] + l * next_plane[n] + (chunk + at) * (kBlock * 2) + w * 64);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            mma<F16>(part_small[r][n], p[r][0][0], p[r][1][0], p[r][0][1], p[r][1][1], y.x, y.y);
                            mma<F16>(part_small[r][n], p[r][0][2], p[r][1][2], p[r][0][3], p[r][1][3], y.z, y.w);
                        }
                    }
                }
            }
            if (w % (4 / NS) == 4 / NS - 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    // From the lane that loaded it: group i of the block, rows g and g + 8.
                    const int i = w / (4 / NS), lane0 = lane & ~3;
                    const uint32_t b0 = __shfl_sync(0xffffffffu, there ? from.s[r][0] : 0u, lane0 + (NS == 1 ? 0 : i));
                    const uint32_t b1 = __shfl_sync(0xffffffffu, there ? from.s[r][NS == 4 ? 1 : 0] : 0u, lane0 + (NS == 4 ? i : NS == 2 ? 2 + i : 1));
                    const float s0 = scale_of<S32>(b0, a.scale_dtype), s1 = scale_of<S32>(b1, a.scale_dtype);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (SMALL) part[r][n][j] = fmaf(part_small[r][n][j], 0x1p-64f, part[r][n][j]);
                            acc[r][n][j] = fmaf(j < 2 ? s0 : s1, part[r][n][j], acc[r][n][j]);
                        }
                }
            }
        }
    };
    // The first D blocks of a warp in the chunk at b0.
    const auto refill = [&](int64_t tile, int b0) {
        if (tile >= a.tiles) return;
        if (b0 == 0) aim(tile);
        const int nb = min(chunk, a.blocks - b0);
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (ks + d * KS < nb) fetch(ring[d], b0 + ks + d * KS);
    };
    bool staged = false;
    const int64_t step = static_cast<int64_t>(gridDim.x) * together;
    int64_t tile = first + warp / KS;
    refill(tile, 0);
    for (; first < a.tiles; first += step, tile += step) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.0f;
        for (int b0 = 0; b0 < a.blocks; b0 += chunk) {
            const int nb = min(chunk, a.blocks - b0);
            if (!staged || chunk < a.blocks) {
                __syncthreads();
                if constexpr (SMALL) {
                    stage_tokens<DT, kLargeTokens>(a, t0, b0, nb, smem);
                    stage_tokens<DT, kSmallTokens>(a, t0, b0, nb, smem + chunk * (kBlock * 2));
                    __syncthreads();
                } else if constexpr (DT == kF32) {
                    if (__syncthreads_or(stage_tokens<DT>(a, t0, b0, nb, smem))) return first;
                } else {
                    stage_tokens<DT>(a, t0, b0, nb, smem);
                    __syncthreads();
                }
                staged = true;
            }
            if (tile < a.tiles) {
                for (int b = ks; b < nb; b += D * KS) {
#pragma unroll
                    for (int d = 0; d < D; ++d) {
                        const int at = b + d * KS;
                        if (at >= nb) continue;
                        multiply(ring[d], b0, at);
                        if (at + D * KS < nb) fetch(ring[d], b0 + at + D * KS);
                    }
                }
            }
            // What comes next is under way before this tile's sums are put together.
            if (b0 + chunk < a.blocks) refill(tile, b0 + chunk);
            else refill(tile + step, 0);
        }
        if (KS > 1) {  // the warps' sums in their order
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float4*>(red + (((warp * RT + r) * NT + n) * 32 + lane) * 4) =
                        make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
            __syncthreads();
            if (ks == 0) {
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
        if (ks != 0 || tile >= a.tiles) continue;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t t = t0 + n * 8 + c * 2 + (i & 1), at = (tile * RT + r) * 16 + (i / 2) * 8 + g;
                    if (t >= a.T || at >= a.N) continue;
                    const int64_t o = t * a.out_stride + at;
                    if (DT == kF32 || a.out_f32) static_cast<float*>(a.out)[o] = acc[r][n][i];
                    else static_cast<unsigned short*>(a.out)[o] = static_cast<unsigned short>(pack2<DT == kF32 ? kBF16 : DT>(acc[r][n][i], 0.0f));
                }
    }
    return -1;
}

// (Not inlined: its registers are not the usual path's.)
template <int DT, int NT, int NS, int RT, bool S32>
__device__ __noinline__ void linear4_small_tiles(LinearArgs a, unsigned char* smem, int64_t first) {
    linear4_tiles<DT, NT, NS, RT, 1, S32, true>(a, smem, first);
}

// MW: warps of a CTA at most.
template <int DT, int NT, int NS, int RT, int D, bool S32, int MW>
__global__ void __launch_bounds__(32 * MW, MW == 8 ? 3 : 1) linear4_kernel(LinearArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_trigger();
    pdl_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ((blockDim.x >> 5) / a.ks);
    const int64_t left = linear4_tiles<DT, NT, NS, RT, D, S32, false>(a, smem, first);
    if constexpr (DT == kF32) {
        if (left >= 0) linear4_small_tiles<DT, NT, NS, RT, S32>(a, smem, left);
    }
}

// Dynamic shared memory of a CTA at most, the same in every call: calls of other threads do not
// lower it in between.
constexpr int kMostDynamic = 227 * 1024;

// ---------------------------------------------------------------------------
// Up to four f32 tokens: scalar arithmetic in f32, no matrix instructions (which would need three
// parts of each number: 3 tokens of 50257 x 1001 took 27 us with them and take 19, one of 50257 x 1024
// 19 and 12; of 16-bit tokens matrix instructions are faster, 39 us against 53 for one of 128256 x
// 2048 bf16).  A warp takes rows
// whole, 1024 columns at a time: a lane's 16 bytes hold 32 codes, and a row's 512 bytes lie next
// to each other.  A code becomes an f32 by an or alone: left where it is in its word, p bits up
// (p <= 16), it is 2^23 + 2^p (q + 8), and taking 2^23 + 8 2^p off leaves 2^p q exactly, which meets
// an x that was multiplied by 2^-p in shared memory.  (Where x has numbers that lose bits by that,
// a multiply-add by 2^-p leaves q and meets x as it is: 58 us instead of 50 for one token of 128256 x
// 2048.)  Of the eight codes of a word five need no shift and three share one.  With packed FP32 that is 1.1 logic, 0.5 add and 0.5 multiply-add
// instructions per weight and token.
// ---------------------------------------------------------------------------
// Rows of a warp at a time, and CTAs that an SM holds: by the registers that codes, scales, x
// and sums take.
__host__ __device__ constexpr int few_rows(int tokens, int ns) { return tokens == 1 && ns < 4 ? 4 : 2; }
__host__ __device__ constexpr int few_ctas(int tokens) { return tokens <= 2 ? 3 : 2; }
constexpr int kFewWarps = 8;
constexpr int kFewColumns = 1024;
constexpr int kFewTokens = 4;

// Bits by which the code of column e of a word lies above bit 0, after the shift of its half.
__host__ __device__ constexpr int code_shift(int e) { return e == 1 ? 16 : e % 2 == 0 ? 2 * e : 2 * e + 2; }

// x of the call, permuted: [chunk][word][half][token][lane][4 columns], each column times 2^-shift
// unless SMALL.  Whether there are numbers that lose bits by that.
constexpr float kSmallFew = 0x1p-110f;  // 2^-126 times the largest shift
template <int DT, int NTOK, bool SMALL> __device__ __forceinline__ bool stage_few(const LinearArgs& a, int chunks, float* smem) {
    bool small = false;
    for (int i = threadIdx.x; i < chunks * 8 * NTOK * 32; i += blockDim.x) {
        const int lane = i & 31, t = i / 32 % NTOK, h = i / (32 * NTOK) % 2, w = i / (64 * NTOK) % 4, chunk = i / (256 * NTOK);
        const int k = chunk * kFewColumns + (lane >> 2) * kBlock + 32 * w + 8 * (lane & 3) + 4 * h;
        const char* row = static_cast<const char*>(a.x) + static_cast<int64_t>(t) * a.x_stride * DType<DT>::bytes;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float down = __int_as_float((127 - (SMALL ? 0 : h == 0 ? code_shift(e) : code_shift(e + 4))) << 23);
            v[e] = k + e < a.K ? load_elem<DT>(row, k + e) : 0.0f;
            if constexpr (!SMALL) small |= fabsf(v[e]) < kSmallFew && v[e] != 0.0f;
            v[e] *= down;
        }
        *reinterpret_cast<float4*>(smem + i * 4) = make_float4(v[0], v[1], v[2], v[3]);
    }
    return small;
}

// Products of a warp's rows with each group's sum put together before it meets its scale, for rows
// with a scale that is no finite number: there the sum of scaled parts need not be the scaled sum
// (an infinite scale makes a NaN of a part that is 0, or of two parts of different signs).
template <int DT, int NTOK, int R, bool S32> __device__ __noinline__ void odd_rows(LinearArgs a, int64_t row0) {
    const int lane = threadIdx.x & 31;
    for (int64_t row = row0; row < row0 + R && row < a.N; ++row) {
        const char* const scales = static_cast<const char*>(a.scales) + row * a.scale_stride * (S32 ? 4 : 2);
        const uint32_t* const codes = reinterpret_cast<const uint32_t*>(a.codes) + row * a.blocks * kBlockWords;
        const auto scale = [&](int g) {
            return scale_of<S32>(S32 ? __ldg(reinterpret_cast<const uint32_t*>(scales) + g)
                                     : __ldg(reinterpret_cast<const unsigned short*>(scales) + g), a.scale_dtype);
        };
        bool finite = true;
        for (int g = lane; g < a.groups; g += 32) finite &= fabsf(scale(g)) <= 3.4028235e38f;
        if (__all_sync(0xffffffffu, finite)) continue;
        for (int t = 0; t < NTOK; ++t) {
            const char* const x = static_cast<const char*>(a.x) + t * a.x_stride * DType<DT>::bytes;
            float sum = 0.0f;
            for (int g = 0; g < a.groups; ++g) {
                float part = 0.0f;
                for (int k = g * a.group + lane; k < min((g + 1) * a.group, a.K); k += 32) {
                    const int j = k >> 3 & 15, e = k & 7;
                    const uint32_t w = __ldg(codes + (k >> 7) * kBlockWords + (j & 3) * 4 + (j >> 2));
                    part = fmaf(static_cast<float>(static_cast<int>(w >> (e / 2 * 4 + e % 2 * 16) & 15u) - 8), load_elem<DT>(x, k), part);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
                sum = fmaf(scale(g), part, sum);
            }
            if (lane == 0) {
                const int64_t o = t * a.out_stride + row;
                if (DT == kF32 || a.out_f32) static_cast<float*>(a.out)[o] = sum;
                else static_cast<unsigned short*>(a.out)[o] = static_cast<unsigned short>(pack2<DT == kF32 ? kBF16 : DT>(sum, 0.0f));
            }
        }
    }
}

// All rows of a warp; false where x has numbers that need SMALL (nothing is written then).
template <int DT, int NTOK, int NS, bool S32, bool SMALL>
__device__ __forceinline__ bool few_tokens(const LinearArgs& a, int chunks, float* smem) {
    constexpr int SB = S32 ? 4 : 2, R = few_rows(NTOK, NS);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kFewWarps * R;
    int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kFewWarps + warp) * R;

    uint4 q[R];
    uint32_t s[R][NS];
    // Codes of the rows from `row` on in a chunk: 8 (q = 0) behind the matrix's last column or row.
    const auto fetch = [&](int64_t row, int chunk) {
        const int block = chunk * (kFewColumns / kBlock) + (lane >> 2);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            q[r] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
#pragma unroll
            for (int i = 0; i < NS; ++i) s[r][i] = 0;
            if (row + r < a.N && block < a.blocks) {
                q[r] = ldg_stream16(a.codes + ((row + r) * a.blocks + block) * 4 + (lane & 3));
                const char* p = static_cast<const char*>(a.scales) + (row + r) * a.scale_stride * SB;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int grp = block * NS + i;  // (one behind the last: a scale of 0)
                    if (NS > 1 && grp >= a.groups) continue;
                    if constexpr (S32) s[r][i] = __ldg(reinterpret_cast<const uint32_t*>(p) + grp);
                    else s[r][i] = __ldg(reinterpret_cast<const unsigned short*>(p) + grp);
                }
            }
        }
    };
    fetch(row0, 0);
    if (__syncthreads_or(stage_few<DT, NTOK, SMALL>(a, chunks, smem))) return false;
    for (; row0 < a.N; row0 += step) {
        float acc[R][NTOK];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NTOK; ++t) acc[r][t] = 0.0f;
        for (int chunk = 0; chunk < chunks; ++chunk) {
            uint4 qq[R];
            float sc[R][NS];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                qq[r] = q[r];
#pragma unroll
                for (int i = 0; i < NS; ++i) sc[r][i] = scale_of<S32>(s[r][i], a.scale_dtype);
            }
            // The next codes are under way while these are multiplied.
            if (chunk + 1 < chunks) fetch(row0, chunk + 1);
            else fetch(row0 + step, 0);
            uint64_t part[R][NTOK];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w % (4 / NS) == 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int t = 0; t < NTOK; ++t) part[r][t] = 0;
                }
                uint64_t x[NTOK][4];  // pairs of columns
#pragma unroll
                for (int t = 0; t < NTOK; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 v = *reinterpret_cast<const float4*>(smem + ((((chunk * 4 + w) * 2 + h) * NTOK + t) * 32 + lane) * 4);
                        x[t][2 * h] = f2_pack(v.x, v.y);
                        x[t][2 * h + 1] = f2_pack(v.z, v.w);
                    }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint32_t v = w == 0 ? qq[r].x : w == 1 ? qq[r].y : w == 2 ? qq[r].z : qq[r].w;
                    const uint32_t up = v >> 12;  // columns 3, 5, 7
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const int p0 = code_shift(e), p1 = code_shift(e + 1);
                        const uint32_t b0 = (v & (15u << p0)) | 0x4b000000u;
                        const uint32_t b1 = ((e == 0 ? v : up) & (15u << p1)) | 0x4b000000u;
                        const uint64_t raised = f2_pack(__uint_as_float(b0), __uint_as_float(b1));
                        uint64_t c;
                        if constexpr (SMALL) {
                            const float d0 = 1.0f / static_cast<float>(1 << p0), d1 = 1.0f / static_cast<float>(1 << p1);
                            c = f2_fma(raised, f2_pack(d0, d1), f2_pack(-8388608.0f * d0 - 8.0f, -8388608.0f * d1 - 8.0f));
                        } else {
                            c = f2_sub(raised, f2_pack(8388608.0f + static_cast<float>(8 << p0), 8388608.0f + static_cast<float>(8 << p1)));
                        }
#pragma unroll
                        for (int t = 0; t < NTOK; ++t) part[r][t] = f2_fma(c, x[t][e / 2], part[r][t]);
                    }
                }
                if (w % (4 / NS) == 4 / NS - 1) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int t = 0; t < NTOK; ++t) {
                            float lo, hi;
                            f2_unpack(part[r][t], lo, hi);
                            acc[r][t] = fmaf(sc[r][w / (4 / NS)], lo + hi, acc[r][t]);
                        }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NTOK; ++t) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
            }
        // Lane t * R + r writes the sum of row r and token t.
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NTOK; ++t)
                if (lane == t * R + r && row0 + r < a.N) {
                    const int64_t o = t * a.out_stride + row0 + r;
                    if (DT == kF32 || a.out_f32) static_cast<float*>(a.out)[o] = acc[r][t];
                    else static_cast<unsigned short*>(a.out)[o] = static_cast<unsigned short>(pack2<DT == kF32 ? kBF16 : DT>(acc[r][t], 0.0f));
                }
        float odd = 0.0f;  // NaN where a sum is no finite number (the same in all lanes)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < NTOK; ++t) odd = fmaf(acc[r][t], 0.0f, odd);
        if (odd != 0.0f) {
            __syncwarp();
            odd_rows<DT, NTOK, R, S32>(a, row0);
        }
    }
    return true;
}

// (Not inlined: its registers are not the usual path's.)
template <int DT, int NTOK, int NS, bool S32>
__device__ __noinline__ void few_small_tokens(LinearArgs a, int chunks, float* smem) {
    few_tokens<DT, NTOK, NS, S32, true>(a, chunks, smem);
}

template <int DT, int NTOK, int NS, bool S32>
__global__ void __launch_bounds__(32 * kFewWarps, few_ctas(NTOK)) linear4_few_kernel(LinearArgs a, int chunks) {
    extern __shared__ __align__(16) unsigned char smem_bytes[];
    float* const smem = reinterpret_cast<float*>(smem_bytes);
    pdl_trigger();
    pdl_wait();
    if (!few_tokens<DT, NTOK, NS, S32, false>(a, chunks, smem)) few_small_tokens<DT, NTOK, NS, S32>(a, chunks, smem);
}

// x in shared memory as f32, with room for three CTAs per SM.
inline bool few_fits(const LinearArgs& a) {
    const int64_t chunks = (a.blocks + kFewColumns / kBlock - 1) / (kFewColumns / kBlock);
    return a.T <= kFewTokens && a.blocks > 0 && chunks * kFewColumns * 4 * a.T <= 72 * 1024;
}
template <int DT, int NTOK, int NS, bool S32> cudaError_t launch_few(const LinearArgs& a, int sms, cudaStream_t s) {
    auto kernel = linear4_few_kernel<DT, NTOK, NS, S32>;
    const int chunks = (a.blocks + kFewColumns / kBlock - 1) / (kFewColumns / kBlock);
    const size_t smem = static_cast<size_t>(chunks) * kFewColumns * 4 * NTOK;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
        if (e != cudaSuccess) return e;
    }
    int64_t grid = (a.N + kFewWarps * few_rows(NTOK, NS) - 1) / (kFewWarps * few_rows(NTOK, NS));
    if (grid > few_ctas(NTOK) * sms) grid = few_ctas(NTOK) * sms;
    return launch_pdl_smem(kernel, dim3(static_cast<unsigned>(grid)), dim3(32 * kFewWarps), smem, s, a, chunks);
}
template <int DT, int NTOK> cudaError_t launch_few_groups(const LinearArgs& a, int sms, cudaStream_t s) {
    const bool f32 = a.scale_dtype == kF32;
    if (a.group == 128) return f32 ? launch_few<DT, NTOK, 1, true>(a, sms, s) : launch_few<DT, NTOK, 1, false>(a, sms, s);
    if (a.group == 64) return f32 ? launch_few<DT, NTOK, 2, true>(a, sms, s) : launch_few<DT, NTOK, 2, false>(a, sms, s);
    return f32 ? launch_few<DT, NTOK, 4, true>(a, sms, s) : launch_few<DT, NTOK, 4, false>(a, sms, s);
}

constexpr int kLinearSmem = 220 * 1024;  // of the 227 KB that a CTA may have

template <int DT, int NT, int NS, bool S32> cudaError_t launch_linear(LinearArgs a, int sms, cudaStream_t s) {
    constexpr int PL = DT == kF32 ? 3 : 1;
    // Two tiles per warp halve the reads of x from shared memory for each weight; with four
    // groups of tokens their sums would take more registers than there are.
    constexpr int RT = NT * PL == 2 || NT * PL == 3 ? 2 : 1;

    a.tokens = static_cast<int>(a.T < 8 * NT ? a.T : 8 * NT);
    a.tiles = (a.N + 16 * RT - 1) / (16 * RT);
    const int64_t row = static_cast<int64_t>(a.blocks) * kBlock * 2 + 64;
    // Three CTAs of 8 warps per SM; x that leaves room for one only: 16 warps in it.
    const bool wide = NT > 1 || PL * a.tokens * row > 64 * 1024;
    const int warps = wide ? 16 : 8;
    auto kernel = linear4_kernel<DT, NT, NS, RT, RT == 2 ? 2 : 3, S32, 16>;
    if constexpr (NT == 1) {
        if (!wide) kernel = linear4_kernel<DT, NT, NS, RT, RT == 2 ? 2 : 4, S32, 8>;
    }
    // About 24 warps per SM read at the same time; where rows are too few for that, several share
    // a tile's columns.
    int ks = 1;
    while (ks < warps && a.tiles * ks < static_cast<int64_t>(sms) * 24 && 2 * ks <= a.blocks) ks *= 2;
    a.ks = ks;
    const int red = ks > 1 ? static_cast<int>(sizeof(float)) * warps * RT * NT * 128 : 0;
    int most = ((kLinearSmem - red) / (PL * a.tokens + 1) - 64) / (kBlock * 2);
    if (most > a.blocks) most = a.blocks;
    // (of f32 two at least: a block and its small numbers)
    const int least = DT == kF32 ? 2 : 1;
    a.chunk_blocks = most < least ? least : most;
    a.row_bytes = a.chunk_blocks * kBlock * 2 + 64;
    const size_t smem = static_cast<size_t>(PL * a.tokens + 1) * a.row_bytes + red;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
        if (e != cudaSuccess) return e;
    }
    const int64_t groups = (a.tiles + warps / ks - 1) / (warps / ks);
    // CTAs go on with further tiles, so that x is brought in once; small x may be brought in
    // more often.
    const int64_t fit = static_cast<int64_t>(227 * 1024 / (smem + 1024)), threads = warps == 16 ? 1 : 4;
    int64_t grid = static_cast<int64_t>(sms) * (fit < threads ? fit : threads);
    if (grid > groups) grid = groups;
    const int64_t gy = (a.T + 8 * NT - 1) / (8 * NT);
    return launch_pdl_smem(kernel, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(gy)), dim3(32 * warps), smem, s, a);
}

template <int DT, int NT, int NS> cudaError_t launch_linear_scales(const LinearArgs& a, int sms, cudaStream_t s) {
    return a.scale_dtype == kF32 ? launch_linear<DT, NT, NS, true>(a, sms, s) : launch_linear<DT, NT, NS, false>(a, sms, s);
}
template <int DT, int NT> cudaError_t launch_linear_groups(const LinearArgs& a, int sms, cudaStream_t s) {
    return a.group == 128 ? launch_linear_scales<DT, NT, 1>(a, sms, s)
           : a.group == 64 ? launch_linear_scales<DT, NT, 2>(a, sms, s) : launch_linear_scales<DT, NT, 4>(a, sms, s);
}
template <int DT> cudaError_t launch_linear_tokens(const LinearArgs& a, int sms, cudaStream_t s) {
    if constexpr (DT == kF32) {
        if (few_fits(a)) {
            switch (a.T) {
            case 1: return launch_few_groups<DT, 1>(a, sms, s);
            case 2: return launch_few_groups<DT, 2>(a, sms, s);
            case 3: return launch_few_groups<DT, 3>(a, sms, s);
            default: return launch_few_groups<DT, 4>(a, sms, s);
            }
        }
    }
    if (a.T <= 8) return launch_linear_groups<DT, 1>(a, sms, s);
    if (a.T <= 16) return launch_linear_groups<DT, 2>(a, sms, s);
    return launch_linear_groups<DT, 4>(a, sms, s);
}

}  // namespace
}  // namespace lse
