// lse_stats.cuh -- token statistics of rows of logits: the kernels and their launch for
// one element type (sm_103a).  Included by one translation unit per type.
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
// a sum of two non-negative terms.  (m, s, u) is kept online:
// raising the maximum by d (in units of z) turns u into (u + d s) 2^-d and s into
// s 2^-d.
#pragma once

#include <atomic>
#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_edges.cuh"
#include "lse_internal.h"
#include "lse_stats_common.cuh"
#include "lse_topk.cuh"

namespace lse {
namespace {

// The exponentials' argument is z = x log2 e - c, c = fl(mu log2 e), by one FMA, so
// every term carries the factor 2^r, r = mu log2 e - c, which the logarithm takes
// out again; the entropy does not change with it but for rounding, as r enters log2 s
// and u / s with opposite signs.  In a row with nearly all of p on one token that is all
// there is, so what must not be negative (H, log sum exp(x - max)) ends at 0.  Beyond
// |mu| = 2^24 (r would
// exceed an octave), and for f16 where mu is next to the lowest value, z is
// (x - mu) log2 e in two steps and r is 0.
struct Shift {
    float mu, c;
    bool two_step;
};

template <int DT>
__device__ __forceinline__ Shift make_shift(float m) {
    const float mu = shift_of(m);
    return Shift{mu, mu * kLog2e, fabsf(mu) > 0x1.0p24f || (DT == kF16 && mu < -60000.0f)};
}
template <int DT>
__device__ __forceinline__ float shift_residue(float m) {
    const Shift h = make_shift<DT>(m);
    return h.two_step ? 0.0f : fmaf(h.mu, kLog2e, -h.c);
}

struct StatAcc {
    float m, s, u;
};

__device__ __forceinline__ StatAcc stat_identity() { return StatAcc{__int_as_float(kNegInfF32), 0.0f, 0.0f}; }

// The sums against the shift of another maximum m >= the accumulator's own, which is
// d octaves higher: s 2^-d and (u + d s) 2^-d.
template <int DT>
__device__ __forceinline__ StatAcc stat_shift(StatAcc a, float m) {
    float d = (shift_of(m) - a.m) * kLog2e + (shift_residue<DT>(a.m) - shift_residue<DT>(m));
    d = fminf(d, -kFarBelow);  // (from no maximum at all: +inf)
    const float f = ex2(-d);
    return StatAcc{m, a.s * f, fmaf(d, a.s, a.u) * f};
}

// One accumulator of those of `WIDTH` neighbouring lanes, the same in all of them.
template <int DT, int WIDTH>
__device__ __forceinline__ StatAcc stat_lanes_merge(StatAcc a) {
    float m = a.m;
#pragma unroll
    for (int off = 1; off < WIDTH; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    a = stat_shift<DT>(a, m);
#pragma unroll
    for (int off = 1; off < WIDTH; off <<= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, off);
        a.u += __shfl_xor_sync(0xffffffffu, a.u, off);
    }
    return a;
}

// What the outputs of a row are made from.
struct RowStats {
    float m;     // maximum
    float lse;
    float logs;  // log sum exp(x - m); NaN where the row is no distribution
};

template <int DT>
__device__ __forceinline__ RowStats row_stats(StatAcc a) {
    RowStats r{a.m, a.s, __int_as_float(0x7fc00000)};
    if (a.s != a.s) return r;  // NaN in the row
    r.lse = a.m;               // +inf in it, or nothing but -inf
    if (!(fabsf(a.m) < __int_as_float(0x7f800000))) return r;
    r.logs = fmaxf(kLn2 * (lg2(a.s) - shift_residue<DT>(a.m)), 0.0f);
    r.lse = a.m + r.logs;
    return r;
}

// NaN for a row that is no distribution.
__device__ __forceinline__ float stat_entropy(StatAcc a, const RowStats& r) {
    if (r.logs != r.logs) return r.logs;
    const float h = kLn2 * (lg2(a.s) + a.u / a.s);
    return h <= 0.0f ? 0.0f : h;
}

// x - lse as (x - max) - log sum exp(x - max): next to a large maximum lse itself
// has few digits left for the logarithm.
__device__ __forceinline__ float stat_logprob(float x, const RowStats& r) {
    return r.logs != r.logs ? x - r.lse : (x - r.m) - r.logs;
}

// The larger of each packed 16-bit pair; a NaN stays.
template <int DT>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (DT == kBF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Add sum 2^z and sum 2^z (-z) over W raw words, two elements at a time (packed
// FP32).  A masked element (z = -inf) must add 0 to u and not 0 * inf: f32 words
// bound z from below, 16-bit ones the packed pair itself, 100 or more below mu, at
// half the instructions.  A NaN stays in s, which decides.
template <int DT, int W, bool TWO_STEP>
__device__ __forceinline__ void stat_sum_words(StatAcc& a, const Shift& h, const uint32_t (&w)[W]) {
    const uint64_t log2e2 = f2_pack(kLog2e, kLog2e);
    const uint64_t sub2 = TWO_STEP ? f2_pack(h.mu, h.mu) : f2_pack(-h.c, -h.c);
    uint32_t floor2 = 0;
    if constexpr (!TWO_STEP && DT != kF32) {
        const float low = h.mu - fmaf(fabsf(h.mu), 0x1.0p-6f, 200.0f);
        floor2 = pack2<DT>(low, low);
    }
    uint64_t s[2] = {0ull, 0ull}, u[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < W; i += DT == kF32 ? 2 : 1) {
        uint64_t x;
        if constexpr (DT == kF32) {
            x = f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
        } else {
            const uint32_t v = TWO_STEP ? w[i] : max2_nan<DT>(w[i], floor2);
            x = f2_pack(word_lo<DT>(v), word_hi<DT>(v));
        }
        const int k = DT == kF32 ? (i >> 1) & 1 : i & 1;
        const uint64_t z = TWO_STEP ? f2_mul(f2_sub(x, sub2), log2e2) : f2_fma(x, log2e2, sub2);
        float z0, z1;
        f2_unpack(z, z0, z1);
        const uint64_t e = f2_pack(ex2(z0), ex2(z1));
        s[k] = f2_add(s[k], e);
        if constexpr (TWO_STEP || DT == kF32) u[k] = f2_fma(e, f2_pack(fmaxf(z0, kFarBelow), fmaxf(z1, kFarBelow)), u[k]);
        else u[k] = f2_fma(e, z, u[k]);
    }
    float s0, s1, s2, s3, u0, u1, u2, u3;
    f2_unpack(s[0], s0, s1);
    f2_unpack(s[1], s2, s3);
    f2_unpack(u[0], u0, u1);
    f2_unpack(u[1], u2, u3);
    a.s += (s0 + s1) + (s2 + s3);
    a.u -= (u0 + u1) + (u2 + u3);
}

template <int DT, int W>
__device__ __forceinline__ void stat_add_words(StatAcc& a, const Shift& h, const uint32_t (&w)[W]) {
    if (h.two_step) stat_sum_words<DT, W, true>(a, h, w);
    else stat_sum_words<DT, W, false>(a, h, w);
}

// ---------------------------------------------------------------------------
// Rows as 16-byte vectors: the aligned vectors that cover the row, the elements
// outside it masked with -inf.
// ---------------------------------------------------------------------------
struct Row {
    const char* a0;    // 16-byte boundary at or before the row
    uint32_t off;      // bytes from there to the row
    int64_t end;       // the row's end, bytes from a0
    int64_t vectors;
};

template <int DT>
__device__ __forceinline__ Row make_row(const void* x, int64_t row, int64_t row_stride, int64_t N) {
    const char* rp = static_cast<const char*>(x) + row * row_stride * DType<DT>::bytes;
    Row r;
    r.off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(rp) & 15u);
    r.a0 = rp - r.off;
    r.end = r.off + N * DType<DT>::bytes;
    r.vectors = N > 0 ? (r.end + 15) >> 4 : 0;
    return r;
}

// Vector k of the row into 4 words of w; -inf past `limit`.
template <int DT>
__device__ __forceinline__ void load_vector(const Row& r, int64_t k, int64_t limit, uint32_t* w) {
    if (k < limit) {
        const uint4 v = ldg_stream16(r.a0 + k * 16);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        w[0] = w[1] = w[2] = w[3] = neg_inf_word<DT>();
    }
}

template <int DT>
__device__ __forceinline__ void mask_vector(const Row& r, int64_t k, uint32_t* w) {
    uint32_t q[4] = {w[0], w[1], w[2], w[3]};
    if (k == 0) mask_prefix<DT>(q, static_cast<int>(r.off));
    if (k == r.vectors - 1) mask_suffix<DT>(q, static_cast<int>(r.end - k * 16));
    w[0] = q[0]; w[1] = q[1]; w[2] = q[2]; w[3] = q[3];
}

// The column of element i of vector k (out of [0, N) for the masked ones).
template <int DT>
__device__ __forceinline__ int64_t column_of(const Row& r, int64_t k, int i) {
    return (k * 16 - static_cast<int64_t>(r.off)) / DType<DT>::bytes + i;
}

// ---------------------------------------------------------------------------
// The K largest keys.
//
// While the row streams by, nothing is kept of it but the maximum of every
// thread's chunk (a few vectors).  The K-th largest of the maxima of 32 groups of
// threads is a bound that at least K elements reach, so the K largest are among
// the elements that reach it -- for values in no particular order a few more than
// K.  Only the chunks whose maximum reaches the bound are read again, and each
// element found there takes the place that the number of larger ones gives it.
// Rows where this finds too many (long runs of equal values), too few (nearly
// everything masked with -inf) or a NaN are scanned once more in full.
// ---------------------------------------------------------------------------

// Packed 16-bit maxima; NaN lanes are ignored.  f32 maxima are kept as bf16, rounded
// to nearest: rounding keeps the order, so what reaches a bound reaches the rounded
// bound after it too.
template <int DT>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return DT == kF16 ? hmax2_f16(a, b) : hmax2_bf16(a, b);
}
template <int DT> __device__ __forceinline__ float half_lo(uint32_t w) { return word_lo<DT == kF16 ? kF16 : kBF16>(w); }
template <int DT> __device__ __forceinline__ float half_hi(uint32_t w) { return word_hi<DT == kF16 ? kF16 : kBF16>(w); }
template <int DT>
__device__ __forceinline__ float round16(float x) {
    return DT == kF32 ? word_lo<kBF16>(pack2<kBF16>(x, x)) : x;  // (16-bit elements are as they are)
}

// A value that no f32 maximum kept as bf16 v lies below (16-bit ones are as they are).
template <int DT>
__device__ __forceinline__ float step_down(float v) {
    if (DT != kF32 || !(fabsf(v) <= 3.4e38f)) return DT == kF32 && v > 0.0f ? 3.3e38f : v;
    const float d = v - fmaxf(fabsf(v) * 0x1.0p-8f, 0x1.0p-126f);
    return d;
}

// The maxima of the U / 2 pairs of neighbouring vectors of a batch, two per word, and
// the largest of all.
template <int DT, int U>
__device__ __forceinline__ float batch_maxima(const uint32_t (&w)[4 * U], uint32_t (&maxima)[U / 4]) {
    float all[U / 4];
#pragma unroll
    for (int h = 0; h < U / 4; ++h) {
        const uint32_t* const v = w + 16 * h;  // two pairs
        if constexpr (DT == kF32) {
            float c[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                c[q] = fmax3(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1]), __uint_as_float(v[8 * q + 2]));
                c[q] = fmax3(c[q], __uint_as_float(v[8 * q + 3]), __uint_as_float(v[8 * q + 4]));
                c[q] = fmax3(c[q], __uint_as_float(v[8 * q + 5]), __uint_as_float(v[8 * q + 6]));
                c[q] = fmaxf(c[q], __uint_as_float(v[8 * q + 7]));
            }
            maxima[h] = pack2<kBF16>(c[0], c[1]);
            all[h] = fmaxf(c[0], c[1]);
        } else {
            uint32_t c[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                c[q] = max2<DT>(max2<DT>(max2<DT>(v[8 * q], v[8 * q + 1]), max2<DT>(v[8 * q + 2], v[8 * q + 3])),
                                max2<DT>(max2<DT>(v[8 * q + 4], v[8 * q + 5]), max2<DT>(v[8 * q + 6], v[8 * q + 7])));
            // Both halves of the two words at once.
            maxima[h] = max2<DT>(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[0], c[1], 0x7632));
        }
    }
    if constexpr (DT == kF32) {
        return U == 4 ? all[0] : fmaxf(all[0], all[U / 4 - 1]);
    } else {
        const uint32_t m = U == 4 ? maxima[0] : max2<DT>(maxima[0], maxima[U / 4 - 1]);
        return fmaxf(word_lo<DT>(m), word_hi<DT>(m));
    }
}

// K-th largest of the G * M values of a group of G lanes, M (1 or 2) per lane, K <= G M
// (bitonic sort; value m of lane l is number m G + l).
template <int G, int M>
__device__ __forceinline__ float kth_largest(float (&v)[M], int K, int lane) {
#pragma unroll
    for (int size = 2; size <= G * M; size <<= 1) {
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            if (stride == G) {  // (the last size: descending)
                const float low = fminf(v[0], v[M - 1]);
                v[0] = fmaxf(v[0], v[M - 1]);
                v[M - 1] = low;
                continue;
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float o = __shfl_xor_sync(0xffffffffu, v[m], stride);
                const bool falling = size == G * M || (size == G ? m == 0 : (lane & size) == 0);
                const bool high = ((lane & stride) == 0) == falling;
                v[m] = high ? fmaxf(v[m], o) : fminf(v[m], o);
            }
        }
    }
    return __shfl_sync(0xffffffffu, M == 2 && K > G ? v[M - 1] : v[0], (K - 1) & (G - 1), G);
}

// The same for M = 32 or 64 values in shared memory (16-byte aligned): the smallest of
// those that fewer than K exceed.
template <int M>
__device__ __forceinline__ float kth_largest_of(const float* values, int K, int lane) {
    const float v = values[lane], u = M > 32 ? values[lane + M - 32] : 0.0f;
    int above_v = 0, above_u = 0;
#pragma unroll
    for (int j = 0; j < M; j += 4) {
        const float4 o = *reinterpret_cast<const float4*>(values + j);
        above_v += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
        if (M > 32) above_u += (o.x > u) + (o.y > u) + (o.z > u) + (o.w > u);
    }
    uint32_t least = above_v < K ? order_bits(v) : 0xffffffffu;
    if (M > 32 && above_u < K) least = min(least, order_bits(u));
    return order_value(__reduce_min_sync(0xffffffffu, least));
}

// Element e of W / 4 vectors held in registers, e not known at compile time.
template <int DT, int W>
__device__ __forceinline__ float pick_elem(const uint32_t (&w)[W], int e) {
    constexpr int EPW = 4 / DType<DT>::bytes;
    const int q = e / EPW;
    uint32_t v = w[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = q == i ? w[i] : v;
    if constexpr (DT == kF32) return __uint_as_float(v);
    else return (e & 1) ? word_hi<DT>(v) : word_lo<DT>(v);
}

// A warp's list of the K largest keys of vectors [k0, k1), read in order.  Past
// the first few vectors nearly every one is dismissed by its values alone: none
// above the K-th so far (an equal one later in the row ranks lower).
template <int DT>
__device__ __forceinline__ uint64_t scan_vectors(const Row& r, int64_t k0, int64_t k1, int64_t N,
                                                 int K, int lane) {
    constexpr int EPV = 16 / DType<DT>::bytes;
    uint64_t best = 0, bar = 0;
    float bar_value = __int_as_float(kNegInfF32);
    bool full = false;  // K keys found: values equal to the K-th no longer count
    for (int64_t k = k0; k < k1; k += 32) {
        uint32_t w[4];
        load_vector<DT>(r, k + lane, k1, w);
        bool any = false;
#pragma unroll
        for (int i = 0; i < EPV; ++i) {
            const float x = word_elem<DT>(w, i);
            any |= !full || x > bar_value || x != x;
        }
        if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll 1
        for (int i = 0; i < EPV; ++i) {
            const int64_t col = column_of<DT>(r, k + lane, i);
            uint64_t key = 0;
            if (k + lane < k1 && col >= 0 && col < N) key = topk_key(word_elem<DT>(w, i), static_cast<uint32_t>(col));
            if (!__any_sync(0xffffffffu, key > bar)) continue;
            best = list_merge(best, list_sort(key, lane), lane);
            bar = __shfl_sync(0xffffffffu, best, K - 1);
            full = bar != 0;
            bar_value = full ? key_value(bar) : bar_value;
        }
    }
    return best;
}

// What is lost when lse = max + log sum exp(x - max) is rounded to f32, exactly (the
// error of a sum is a float): the gradient takes x - lse from both.
__device__ __forceinline__ float lse_rest(const RowStats& r) {
    if (r.logs != r.logs) return 0.0f;  // no distribution: lse is infinite or NaN
    const float b = __fsub_rn(r.lse, r.m);
    return __fadd_rn(__fsub_rn(r.m, __fsub_rn(r.lse, b)), __fsub_rn(r.logs, b));
}

// Writes of one row's results.
__device__ __forceinline__ void put_row(const StatsArgs& a, int64_t row, const StatAcc& acc, const RowStats& r, float xt) {
    if (a.lse) a.lse[row] = r.lse;
    if (a.lse_low) a.lse_low[row] = lse_rest(r);
    if (a.entropy) a.entropy[row] = stat_entropy(acc, r);
    if (a.logprob) a.logprob[row] = stat_logprob(xt, r);
}
__device__ __forceinline__ void put_top(const StatsArgs& a, int64_t row, int place, uint64_t key, const RowStats& r) {
    a.top_index[row * a.K + place] = key ? key_column(key) : -1;
    a.top_logprob[row * a.K + place] = key ? stat_logprob(key_value(key), r) : __int_as_float(kNegInfF32);
}

// The keys of from[0, n) (all different; 0 is none) that fewer than K of them exceed:
// put(place, key) for each.  Called by whole warps; LANES lanes count for one key.
template <int LANES, typename PUT>
__device__ __forceinline__ void rank_keys(const uint64_t* from, int n, int K, int tid, int threads, PUT put) {
    for (int i0 = 0; i0 < n; i0 += threads / LANES) {
        const int i = i0 + tid / LANES;
        const uint64_t key = i < n ? from[i] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = tid % LANES; j < n; j += LANES) rank += from[j] > key;
#pragma unroll
        for (int off = 1; off < LANES; off <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, off);
        if (tid % LANES == 0 && key != 0 && rank < K) put(rank, key);
    }
}

// Cluster barrier and the place of a shared variable in another CTA of the cluster.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
template <typename V>
__device__ __forceinline__ V* cluster_map(V* p, uint32_t cta) {
    uint64_t q;
    asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(reinterpret_cast<uint64_t>(p)), "r"(cta));
    return reinterpret_cast<V*>(q);
}

// ---------------------------------------------------------------------------
// Long rows: a CTA per row, or a cluster of CTAs that share one.
// ---------------------------------------------------------------------------
// Vectors per thread and batch: eight; four in one-warp rows, which are short, so that
// less of the last batch is empty.
__host__ __device__ constexpr int stat_u(int T) { return T == 32 ? 4 : 8; }
// A chunk is two vectors of a thread (and, in rows of more batches than maxima are kept
// of, the same two of 2^chunk_shift batches in a row); its maximum is kept in 16 bits.
__host__ __device__ constexpr int stat_batches(int T) { return 128 / stat_u(T); }
// The bound is taken from the maxima of 32 groups of threads, or of 64 for larger K,
// for which 32 would let many more elements through (K = 32: about 130 against 44).
constexpr int kWideGroupsK = 24;
constexpr int kChunkList = 64;    // chunks that a warp may read again
constexpr int kMaxCluster = 16;
constexpr int kUnitsPerCta = 8;   // one-warp rows per CTA
constexpr int kPartKeys = 48;     // keys that a part hands on as it found them

template <int T, bool CLUSTER>
struct StatsShared {
    static constexpr int kFoundList = T == 32 ? 128 : 512;  // elements that may reach the bound
    float4 group_max4[16];
    alignas(16) uint32_t chunk_max[stat_u(T) / 4 * stat_batches(T) * T];
    uint64_t found[kFoundList];
    uint64_t own[kMaxTopK];
    // In the cluster's first CTA: the parts' keys, how many, their accumulators, and
    // the maxima of 32 or 64 groups of threads of the whole cluster.
    uint64_t keys[CLUSTER ? kMaxCluster * kPartKeys : 1];
    int key_count[CLUSTER ? kMaxCluster : 1];
    float acc[3][CLUSTER ? kMaxCluster : 1];
    float4 cluster_max4[CLUSTER ? 16 : 1];
    float part[3][T / 32];
    RowStats row;
    int16_t chunk[T / 32][kChunkList];
    int founds;
    int overflow;
};

template <int W>
__device__ __forceinline__ void put_words(uint32_t* to, const uint32_t (&v)[W]) {
    if constexpr (W == 2) *reinterpret_cast<uint2*>(to) = make_uint2(v[0], v[1]);
    else *to = v[0];
}

// T threads per row: a CTA, or (32) one of the kUnitsPerCta warps of a CTA, which then
// need no barrier and overlap one row's end with other rows' loads.
//
// Bound by the one read of x: 2048 rows of 128256 bf16 with K = 20 in 90 us, 5.9 TB/s
// (K = 0: 84); 599 of 200003 f32 with K = 20 in 75, 6.4 TB/s.  Eight 16-byte loads per
// thread (64 registers, 32 warps per SM) keep 128 KB per SM in flight.  bf16 issues at 58 %
// of the rate: per element an FMA, an ex2, half a packed add and half a packed FMA.  What a
// row's end costs with alternatives (bound, list, second read, ranking: about 9 us for one
// row) is hidden only by other rows' CTAs, which is what small CTAs are for; a persistent
// CTA that fetched its next row meanwhile measured 101 us.  One row alone is latency: 6.4
// us on 8 CTAs, of it about 2 for the launch.
template <int DT, int T, bool CLUSTER>
__global__ void __launch_bounds__(T == 32 ? 32 * kUnitsPerCta : T, T == 32 ? 32 / kUnitsPerCta : 1024 / T)
lse_stats_kernel(const __grid_constant__ StatsArgs a) {
    constexpr int U = stat_u(T), MW = U / 4, NW = T / 32, EPV = 16 / DType<DT>::bytes, UNITS = T == 32 ? kUnitsPerCta : 1;
    __shared__ StatsShared<T, CLUSTER> sh_units[UNITS];
    StatsShared<T, CLUSTER>& sh = sh_units[UNITS > 1 ? threadIdx.x / 32 : 0];
    constexpr int kFoundList = StatsShared<T, CLUSTER>::kFoundList;
    float* const group_max = reinterpret_cast<float*>(sh.group_max4);
    const int tid = UNITS > 1 ? threadIdx.x & 31 : threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const auto sync = [] {
        if (T == 32) __syncwarp();
        else __syncthreads();
    };
    pdl_trigger();
    if (CLUSTER) cluster_arrive();  // (waited for before the first remote store)
    pdl_wait();

    const int P = CLUSTER ? a.cluster : 1;
    const int64_t row = UNITS > 1 ? static_cast<int64_t>(blockIdx.x) * UNITS + threadIdx.x / 32 : blockIdx.x / P;
    if (UNITS > 1 && row >= a.B) return;
    const int seg = CLUSTER ? static_cast<int>(blockIdx.x - row * P) : 0;
    const Row r = make_row<DT>(a.x, row, a.row_stride, a.N);
    const int64_t per = CLUSTER ? (r.vectors + P - 1) / P : r.vectors;
    const int64_t k_begin = seg * per < r.vectors ? seg * per : r.vectors;
    const int64_t k_end = k_begin + per < r.vectors ? k_begin + per : r.vectors;

    const bool gather = a.logprob != nullptr && seg == 0 && tid == 0;
    const int64_t target = gather ? __ldg(a.target + row) : -1;
    float xt = __int_as_float(0x7fc00000);
    if (target >= 0 && target < a.N) xt = load_elem<DT>(r.a0 + r.off, target);
    if (tid == 0) sh.founds = sh.overflow = 0;
    if (CLUSTER && tid < kMaxTopK) sh.own[tid] = 0;

    // The row, in batches of U vectors per thread.
    StatAcc acc = stat_identity();
    {
        Shift shift = make_shift<DT>(acc.m);
        constexpr uint32_t low16 = DT == kF16 ? kNegInfF16x2 : kNegInfBF16x2;
        uint32_t chunk_max[MW];
#pragma unroll
        for (int h = 0; h < MW; ++h) chunk_max[h] = low16;
        int chunk = 0, in_chunk = 0;
        for (int64_t k = k_begin + tid; k - tid < k_end; k += U * T) {
            uint32_t w[4 * U];
            if (k - tid + U * T <= k_end) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint4 v = ldg_stream16(r.a0 + (k + j * T) * 16);
                    w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < U; ++j) load_vector<DT>(r, k + j * T, k_end, &w[4 * j]);
            }
            if (k == 0 || (k - tid <= r.vectors - 1 && r.vectors - 1 < k - tid + U * T)) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    if (k + j * T == 0 || k + j * T == r.vectors - 1) mask_vector<DT>(r, k + j * T, &w[4 * j]);
                }
            }
            uint32_t maxima[MW];
            const float cm = batch_maxima<DT, U>(w, maxima);
            if (cm > acc.m) {
                acc = stat_shift<DT>(acc, cm);
                shift = make_shift<DT>(cm);
            }
            stat_add_words<DT, 4 * U>(acc, shift, w);
#pragma unroll
            for (int h = 0; h < MW; ++h) chunk_max[h] = max2<DT>(chunk_max[h], maxima[h]);
            if (++in_chunk == 1 << a.chunk_shift) {
                put_words<MW>(sh.chunk_max + (chunk * T + tid) * MW, chunk_max);
#pragma unroll
                for (int h = 0; h < MW; ++h) chunk_max[h] = low16;
                in_chunk = 0;
                ++chunk;
            }
        }
        if (in_chunk > 0) put_words<MW>(sh.chunk_max + (chunk * T + tid) * MW, chunk_max);
    }
    // The warp's maximum, and on the way to it those of `apart` neighbouring threads.
    const bool wide = a.K > kWideGroupsK;
    const int apart = wide && T > 32 ? NW / 2 : NW;
    float warp_max = acc.m;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        if (off == apart && tid % apart == 0) group_max[tid / apart] = warp_max;
        warp_max = fmaxf(warp_max, __shfl_xor_sync(0xffffffffu, warp_max, off));
    }
    if (T == 32 && wide) {
        // Two groups per lane, from its chunks' maxima (two to a word).  f32 ones have been
        // rounded to bf16, maybe up: one step down is a bound for sure.
        const int64_t batches = (k_end - k_begin + U * T - 1) / (U * T);
        const int groups = static_cast<int>((batches + (1 << a.chunk_shift) - 1) >> a.chunk_shift);
        uint32_t both = DT == kF16 ? kNegInfF16x2 : kNegInfBF16x2;
        for (int c = 0; c < groups; ++c) both = max2<DT>(both, sh.chunk_max[(c * T + tid) * MW]);
        group_max[lane] = step_down<DT>(half_lo<DT>(both));
        group_max[lane + 32] = step_down<DT>(half_hi<DT>(both));
    }
    acc = stat_shift<DT>(acc, warp_max);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        acc.s += __shfl_xor_sync(0xffffffffu, acc.s, off);
        acc.u += __shfl_xor_sync(0xffffffffu, acc.u, off);
    }
    if (lane == 0) {
        sh.part[0][wid] = acc.m;
        sh.part[1][wid] = acc.s;
        sh.part[2][wid] = acc.u;
    }
    sync();
    bool nan = false;
#pragma unroll
    for (int w = 0; w < NW; ++w) nan |= sh.part[1][w] != sh.part[1][w];
    if (wid == 0) {
        acc = lane < NW ? StatAcc{sh.part[0][lane], sh.part[1][lane], sh.part[2][lane]} : stat_identity();
        acc = stat_lanes_merge<DT, NW>(acc);
        if (!CLUSTER && lane == 0) {
            const RowStats rs = row_stats<DT>(acc);
            sh.row = rs;
            put_row(a, row, acc, rs, xt);
        }
    }

    if (a.K > 0) {
        const float bound = wide ? kth_largest_of<64>(group_max, a.K, lane)
                                 : kth_largest_of<32>(group_max, a.K, lane);
        bool scan = nan || bound == __int_as_float(kNegInfF32);  // NaN, or too few left
        if (!scan && warp_max >= bound) {
            const int batches = static_cast<int>((k_end - k_begin + U * T - 1) / (U * T));
            const int groups = (batches + (1 << a.chunk_shift) - 1) >> a.chunk_shift;
            // The thread's chunks that reach the bound, a bit each; then one of them per
            // lane and round goes to the warp's list.
            uint64_t flags = 0;
            const float bound16 = round16<DT>(bound);
#pragma unroll 4
            for (int c = 0; c < groups; ++c) {
                uint32_t f = 0;
#pragma unroll
                for (int h = 0; h < MW; ++h) {
                    const uint32_t m = sh.chunk_max[(c * T + tid) * MW + h];
                    f |= (half_lo<DT>(m) >= bound16 ? 1u : 0u) << (2 * h) | (half_hi<DT>(m) >= bound16 ? 2u : 0u) << (2 * h);
                }
                flags |= static_cast<uint64_t>(f) << (2 * MW * c);
            }
            int n = 0;
            for (uint32_t who; (who = __ballot_sync(0xffffffffu, flags != 0)) != 0; n += __popc(who)) {
                if (flags == 0) continue;
                const int c = __ffsll(static_cast<long long>(flags)) - 1;
                flags &= flags - 1;
                const int at = n + __popc(who & ((1u << lane) - 1));
                if (at < kChunkList) sh.chunk[wid][at] = static_cast<int16_t>(c * 32 + lane);
            }
            if (n > kChunkList) {
                n = 0;
                sh.overflow = 1;
            }
            __syncwarp();
            const int item_shift = 1 + a.chunk_shift;  // log2 of a chunk's vectors
            const int items = n << item_shift;
            // H vectors of the chunks per lane and round: two for one-warp rows, which read
            // all of the row's chunks.
            constexpr int H = T == 32 ? 2 : 1;
            int found = 0;  // (one-warp rows count for themselves)
            for (int i0 = 0; i0 < items; i0 += 32 * H) {
                uint32_t w[4 * H], col[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int i = i0 + 32 * h + lane;
                    const int c = i < items ? sh.chunk[wid][i >> item_shift] : 0;
                    const int e0 = i & ((1 << item_shift) - 1);  // which of the chunk's vectors
                    // (a part's vectors fit 32 bits: N does)
                    const int pair = (c >> 5) % (U / 2);
                    const int batch = ((c >> 5) / (U / 2) << a.chunk_shift) + (e0 >> 1);
                    const int k = (batch * U + pair * 2 + (e0 & 1)) * T + wid * 32 + (c & 31);
                    load_vector<DT>(r, k_begin + k, i < items ? k_end : 0, &w[4 * h]);
                    col[h] = static_cast<uint32_t>(column_of<DT>(r, k_begin + k, 0));  // (wraps before the row)
                }
                uint32_t mine = 0;
#pragma unroll
                for (int e = 0; e < H * EPV; ++e)
                    mine |= (word_elem<DT>(&w[e / EPV * 4], e % EPV) >= bound ? 1u : 0u) << e;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (col[h] > static_cast<uint32_t>(a.N) - EPV) {  // the row's ends: elements outside it
#pragma unroll
                        for (int e = 0; e < EPV; ++e)
                            if (col[h] + e >= a.N) mine &= ~(1u << (h * EPV + e));
                    }
                int at = found;
                if (T > 32) {
                    const int total = __reduce_add_sync(0xffffffffu, __popc(mine));
                    if (total == 0) continue;
                    if (lane == 0) at = atomicAdd(&sh.founds, total);
                    at = __shfl_sync(0xffffffffu, at, 0);
                }
                for (uint32_t who; (who = __ballot_sync(0xffffffffu, mine != 0)) != 0; at += __popc(who)) {
                    if (mine == 0) continue;
                    const int e = __ffs(mine) - 1;
                    mine &= mine - 1;
                    const int place = at + __popc(who & ((1u << lane) - 1));
                    const uint32_t column = (H == 1 || e < EPV ? col[0] : col[H - 1] - EPV) + e;
                    if (place < kFoundList) sh.found[place] = topk_key(pick_elem<DT, 4 * H>(w, e), column);
                }
                if (T == 32) found = at;
            }
            if (T == 32 && lane == 0) sh.founds = found;
        }
        sync();
        scan = scan || sh.overflow != 0 || sh.founds > kFoundList;
        const int n = scan ? T : sh.founds;
        if (scan) {  // a part of the vectors per warp, in order
            sync();
            const int64_t share = (k_end - k_begin + NW - 1) / NW;
            const int64_t k0 = k_begin + wid * share < k_end ? k_begin + wid * share : k_end;
            const int64_t k1 = k0 + share < k_end ? k0 + share : k_end;
            sh.found[tid] = scan_vectors<DT>(r, k0, k1, a.N, a.K, lane);
            sync();
        }
        if (!CLUSTER) {
            const RowStats rs = sh.row;
            rank_keys<T == 32 ? 1 : 4>(sh.found, n, a.K, tid, T, [&](int place, uint64_t key) { put_top(a, row, place, key, rs); });
            return;
        }
        // A part hands on what it found, or the K largest of many.
        int count = n;
        const uint64_t* from = sh.found;
        if (n > kPartKeys) {
            rank_keys<4>(sh.found, n, a.K, tid, T, [&](int place, uint64_t key) { sh.own[place] = key; });
            count = a.K;
            from = sh.own;
            sync();
        }
        cluster_wait();
        if (tid < count) cluster_map(sh.keys, 0)[seg * kPartKeys + tid] = from[tid];
        if (tid == 0) cluster_map(sh.key_count, 0)[seg] = count;
        const int groups_here = (wide ? 64 : 32) / P;  // of its threads
        if (tid >= T - 32 && lane < groups_here) {
            float m = group_max[lane * P];
            for (int i = 1; i < P; ++i) m = fmaxf(m, group_max[lane * P + i]);
            reinterpret_cast<float*>(cluster_map(sh.cluster_max4, 0))[seg * groups_here + lane] = m;
        }
    } else if (CLUSTER) {
        cluster_wait();
    }
    if (CLUSTER) {
        if (tid == 0) {
            float* to = cluster_map(&sh.acc[0][0], 0) + seg;
            to[0] = acc.m;
            to[kMaxCluster] = acc.s;
            to[2 * kMaxCluster] = acc.u;
        }
        cluster_arrive();
        if (seg != 0) return;
        cluster_wait();
        if (wid == 0) {
            acc = lane < P ? StatAcc{sh.acc[0][lane], sh.acc[1][lane], sh.acc[2][lane]} : stat_identity();
            acc = stat_lanes_merge<DT, kMaxCluster>(acc);
            if (lane == 0) {
                const RowStats rs = row_stats<DT>(acc);
                sh.row = rs;
                put_row(a, row, acc, rs, xt);
            }
        }
        if (a.K == 0) return;
        // Of the parts' keys, those that reach the bound of the whole row.
        static_assert(!CLUSTER || (kMaxCluster * kPartKeys * 2 <= sizeof(sh.chunk_max) / 4 && kPartKeys % 16 == 0), "whole warps");
        uint64_t* reached = reinterpret_cast<uint64_t*>(sh.chunk_max);  // (no longer needed)
        if (tid == 0) sh.founds = 0;
        const float* const cluster_max = reinterpret_cast<const float*>(sh.cluster_max4);
        const float bound = wide ? kth_largest_of<64>(cluster_max, a.K, lane) : kth_largest_of<32>(cluster_max, a.K, lane);
        __syncthreads();
        for (int i = tid; i < P * kPartKeys; i += T) {
            const int part = i / kPartKeys;
            const uint64_t key = i - part * kPartKeys < sh.key_count[part] ? sh.keys[i] : 0;
            const bool in = key != 0 && !(key_value(key) < bound);  // (a NaN reaches every bound)
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            if (who == 0) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&sh.founds, __popc(who));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
            if (in) reached[at] = key;
        }
        __syncthreads();
        const RowStats rs = sh.row;
        rank_keys<4>(reached, sh.founds, a.K, tid, T, [&](int place, uint64_t key) { put_top(a, row, place, key, rs); });
    }
}

// ---------------------------------------------------------------------------
// Short rows: G lanes per row, which hold it in registers (V vectors per lane).  The
// bound comes from the maxima of G lanes, or (M = 2) of 2 G half lanes.
// ---------------------------------------------------------------------------
constexpr int kShortThreads = 256;
constexpr int kShortWarps = kShortThreads / 32;
// Elements of a warp's rows that may reach their bounds.
__host__ __device__ constexpr int short_found(int G) { return G == 32 ? 192 : 128; }

// Keys of short rows: f32 ones as elsewhere; a 16-bit element's fits 32 bits, its
// ordered bits above the complement of its column (< 2^16).  No NaN comes here.
template <int DT> struct ShortKey {
    using type = uint32_t;
    static __device__ __forceinline__ uint32_t make(const char* p, int column) {
        uint32_t b = *reinterpret_cast<const unsigned short*>(p);
        if (b == 0x8000u) b = 0;  // -0
        return ((b ^ ((b & 0x8000u) ? 0xffffu : 0x8000u)) << 16) | (0xffffu - static_cast<uint32_t>(column));
    }
    static __device__ __forceinline__ float value(uint32_t k) {
        const uint32_t o = k >> 16;
        return word_lo<DT>(o ^ ((o & 0x8000u) ? 0x8000u : 0xffffu));
    }
    static __device__ __forceinline__ int64_t column(uint32_t k) { return 0xffff - static_cast<int>(k & 0xffffu); }
};
template <> struct ShortKey<kF32> {
    using type = uint64_t;
    static __device__ __forceinline__ uint64_t make(const char* p, int column) {
        return topk_key(*reinterpret_cast<const float*>(p), static_cast<uint32_t>(column));
    }
    static __device__ __forceinline__ float value(uint64_t k) { return key_value(k); }
    static __device__ __forceinline__ int64_t column(uint64_t k) { return key_column(k); }
};

template <bool WIDE> struct ShortBits {
    using type = uint32_t;
    static __device__ __forceinline__ int first(uint32_t b) { return __ffs(static_cast<int>(b)) - 1; }
};
template <> struct ShortBits<true> {
    using type = uint64_t;
    static __device__ __forceinline__ int first(uint64_t b) { return __ffsll(static_cast<long long>(b)) - 1; }
};

// Bound by instructions wherever alternatives are asked for: 65536 rows of 261 f32 in 17 us
// with K = 0 and 30.6 with K = 8 (340 instructions per row, four rows per warp, 63 % of the
// issue rate), against 11.2 for the bytes.  The row stays in registers (V is a template
// parameter, so no lane loops), and a copy in shared memory serves to pick elements by
// number.  Fewer lanes per row cost fewer shuffles but more registers; M = 2 halves the
// elements that reach the bound when nearly all of the lanes' maxima are among the K
// (468750 rows of 256 bf16, K = 32: 445 us against 983 with the second value left empty).
template <int DT, int G, int M, int V>
__global__ void __launch_bounds__(kShortThreads, V <= 4 ? 5 : V <= 6 ? 4 : 3)
lse_stats_short_kernel(const __grid_constant__ StatsArgs a) {
    constexpr int EB = DType<DT>::bytes, EPV = 16 / EB, RPW = 32 / G;
    static_assert(V * EPV <= 64, "a bit for each of a lane's elements");
    constexpr int kShortFound = short_found(G);
    constexpr int kCap = kShortFound / RPW - 4;  // per row (and room for empty keys after the last)
    using Key = typename ShortKey<DT>::type;
    __shared__ uint4 stage_all[kShortWarps][32 * V];  // the warp's vectors, to be picked from
    __shared__ alignas(16) Key found_all[kShortWarps][kShortFound];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int sub = lane & (G - 1), group = lane / G;
    uint4* const stage = stage_all[wid];
    Key* const found = found_all[wid] + group * (kShortFound / RPW);
    pdl_trigger();
    pdl_wait();
    for (int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kShortWarps + wid) * RPW; row0 < a.B;
         row0 += static_cast<int64_t>(gridDim.x) * kShortWarps * RPW) {
        const int64_t row = row0 + group;
        const bool live = RPW == 1 || row < a.B;
        // Short rows: everything inside one fits 32 bits.
        const char* rp = static_cast<const char*>(a.x) + row * a.row_stride * EB;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(rp) & 15u);
        const char* a0 = rp - off;
        const int end = off + static_cast<int>(a.N) * EB;
        const int vectors = live && a.N > 0 ? (end + 15) >> 4 : 0;
        uint32_t w[4 * V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (sub + G * j < vectors) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(a0 + (sub + G * j) * 16));
                w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
            } else {
                w[4 * j] = w[4 * j + 1] = w[4 * j + 2] = w[4 * j + 3] = neg_inf_word<DT>();
            }
        }
        float xt = __int_as_float(0x7fc00000);
        if (a.logprob && sub == 0 && live) {
            const int64_t t = __ldg(a.target + row);
            if (t >= 0 && t < a.N) xt = load_elem<DT>(rp, t);
        }
        if (off != 0 && sub == 0) {
            uint32_t q[4] = {w[0], w[1], w[2], w[3]};
            mask_prefix<DT>(q, off);
            w[0] = q[0]; w[1] = q[1]; w[2] = q[2]; w[3] = q[3];
        }
        if ((end & 15) != 0) {
            const int last = vectors - 1;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (sub + G * j == last) {
                    uint32_t q[4] = {w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
                    mask_suffix<DT>(q, end - last * 16);
                    w[4 * j] = q[0]; w[4 * j + 1] = q[1]; w[4 * j + 2] = q[2]; w[4 * j + 3] = q[3];
                }
        }
        float part_max[M];
        float m;
        if constexpr (M == 1) {
            m = part_max[0] = words_max<DT, 4 * V>(w);
        } else {  // the halves of the lane's words
            uint32_t half[2 * V];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) half[i] = w[2 * V * q + i];
                part_max[q] = words_max<DT, 2 * V>(half);
            }
            m = fmaxf(part_max[0], part_max[1]);
        }
#pragma unroll
        for (int off2 = G / 2; off2 > 0; off2 >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off2));
        StatAcc acc{m, 0.0f, 0.0f};
        stat_add_words<DT, 4 * V>(acc, make_shift<DT>(m), w);
#pragma unroll
        for (int off2 = G / 2; off2 > 0; off2 >>= 1) {
            acc.s += __shfl_xor_sync(0xffffffffu, acc.s, off2);
            acc.u += __shfl_xor_sync(0xffffffffu, acc.u, off2);
        }
        const RowStats rs = row_stats<DT>(acc);
        if (sub == 0 && live) put_row(a, row, acc, rs, xt);
        if (a.K == 0) continue;

        const float bound = kth_largest<G, M>(part_max, a.K, lane);
        bool scan = acc.s != acc.s || bound == __int_as_float(kNegInfF32);
        // Which of the lane's elements reach the bound, one bit each; then one of them
        // per lane and round goes to the row's list, in turn within the round.
        using Bits = typename ShortBits<(V * EPV > 32)>::type;
        Bits mine = 0;
#pragma unroll
        for (int i = 0; i < V * EPV; ++i)
            mine |= static_cast<Bits>(word_elem<DT>(&w[i / EPV * 4], i % EPV) >= bound ? 1 : 0) << i;
        if (scan || !live) mine = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) stage[32 * j + lane] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        int n = 0;
        const int column0 = (sub * 16 - off) / EB;
        const uint32_t group_bits = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1) << (group * G);
        const uint32_t before = group_bits & ((1u << lane) - 1);
        for (uint32_t who; (who = __ballot_sync(0xffffffffu, mine != 0)) != 0;) {
            if (mine != 0) {
                const int i = ShortBits<(V * EPV > 32)>::first(mine);
                mine &= mine - 1;
                const int at = n + __popc(who & before);
                if (at < kCap)
                    found[at] = ShortKey<DT>::make(reinterpret_cast<const char*>(stage + 32 * (i / EPV) + lane) + i % EPV * EB,
                                                   column0 + (i / EPV) * (G * EPV) + i % EPV);
            }
            n += __popc(who & group_bits);
        }
        scan |= n > kCap;
        if (!scan && sub < 4) found[n + sub] = 0;
        __syncwarp();
        if (!scan) {
            constexpr int PER = 16 / sizeof(Key);  // keys per load
            for (int i = sub; i < n; i += G) {
                const Key key = found[i];
                int rank = 0;
                for (int j = 0; j < n; j += PER) {
                    const uint4 v = *reinterpret_cast<const uint4*>(found + j);
                    if constexpr (PER == 4) {
                        rank += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
                    } else {
                        rank += ((static_cast<uint64_t>(v.y) << 32 | v.x) > key) + ((static_cast<uint64_t>(v.w) << 32 | v.z) > key);
                    }
                }
                if (rank < a.K) {
                    a.top_index[row * a.K + rank] = ShortKey<DT>::column(key);
                    a.top_logprob[row * a.K + rank] = stat_logprob(ShortKey<DT>::value(key), rs);
                }
            }
        }
        // Rows that need the scan, by the whole warp in turn.
        uint32_t todo = __ballot_sync(0xffffffffu, scan && live && sub == 0);
        while (todo != 0) {
            const int q = __ffs(todo) - 1;
            todo &= todo - 1;
            const Row r = make_row<DT>(a.x, row0 + q / G, a.row_stride, a.N);
            const uint64_t key = scan_vectors<DT>(r, 0, r.vectors, a.N, a.K, lane);
            const RowStats of{__shfl_sync(0xffffffffu, rs.m, q), __shfl_sync(0xffffffffu, rs.lse, q),
                              __shfl_sync(0xffffffffu, rs.logs, q)};
            if (lane < a.K) put_top(a, row0 + q / G, lane, key, of);
        }
        __syncwarp();
    }
}

template <int DT, int T, bool CLUSTER>
cudaError_t launch_stats_long(const StatsArgs& a, cudaStream_t stream) {
    const auto kernel = lse_stats_kernel<DT, T, CLUSTER>;
    const int64_t ctas = T == 32 ? (a.B + kUnitsPerCta - 1) / kUnitsPerCta : a.B * a.cluster;
    const dim3 grid(static_cast<unsigned>(ctas));
    if (!CLUSTER) return launch_pdl(kernel, grid, dim3(T == 32 ? 32 * kUnitsPerCta : T), stream, a);
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(T);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaSuccess;
    if (a.cluster > 8) {  // more than the portable size: allowed once per device
        static std::atomic<uint64_t> allowed{0};
        int dev = 0;
        e = cudaGetDevice(&dev);
        const uint64_t bit = 1ull << (dev & 63);
        if (e == cudaSuccess && (allowed.load() & bit) == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) allowed.fetch_or(bit);
        }
    }
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int DT, int G, int M>
cudaError_t launch_stats_short(const StatsArgs& a, int64_t vectors, int sms, cudaStream_t stream) {
    const int64_t rows = kShortWarps * (32 / G);
    const int64_t ctas = (a.B + rows - 1) / rows;
    const int64_t most = static_cast<int64_t>(sms) * 64;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most)), block(kShortThreads);
    switch ((vectors + G - 1) / G) {
    case 0:
    case 1: return launch_pdl(lse_stats_short_kernel<DT, G, M, 1>, grid, block, stream, a);
    case 2: return launch_pdl(lse_stats_short_kernel<DT, G, M, 2>, grid, block, stream, a);
    case 3: return launch_pdl(lse_stats_short_kernel<DT, G, M, 3>, grid, block, stream, a);
    case 4: return launch_pdl(lse_stats_short_kernel<DT, G, M, 4>, grid, block, stream, a);
    case 5: return launch_pdl(lse_stats_short_kernel<DT, G, M, 5>, grid, block, stream, a);
    case 6: return launch_pdl(lse_stats_short_kernel<DT, G, M, 6>, grid, block, stream, a);
    case 7:
    case 8: return launch_pdl(lse_stats_short_kernel<DT, G, M, 8>, grid, block, stream, a);
    default:
        if constexpr (G < 32 && DT == kF32) return launch_pdl(lse_stats_short_kernel<DT, G, M, 10>, grid, block, stream, a);
        else return cudaErrorInvalidValue;
    }
}

// The mapping of a call: rows of up to 256 vectors take a warp each; longer ones a
// CTA, or a cluster of CTAs while the rows alone would leave SMs without work.
template <int DT>
cudaError_t launch_stats(StatsArgs a, int sms, cudaStream_t stream) {
    const int eb = DType<DT>::bytes;
    const bool aligned = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.row_stride * eb) % 16 == 0;
    const int64_t vectors = (a.N * eb + 15) / 16 + (aligned ? 0 : 1);  // at most
    a.cluster = 1;
    a.chunk_shift = 0;
    if (vectors <= 32 * 8) {
        // The fewest lanes per row that hold it in 10 vectors each (16-bit types: 8), and of
        // whose maxima (or half lanes') not nearly all are needed for K.
        const int V = eb == 4 ? 10 : 8;
        if (vectors <= 8 * V && a.K <= 8)
            return a.K <= 4 ? launch_stats_short<DT, 8, 1>(a, vectors, sms, stream)
                            : launch_stats_short<DT, 8, 2>(a, vectors, sms, stream);
        if (vectors <= 16 * V && a.K <= 24)
            return a.K <= 8 ? launch_stats_short<DT, 16, 1>(a, vectors, sms, stream)
                            : launch_stats_short<DT, 16, 2>(a, vectors, sms, stream);
        return a.K <= 24 ? launch_stats_short<DT, 32, 1>(a, vectors, sms, stream)
                         : launch_stats_short<DT, 32, 2>(a, vectors, sms, stream);
    }
    // Threads of a CTA: 256 while rows are few (10 rows of 16384 bf16: 4.8 us against 5.8
    // with 128); otherwise 128, so that rows at their ends overlap with more rows under way
    // (400 rows of 8192 f32: 7.0 against 7.3), but for long rows 256 up to 4 rows per SM.
    int T = 256;
    if (a.B >= 4LL * sms || (a.B > 2LL * sms && vectors < 2LL * stat_u(T) * T)) T = 128;
    // Rows of up to 1024 vectors by the thousand: a warp each.
    if (vectors <= 1024 && a.B >= 16LL * sms) T = 32;
    // Few rows: a cluster of 256-thread CTAs per row, as many as leave each three quarters
    // of a batch and are all resident at once -- in 15 of 16 SMs: some take no clusters
    // (us; 128256 bf16, K = 20, one row: 6.4 with 8 CTAs, 7.4 with 4, 6.6 with 16; 200003
    // f32: 60 rows 13.6 with 8, 16.8 with 4; 76 rows 19.4 and 17.7; 144 rows 23.6 with 4,
    // 149 rows 30.3).  Two CTAs pay for the cluster's barriers only in long rows that are
    // about as many as SMs (170 of 128256 bf16, K = 20: 18.3 against 22.4), sixteen with
    // alternatives only while each has an SM to itself (200000 f16, K = 20: 8 rows 7.7
    // against 8.7 with 8, 30 rows 13.5 and 12.4; K = 0, 30 rows 7.2 and 8.6).
    int P = 1;
    if (a.B * 4 <= 5LL * sms) {
        while (2 * P <= kMaxCluster && vectors >= 2LL * P * (stat_u(256) * 256 * 3 / 4) &&
               (P == 1 || a.B * (2 * P) * 256 <= 1024LL * sms * 15 / 16) && (P < 8 || a.K == 0 || a.B * (2 * P) <= sms))
            P *= 2;
        if (P == 2 && vectors < 8192) P = 1;
    }
    a.cluster = P;
    const int64_t batches = ((vectors + P - 1) / P + stat_u(T) * T - 1) / (stat_u(T) * T);
    while ((batches + (1LL << a.chunk_shift) - 1) >> a.chunk_shift > stat_batches(T)) ++a.chunk_shift;
    if (P > 1) return launch_stats_long<DT, 256, true>(a, stream);
    switch (T) {
    case 32: return launch_stats_long<DT, 32, false>(a, stream);
    case 128: return launch_stats_long<DT, 128, false>(a, stream);
    default: return launch_stats_long<DT, 256, false>(a, stream);
    }
}

}  // namespace
}  // namespace lse

// Instantiates the per-type launch declared in lse_stats_common.cuh.
#define LSE_DEFINE_TOKEN_STATS(DT, SUFFIX)                                              \
    namespace lse {                                                                     \
    cudaError_t launch_token_stats_##SUFFIX(const StatsArgs& a, int sms, cudaStream_t s) { \
        return launch_stats<DT>(a, sms, s);                                             \
    }                                                                                   \
    }
