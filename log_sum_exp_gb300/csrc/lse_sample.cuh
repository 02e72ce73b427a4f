// lse_sample.cuh -- drawing a token from every row of logits (sm_103a).
//
// With the tokens of a row in the order (value descending, column ascending) and
// w = exp((x - m) / T), m the row's maximum:
//
//     kept   the first top_k; of these, those before which the sum of w is below top_p times
//            the sum of all of these; of these, those with x - m >= T log(min_p)
//     token  the first column n whose sum of w over the kept columns up to n passes
//            u times the sum over all kept columns
//
// Every cut keeps a prefix of the order, so what is kept is every element whose key (value,
// complement of the column) is at least a threshold key.
//
// Precision.  A token changes where a sum passes a border, and a row has N borders, so sums
// in 32 bits would give another token than the formula in one row of a few hundred.  Weights
// are therefore whole numbers of 2^-S (S about 44): 2^z with z the distance to the maximum
// in octaves, taken apart as 2^(k/64) 2^r with the remainder r formed without rounding the
// product and a cubic for 2^r - 1; off by at most about 2^-30 of itself.  Sums of whole numbers do not
// depend on their order.  That takes about 25 instructions, twice what the memory's rate leaves
// for a bf16 element, so the pass over a whole row computes weights with ex2 instead, off by at
// most kFastError of each (2^-22 of the instruction, whose argument carries its own rounding
// error along, and the sums' roundings), and keeps a sum for every chunk of a few
// thousand columns.  Where the drawn number lies further than that from both borders of its
// token the result stands; else the row's sums are taken again exactly.
//
// Threshold.  Every lane's maximum in every chunk is kept in shared memory.  They bound the
// threshold from below (the k-th largest of them is at most the k-th largest element; the same
// for sums), and later passes read only the vectors of lanes and chunks that reach the bound:
// few for peaked rows.  What they find is put in order in shared memory; more than the list
// holds (flat rows) is first narrowed down by histograms of counts and masses over the
// bits of the ordered values.
#pragma once

#include <climits>
#include <cstdint>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_internal.h"
#include "lse_sample_common.cuh"
#include "lse_topk.cuh"

namespace lse {
namespace {

constexpr int kBatch = 8;                // vectors of a lane in flight
constexpr int kBins = 512;
constexpr int kList = 256;
constexpr float kFastError = 6e-7f;
constexpr float kInf = __builtin_inff();

// 2^(j / 64) in units of 2^-30, rounded to nearest.
__constant__ uint32_t kPowers[64] = {
    1073741824u, 1085434106u, 1097253708u, 1109202018u, 1121280436u, 1133490379u, 1145833280u, 1158310587u,
    1170923762u, 1183674286u, 1196563654u, 1209593378u, 1222764986u, 1236080024u, 1249540052u, 1263146652u,
    1276901417u, 1290805962u, 1304861917u, 1319070932u, 1333434672u, 1347954824u, 1362633090u, 1377471191u,
    1392470869u, 1407633882u, 1422962010u, 1438457051u, 1454120821u, 1469955159u, 1485961921u, 1502142985u,
    1518500250u, 1535035634u, 1551751076u, 1568648537u, 1585730000u, 1602997467u, 1620452965u, 1638098541u,
    1655936265u, 1673968228u, 1692196547u, 1710623359u, 1729250827u, 1748081133u, 1767116489u, 1786359126u,
    1805811301u, 1825475297u, 1845353420u, 1865448001u, 1885761398u, 1906295993u, 1927054196u, 1948038440u,
    1969251188u, 1990694927u, 2012372174u, 2034285470u, 2056437387u, 2078830522u, 2101467502u, 2124350982u,
};

template <int TX> __device__ __forceinline__ void row_sync() {
    if constexpr (TX == 32) __syncwarp();
    else __syncthreads();
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// floor(f t) for f < 1 (0 for a negative or NaN f), exactly; whether nothing was cut off.
__device__ __forceinline__ uint64_t part_of(uint64_t t, float f, bool* whole) {
    *whole = true;
    if (!(f > 0.0f)) return 0;
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - static_cast<int>(e ? e : 1);  // f = m 2^-s, s >= 24
    const uint64_t hi = __umul64hi(m, t), lo = m * t;
    const uint64_t q = s < 64 ? (hi << (64 - s)) | (lo >> s) : s < 128 ? hi >> (s - 64) : 0;
    // the product of q and 2^s again: what is left shows whether it was whole
    if (s < 64) *whole = (lo & ((1ull << s) - 1)) == 0;
    else *whole = lo == 0 && (s < 128 ? (hi & ((1ull << (s - 64)) - 1)) == 0 : hi == 0);
    return q;
}

// What a row's kernel shares between its threads.
template <int TX> struct SampleShared {
    static constexpr int W = TX / 32;
    uint32_t powers[64];
    uint32_t count[kBins], mass[kBins];
    uint64_t list[kList];
    uint64_t weights[kList];
    uint64_t warp64[W + 1];
    float warpf[W];
    uint64_t r64[4];
    uint32_t r32[4];
};

template <int DT, int TX> struct Sampler {
    static constexpr int W = TX / 32, EB = DType<DT>::bytes, E = 16 / EB;
    SampleShared<TX>& sh;
    // the row
    const char* base;  // the 16-byte boundary at or before its first element
    int off, end;      // its first and last bytes (end: in the last vector, from its start)
    int slots;         // vectors that cover it
    int N;
    int per_warp, chunk, chunks_per_warp, chunks;  // vectors of a warp's range, of a chunk; chunks
    // per chunk
    float* maxima;     // [chunks, 32]
    uint64_t* sums;    // [chunks + 1]: sums, then sums before
    // weights
    float m, ch, cl;   // maximum; log2 e / T in two floats
    int S;             // fractional bits of a weight
    int lane, warp;

    __device__ __forceinline__ Sampler(SampleShared<TX>& s) : sh(s), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {}

    // -----------------------------------------------------------------------
    // Elements
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void load(int slot, uint32_t (&w)[4]) const {
        const uint4 v = ldg_stream16(base + static_cast<int64_t>(slot) * 16);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        if ((slot == 0 && off != 0) || slot == slots - 1)
            mask_words<DT>(w, 0, slot == 0 ? off : 0, slot == slots - 1 ? end : 16);
    }
    __device__ __forceinline__ int column(int slot, int e) const { return slot * E + e - off / EB; }
    __device__ __forceinline__ int chunk_begin(int c) const {
        const int w = c / chunks_per_warp;
        return w * per_warp + (c - w * chunks_per_warp) * chunk;
    }
    __device__ __forceinline__ int chunk_end(int c) const {
        const int w = c / chunks_per_warp;
        return min(min(chunk_begin(c) + chunk, (w + 1) * per_warp), slots);
    }

    // The weight of an element, a whole number of 2^-S.
    __device__ __forceinline__ uint64_t weight(float x) const {
        const float d = x - m;
        if (!(d * ch >= -static_cast<float>(S + 1))) return 0;
        const float a = d + m, b = d - a, dl = (x - a) + (-m - b);  // x - m = d + dl
        const float kf = fmaf(d, ch * 64.0f, 12582912.0f);
        const int k = __float_as_int(kf) - 0x4b400000;
        float r = fmaf(d, ch, (kf - 12582912.0f) * -0.015625f);
        r = fmaf(d, cl, r);
        r = fmaf(dl, ch, r);
        const float q = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);
        const uint32_t t = sh.powers[k & 63];
        const uint32_t p = t + __float2int_rn(static_cast<float>(t) * q);
        const int s = S - 30 + (k >> 6);
        return s >= 0 ? static_cast<uint64_t>(p) << s : (static_cast<uint64_t>(p) + (1ull << (-s - 1))) >> -s;
    }
    // 2^((x - m) log2 e / T) for x <= m.
    __device__ __forceinline__ double factor(float x) const {
        const float d = x - m;
        if (!(d * ch >= -900.0f)) return 0.0;
        const float a = d + m, b = d - a, dl = (x - a) + (-m - b);
        const float kf = fmaf(d, ch * 64.0f, 12582912.0f);
        const int k = __float_as_int(kf) - 0x4b400000;
        float r = fmaf(d, ch, (kf - 12582912.0f) * -0.015625f);
        r = fmaf(d, cl, r);
        r = fmaf(dl, ch, r);
        const float q = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);
        const uint32_t t = sh.powers[k & 63];
        const uint32_t p = t + __float2int_rn(static_cast<float>(t) * q);
        return static_cast<double>(p) * __hiloint2double((1023 - 30 + (k >> 6)) << 20, 0);
    }

    // f(x, column) for a lane's elements of a chunk, where the lane has one of at least `lo`.
    template <class F> __device__ __forceinline__ void each(int c, uint32_t lo, F&& f) const {
        if (order_bits(maxima[c * 32 + lane]) < lo) return;
        const int stop = chunk_end(c);
        for (int s = chunk_begin(c) + lane; s < stop; s += 32) {
            uint32_t w[4];
            load(s, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = word_elem<DT>(w, e);
                if (order_bits(x) >= lo) f(x, column(s, e));
            }
        }
    }
    static __device__ __forceinline__ uint64_t key(float x, int col) {
        return (static_cast<uint64_t>(order_bits(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
    }

    // -----------------------------------------------------------------------
    // Reductions
    // -----------------------------------------------------------------------
    __device__ __forceinline__ float row_max(float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if constexpr (TX == 32) return v;
        if (lane == 0) sh.warpf[warp] = v;
        __syncthreads();
        v = sh.warpf[lane % W];
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        __syncthreads();
        return __shfl_sync(0xffffffffu, v, 0);
    }
    __device__ __forceinline__ uint64_t warp_sum(uint64_t v) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    __device__ __forceinline__ uint64_t row_sum(uint64_t v) {
        v = warp_sum(v);
        if constexpr (TX == 32) return v;
        if (lane == 0) sh.warp64[warp] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) v += sh.warp64[i];
        __syncthreads();
        return v;
    }
    // The sum of v over the threads before this one.
    __device__ __forceinline__ uint64_t row_before(uint64_t v) {
        uint64_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t b = shfl_up64(s, o);
            if (lane >= o) s += b;
        }
        if constexpr (TX > 32) {
            if (lane == 31) sh.warp64[warp] = s;
            __syncthreads();
            for (int i = 0; i < warp; ++i) s += sh.warp64[i];
            __syncthreads();
        }
        return s - v;
    }

    // -----------------------------------------------------------------------
    // Sums over chunks, and the column at which a running sum passes a target
    // -----------------------------------------------------------------------
    // sums[c] to the sums before chunk c; returns the sum of all.
    __device__ __forceinline__ uint64_t scan_chunks() {
        row_sync<TX>();
        if (warp == 0) {
            uint64_t run = 0;
            for (int c0 = 0; c0 < chunks; c0 += 32) {
                const uint64_t v = c0 + lane < chunks ? sums[c0 + lane] : 0;
                uint64_t s = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t b = shfl_up64(s, o);
                    if (lane >= o) s += b;
                }
                if (c0 + lane < chunks) sums[c0 + lane] = run + s - v;
                run += __shfl_sync(0xffffffffu, s, 31);
            }
            if (lane == 0) sums[chunks] = run;
        }
        row_sync<TX>();
        return sums[chunks];
    }
    // The sums of f(x, column) over the chunks, elements below `lo` counting 0.
    template <class F> __device__ __forceinline__ uint64_t sum_chunks(uint32_t lo, F&& f) {
        row_sync<TX>();
        for (int i = 0; i < chunks_per_warp; ++i) {
            const int c = warp * chunks_per_warp + i;
            uint64_t s = 0;
            each(c, lo, [&](float x, int col) { s += f(x, col); });
            __syncwarp();
            s = warp_sum(s);
            if (lane == 0) sums[c] = s;
        }
        return scan_chunks();
    }
    // The first column at which the running sum of f passes `target`; sums are scanned.
    // Sets the sums before it and with it; false if there is none in the chunk that the
    // chunks' sums name (they may be approximate).
    template <class F>
    __device__ __forceinline__ bool locate(uint64_t target, F&& f, int* col, float* value, uint64_t* before, uint64_t* with) {
        if (threadIdx.x == 0) sh.r32[1] = 0;
        row_sync<TX>();
        for (int c = threadIdx.x; c < chunks; c += TX)
            if (sums[c] <= target && target < sums[c + 1]) sh.r32[0] = c, sh.r32[1] = 1;
        row_sync<TX>();
        const bool any = sh.r32[1] != 0;
        const int c = sh.r32[0];
        row_sync<TX>();
        if (threadIdx.x == 0) sh.r32[1] = 0;
        if (!any) {
            row_sync<TX>();
            return false;
        }
        const int b = chunk_begin(c), n = chunk_end(c) - b;
        const int per = (n + TX - 1) / TX, s0 = b + threadIdx.x * per, s1 = min(s0 + per, b + n);
        uint64_t own = 0;
        for (int s = s0; s < s1; ++s) {
            uint32_t w[4];
            load(s, w);
#pragma unroll
            for (int e = 0; e < E; ++e) own += f(word_elem<DT>(w, e), column(s, e));
        }
        const uint64_t first = row_before(own);
        const uint64_t rest = target - sums[c];
        row_sync<TX>();
        if (first <= rest && rest < first + own) {
            uint64_t run = first;
            bool found = false;
            for (int s = s0; s < s1 && !found; ++s) {
                uint32_t w[4];
                load(s, w);
                for (int e = 0; e < E && !found; ++e) {
                    const float x = word_elem<DT>(w, e);
                    const uint64_t v = f(x, column(s, e));
                    if (run + v > rest) {
                        sh.r32[0] = column(s, e);
                        sh.r32[1] = 1;
                        sh.r32[2] = __float_as_uint(x);
                        sh.r64[0] = sums[c] + run;
                        sh.r64[1] = sums[c] + run + v;
                        found = true;
                    }
                    run += v;
                }
            }
        }
        row_sync<TX>();
        const bool ok = sh.r32[1] != 0;
        *col = sh.r32[0];
        *value = __uint_as_float(sh.r32[2]);
        *before = sh.r64[0];
        *with = sh.r64[1];
        row_sync<TX>();
        return ok;
    }

    // -----------------------------------------------------------------------
    // Pass over the row: maxima, and sums of fast weights relative to a shift of the warp's
    // -----------------------------------------------------------------------
    __device__ __forceinline__ float batch_sum(const uint32_t (&w)[4 * kBatch], float mu, float dmin) const {
        uint64_t acc[4] = {0, 0, 0, 0};
        const uint64_t mu2 = f2_pack(mu, mu), ch2 = f2_pack(ch, ch), nch2 = f2_pack(-ch, -ch), ncl2 = f2_pack(-cl, -cl);
        const uint64_t nln2 = f2_pack(-kLn2, -kLn2), one2 = f2_pack(1.0f, 1.0f);
#pragma unroll
        for (int i = 0; i < 4 * kBatch; ++i) {
            uint64_t x;
            if constexpr (DT == kF32) {
                if (i & 1) continue;
                x = f2_pack(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
            } else {
                x = f2_pack(word_lo<DT>(w[i]), word_hi<DT>(w[i]));
            }
            uint64_t d = f2_sub(x, mu2);
            uint64_t dl = 0;
            float d0, d1;
            if constexpr (DT == kF32) {  // what the difference of two f32 loses
                const uint64_t a = f2_add(d, mu2), b = f2_sub(d, a);
                dl = f2_add(f2_sub(x, a), f2_sub(f2_pack(-mu, -mu), b));
                float l0, l1;
                f2_unpack(d, d0, d1);
                f2_unpack(dl, l0, l1);
                dl = f2_pack(d0 > dmin ? l0 : 0.0f, d1 > dmin ? l1 : 0.0f);
            } else {
                f2_unpack(d, d0, d1);
            }
            // A weight of 2^-200 is 0; an infinite distance would give inf - inf below.  (A NaN stays.)
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(d0) : "f"(dmin));
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(d1) : "f"(dmin));
            d = f2_pack(d0, d1);
            const uint64_t t = f2_mul(d, ch2);
            uint64_t e = f2_fma(d, nch2, t);  // minus what the product lost
            e = f2_fma(d, ncl2, e);
            if constexpr (DT == kF32) e = f2_fma(dl, nch2, e);
            const int at = DT == kF32 ? (i >> 1) & 3 : i & 3;
            acc[at] = f2_fma(f2_ex2(t), f2_fma(e, nln2, one2), acc[at]);
        }
        float a, b;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a, b);
        return a + b;
    }

    // Leaves (sum, shift) of every chunk in `fast`; returns the lane's maximum.
    __device__ __forceinline__ float first_pass(float2* fast, bool with_sums) {
        float top = -kInf, mu = 0.0f, lim = -kInf;
        const float dmin = -200.0f / ch;
        for (int i = 0; i < chunks_per_warp; ++i) {
            const int c = warp * chunks_per_warp + i;
            const int stop = chunk_end(c);
            float cm = -kInf, hi = 0.0f, lo = 0.0f;
            for (int s0 = chunk_begin(c); s0 < stop; s0 += 32 * kBatch) {
                uint32_t w[4 * kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int s = s0 + lane + 32 * j;
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = neg_inf_word<DT>();
                    if (s < stop) load(s, v);
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[4 * j + q] = v[q];
                }
                const float bm = words_max<DT, 4 * kBatch>(w);
                cm = fmaxf(cm, bm);
                if (!with_sums) {
                    // NaN: a product with 0 and a sum keep it
                    float z = 0.0f;
#pragma unroll
                    for (int q = 0; q < 4 * kBatch; ++q) {
                        if constexpr (DT == kF32) z = __uint_as_float(w[q]) != __uint_as_float(w[q]) ? kInf - kInf : z;
                        else z = (word_lo<DT>(w[q]) != word_lo<DT>(w[q]) || word_hi<DT>(w[q]) != word_hi<DT>(w[q])) ? kInf - kInf : z;
                    }
                    hi += z;
                    continue;
                }
                if (__any_sync(0xffffffffu, bm > lim)) {  // the warp's shift goes up
                    float wm = bm;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
                    if (wm < kInf) {
                        if (hi != 0.0f) {  // sums relative to the old one (rare: a step of 64 octaves)
                            Sampler t = *this;
                            t.m = wm;
                            const double v = (static_cast<double>(hi) + static_cast<double>(lo)) * t.factor(mu);
                            hi = static_cast<float>(v);
                            lo = static_cast<float>(v - static_cast<double>(hi));
                        }
                        mu = wm;
                        lim = mu + 64.0f / ch;
                        if (!(lim > mu)) lim = mu;
                    }
                }
                const float v = batch_sum(w, mu, dmin);
                const float n = hi + v, a = n - v, b = n - a;  // hi + lo + v without loss
                lo += (hi - a) + (v - b);
                hi = n;
            }
            float s = hi + lo;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            maxima[c * 32 + lane] = cm;
            if (lane == 0) fast[c] = make_float2(s, mu);
            top = fmaxf(top, cm);
        }
        return top;
    }

    // -----------------------------------------------------------------------
    // Threshold keys
    // -----------------------------------------------------------------------
    // Histogram of the elements in [lo, hi] (ordered bits) that `source` gives: counts and
    // masses in units of 2^hs weights.
    __device__ __forceinline__ void clear_bins() {
        row_sync<TX>();
        for (int i = threadIdx.x; i < kBins; i += TX) sh.count[i] = sh.mass[i] = 0;
        row_sync<TX>();
    }
    static __device__ __forceinline__ int bin_shift(uint32_t lo, uint32_t hi) {
        const uint32_t span = hi - lo;
        return span < kBins ? 0 : 32 - __clz(span) - 9;  // (span >> shift) < 512
    }
    // From the top: the first bin at which the sum of v (+ one for every element, `over`)
    // reaches `need`, and the sum before it; kBins if none does.
    __device__ __forceinline__ int find_bin(const uint32_t* v, bool over, uint64_t need, uint64_t* before) {
        row_sync<TX>();
        if (warp == 0) {
            constexpr int P = kBins / 32;
            const int b0 = lane * P;
            uint64_t own = 0;
            for (int i = 0; i < P; ++i) own += v[b0 + i] + (over ? sh.count[b0 + i] : 0u);
            uint64_t s = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t p = shfl_up64(s, o);
                if (lane >= o) s += p;
            }
            uint64_t run = s - own;
            if (lane == 0) sh.r32[0] = kBins, sh.r64[0] = 0;
            __syncwarp();
            if (run < need && need <= s) {
                int at = b0;
                for (int i = 0; i < P; ++i) {
                    const uint64_t n = run + v[b0 + i] + (over ? sh.count[b0 + i] : 0u);
                    if (n >= need) {
                        at = b0 + i;
                        break;
                    }
                    run = n;
                }
                sh.r32[0] = at;
                sh.r64[0] = run;
            }
            if (lane == 31 && need > s) sh.r64[0] = s;
        }
        row_sync<TX>();
        const int at = sh.r32[0];
        if (before) *before = sh.r64[0];
        row_sync<TX>();
        return at;
    }

    // The threshold key of the shortest prefix (of the elements with keys >= base) whose count
    // or sum of weights reaches `need` (>= 1), given to within `err`; `base_key` where all of
    // them do not.  `total`: the sum of all weights.  *sure is false where err left it open.
    __device__ uint64_t select(bool by_mass, uint64_t need, uint64_t total, uint64_t err, uint64_t base_key, bool* sure) {
        *sure = true;
        const uint32_t top = order_bits(m);
        uint32_t lo = static_cast<uint32_t>(base_key >> 32), hi = top;
        if (by_mass) {  // lighter elements weigh nothing
            const float x = m - (S + 2) / ch;
            if (x > -kInf) lo = max(lo, order_bits(x));
        }
        lo = min(lo, hi);
        const uint32_t floor = lo;
        const int hs0 = max(0, 33 - __clzll(static_cast<long long>(total)));  // total in 31 bits
        // A bound from the lanes' maxima: they are elements, so as many of them, or as much,
        // as is needed is enough.
        bool bounded = false;
        {
            uint32_t mlo = lo, mhi = hi;
            uint64_t left = by_mass ? ((need + err) >> hs0) + 1 : need;
            for (int round = 0; round < 4; ++round) {
                const int shift = bin_shift(mlo, mhi);
                clear_bins();
                for (int i = threadIdx.x; i < chunks * 32; i += TX) {
                    const float x = maxima[i];
                    const uint32_t o = order_bits(x);
                    if (o < mlo || o > mhi) continue;
                    const int b = (mhi - o) >> shift;
                    if (by_mass) atomicAdd(&sh.mass[b], static_cast<uint32_t>(min(weight(x) >> hs0, static_cast<uint64_t>(left))));
                    else atomicAdd(&sh.count[b], 1u);
                }
                uint64_t before;
                const int b = find_bin(by_mass ? sh.mass : sh.count, false, left, &before);
                if (b == kBins) break;  // (round 0 only: later ones narrow a bin that reaches)
                const uint32_t bin_hi = mhi - (static_cast<uint32_t>(b) << shift);
                const uint32_t width = (1u << shift) - 1;
                mhi = bin_hi;
                mlo = bin_hi - mlo > width ? bin_hi - width : mlo;
                lo = mlo;
                bounded = true;
                left -= before;
                const uint32_t in_bin = sh.count[b];
                row_sync<TX>();
                if (shift == 0 || (!by_mass && in_bin <= 4)) break;
            }
        }
        uint64_t above = 0;      // count or weights of the elements with keys >= base above hi
        uint64_t left = need, range_most = total + err;
        for (int round = 0; round < 64; ++round) {  // (every histogram narrows the range: a few rounds)
            if (bounded || round > 0) {
                // Elements in the range to the list; what lies above it is summed.
                if (threadIdx.x == 0) sh.r32[3] = 0;
                row_sync<TX>();
                uint64_t own = 0;
                for (int i = 0; i < chunks_per_warp; ++i)
                    each(warp * chunks_per_warp + i, lo, [&](float x, int col) {
                        const uint64_t k = key(x, col);
                        if (k < base_key) return;
                        if (static_cast<uint32_t>(k >> 32) > hi) {
                            own += by_mass ? weight(x) : 1;
                        } else {
                            const uint32_t at = atomicAdd(&sh.r32[3], 1u);
                            if (at < kList) sh.list[at] = k;
                        }
                    });
                __syncwarp();
                above = row_sum(own);
                row_sync<TX>();
                const uint32_t n = sh.r32[3];
                if (above >= need) {  // (only where err is wrong)
                    *sure = err == 0;
                    return (static_cast<uint64_t>(hi) + 1) << 32;
                }
                left = need - above;
                if (n <= (TX == 32 ? 64 : kList)) {
                    // Ranks by counting, then the running sum in that order.
                    for (uint32_t i = threadIdx.x; i < n; i += TX) {
                        const uint64_t k = sh.list[i];
                        uint64_t w = 0;
                        for (uint32_t j = 0; j < n; ++j) {
                            const uint64_t o = sh.list[j];
                            if (o >= k) w += by_mass ? weight(order_value(static_cast<uint32_t>(o >> 32))) : 1;
                        }
                        sh.weights[i] = w;  // of the prefix that ends here
                    }
                    if (threadIdx.x == 0) sh.r64[2] = 0, sh.r32[0] = 1;
                    row_sync<TX>();
                    for (uint32_t i = threadIdx.x; i < n; i += TX) {
                        const uint64_t k = sh.list[i], w = sh.weights[i];
                        const uint64_t one = by_mass ? weight(order_value(static_cast<uint32_t>(k >> 32))) : 1;
                        if (w >= left && w - one < left) {
                            sh.r64[2] = k;
                            const uint64_t over = above + w - need, under = need - (above + w - one);
                            if (err && (over <= err || under <= err)) sh.r32[0] = 0;
                        }
                    }
                    row_sync<TX>();
                    const uint64_t k = sh.r64[2];
                    const bool ok = sh.r32[0] != 0;
                    row_sync<TX>();
                    if (k == 0) {
                        *sure = err == 0;
                        return base_key;
                    }
                    *sure = ok;
                    return k;
                }
                if (lo == hi) {  // equal values: a count of columns
                    if (err) {
                        *sure = false;
                        return base_key;
                    }
                    const float x = order_value(lo);
                    const uint64_t one = by_mass ? weight(x) : 1;
                    uint64_t count = one ? (left + one - 1) / one : 1;
                    const uint32_t o = lo;
                    const auto same = [&](float v, int col) -> uint64_t { return order_bits(v) == o && key(v, col) >= base_key; };
                    const uint64_t all = sum_chunks(o, same);
                    if (count > all) count = all;
                    int col = 0;
                    float value;
                    uint64_t b, w;
                    locate(count - 1, same, &col, &value, &b, &w);
                    return (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
                }
                if (err && round >= 3) {
                    *sure = false;
                    return base_key;
                }
            }
            // Narrow the range: to the bins in which the sum can reach what is left.
            const int shift = bin_shift(lo, hi);
            const int hs = by_mass ? max(0, 33 - __clzll(static_cast<long long>(range_most))) : 0;  // in 31 bits
            clear_bins();
            for (int i = 0; i < chunks_per_warp; ++i)
                each(warp * chunks_per_warp + i, lo, [&](float x, int col) {
                    const uint64_t k = key(x, col);
                    const uint32_t o = static_cast<uint32_t>(k >> 32);
                    if (k < base_key || o > hi) return;
                    const int b = (hi - o) >> shift;
                    atomicAdd(&sh.count[b], 1u);
                    if (by_mass) atomicAdd(&sh.mass[b], static_cast<uint32_t>(weight(x) >> hs));
                });
            int b0, b1;
            uint64_t before0 = 0, before1 = 0;
            if (by_mass) {
                const uint64_t low = left > err ? left - err : 1;
                const uint64_t need_low = max(static_cast<uint64_t>(1), low >> hs), need_high = ((left + err) >> hs) + 1;
                b0 = find_bin(sh.mass, true, need_low, &before0);
                b1 = find_bin(sh.mass, false, need_high, &before1);
                if (b0 == kBins) {
                    *sure = err == 0;
                    return base_key;
                }
                if (b1 == kBins) b1 = kBins - 1;
            } else {
                b0 = b1 = find_bin(sh.count, false, left, &before0);
                if (b0 == kBins) return base_key;
            }
            // An upper bound on the mass of the new range sets the next histogram's units.
            if (by_mass) {
                uint64_t mass = 0;
                for (int b = b0; b <= b1; ++b) mass += static_cast<uint64_t>(sh.mass[b]) + sh.count[b];
                range_most = mass << hs;
                row_sync<TX>();
            }
            const uint32_t old_hi = hi;
            hi = old_hi - (static_cast<uint32_t>(b0) << shift);
            const uint64_t reach = (static_cast<uint64_t>(b1) + 1) << shift;
            const uint32_t new_lo = reach > old_hi - lo ? lo : old_hi - static_cast<uint32_t>(reach) + 1;
            if (new_lo == lo && hi == old_hi && err) {
                *sure = false;
                return base_key;
            }
            lo = max(new_lo, floor);
        }
        *sure = err == 0;
        return base_key;
    }
};

template <int DT, int TX> __global__ void __launch_bounds__(TX) sample_kernel(SampleArgs a) {
    using R = Sampler<DT, TX>;
    __shared__ SampleShared<TX> sh;
    extern __shared__ __align__(16) unsigned char dynamic[];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < 64; i += TX) sh.powers[i] = kPowers[i];
    const int64_t row = blockIdx.x;
    R r(sh);
    r.N = static_cast<int>(a.N);
    const char* x0 = static_cast<const char*>(a.x) + row * a.row_stride * R::EB;
    r.off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15);
    r.base = x0 - r.off;
    // (An empty row covers no vector, wherever its pointer is.)
    r.slots = a.N == 0 ? 0 : static_cast<int>((static_cast<int64_t>(r.off) + a.N * R::EB + 15) / 16);
    r.end = static_cast<int>(r.off + a.N * R::EB - (static_cast<int64_t>(r.slots) - 1) * 16);
    r.chunk = a.chunk;
    r.chunks_per_warp = a.chunks_per_warp;
    r.chunks = R::W * a.chunks_per_warp;
    r.per_warp = a.per_warp;
    r.sums = reinterpret_cast<uint64_t*>(dynamic);
    float2* fast = reinterpret_cast<float2*>(r.sums + r.chunks + 1);
    r.maxima = reinterpret_cast<float*>(fast + r.chunks);

    const float temperature = a.temperature ? a.temperature[row] : a.temperature_all;
    const int64_t top_k = a.top_k ? a.top_k[row] : a.top_k_all;
    const float top_p = a.top_p ? a.top_p[row] : a.top_p_all;
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    const float u = a.u[row];
    const bool greedy = temperature < kSampleGreedy;
    const bool use_k = top_k > 0 && top_k < a.N && !greedy, use_p = top_p < 1.0f && !greedy, use_min = min_p > 0.0f && !greedy;
    {   // log2 e / T: the quotient of its first 24 bits, and what the remainder and the next bits add
        const float t = greedy ? 1.0f : temperature;
        r.ch = __fdiv_rn(kLog2e, t);
        r.cl = __fdiv_rn(fmaf(-r.ch, t, kLog2e) + 1.92596299e-8f, t);
    }
    r.S = a.bits;
    row_sync<TX>();
    // A greedy row needs no sums, nor does one whose top_k cuts the rest off before any sum.
    const bool with_sums = !(greedy || use_k);
    r.m = r.row_max(r.first_pass(fast, with_sums));
    row_sync<TX>();
    // Chunks' sums relative to the maximum, in whole numbers.
    bool bad = !(temperature >= 0.0f && temperature <= kSampleHottest) || top_p != top_p || min_p != min_p || !(fabsf(r.m) < kInf);
    int nan = 0;
    for (int c = threadIdx.x; c < r.chunks; c += TX) {
        const float2 f = fast[c];
        nan |= f.x != f.x;
        if (with_sums) {
            const double v = f.x > 0.0f && !bad ? static_cast<double>(f.x) * r.factor(f.y) : 0.0;
            r.sums[c] = v < kInf ? __double2ull_rn(v * __hiloint2double((1023 + r.S) << 20, 0)) : 0;
        }
    }
    if constexpr (TX == 32) nan = __any_sync(0xffffffffu, nan);
    else nan = __syncthreads_or(nan);
    if (bad || nan) {
        if (threadIdx.x == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = __int_as_float(0x7fc00000);
        }
        return;
    }
    const uint32_t top = order_bits(r.m);
    if (greedy) {
        if (threadIdx.x == 0) sh.r32[0] = 0xffffffffu;
        row_sync<TX>();
        for (int i = 0; i < r.chunks_per_warp; ++i)
            r.each(r.warp * r.chunks_per_warp + i, top, [&](float, int col) { atomicMin(&sh.r32[0], static_cast<uint32_t>(col)); });
        row_sync<TX>();
        if (threadIdx.x == 0) {
            a.token[row] = sh.r32[0];
            if (a.logprob) a.logprob[row] = 0.0f;
        }
        return;
    }
    const auto all_weights = [&](float x, int) -> uint64_t { return r.weight(x); };
    uint64_t total = 0, err = 0;
    bool have_sums = false;  // exact ones of what is kept
    if (with_sums) {
        total = r.scan_chunks();
        err = (total >> 21) + (total >> 23) + 1;  // kFastError of it
    }
    uint64_t threshold = 0;
    if (use_k) {
        bool sure;
        threshold = r.select(false, static_cast<uint64_t>(top_k), 0, 0, 0, &sure);
    }
    if (use_p) {
        if (use_k) {
            const uint64_t t = threshold;
            total = r.sum_chunks(static_cast<uint32_t>(t >> 32), [&](float x, int col) -> uint64_t { return R::key(x, col) >= t ? r.weight(x) : 0; });
            err = 0;
        }
        for (;;) {
            bool whole;
            uint64_t need = part_of(total, top_p, &whole);
            if (!whole || need == 0) ++need;
            bool sure;
            const uint64_t t = r.select(true, need, total, err, threshold, &sure);
            if (sure) {
                threshold = t > threshold ? t : threshold;
                break;
            }
            total = r.sum_chunks(0, all_weights);
            err = 0;
        }
    }
    if (use_min) {
        // x - m >= T log(min_p) in 64 bits, as a comparison of x in 32.
        if (threadIdx.x == 0) {
            const double v = static_cast<double>(r.m) + static_cast<double>(temperature) * log(static_cast<double>(fminf(min_p, 1.0f)));
            sh.r32[0] = order_bits(__double2float_ru(v));
        }
        row_sync<TX>();
        const uint64_t t = static_cast<uint64_t>(sh.r32[0]) << 32;
        row_sync<TX>();
        threshold = t > threshold ? t : threshold;
    }
    const auto kept = [&](float x, int col) -> uint64_t { return R::key(x, col) >= threshold ? r.weight(x) : 0; };
    const bool cut = threshold != 0;
    for (;;) {
        if (cut || have_sums) {
            total = r.sum_chunks(static_cast<uint32_t>(threshold >> 32), kept);
            err = 0;
        }
        bool whole;
        uint64_t target = u >= 1.0f ? total - 1 : part_of(total, u, &whole);
        int col = 0;
        float x = 0.0f;
        uint64_t before = 0, with = 0;
        const bool found = r.locate(target, kept, &col, &x, &before, &with);
        if (err && (!found || target - before < err || with - target <= err)) {
            have_sums = true;  // too close to tell
            continue;
        }
        if (threadIdx.x == 0) {
            a.token[row] = found ? col : -1;
            if (a.logprob) {
                // The maximum is kept and weighs 1: log(1 + rest) keeps the digits of a small rest.
                const uint64_t rest = total - min(total, 1ull << r.S);
                a.logprob[row] = (x - r.m) / temperature - log1pf(static_cast<float>(rest) * __int_as_float((127 - r.S) << 23));
            }
        }
        return;
    }
}

template <int DT, int TX> cudaError_t launch_sample_rows(SampleArgs a, cudaStream_t s) {
    constexpr int W = TX / 32, EB = DType<DT>::bytes;
    // Vectors of a row, one more for rows off a boundary; whole batches, and as many chunks
    // as 32 KB of maxima hold.
    const int64_t slots = (a.N * EB + 15) / 16 + 1;
    int64_t per = (slots + W - 1) / W;
    per = (per + 31) / 32 * 32;
    int64_t chunk = 32 * kBatch;
    while ((per + chunk - 1) / chunk * W > 256) chunk *= 2;
    a.per_warp = static_cast<int>(per);
    a.chunk = static_cast<int>(chunk);
    a.chunks_per_warp = static_cast<int>((per + chunk - 1) / chunk);
    const int chunks = a.chunks_per_warp * W;
    const size_t smem = (chunks + 1) * sizeof(uint64_t) + chunks * (sizeof(float2) + 32 * sizeof(float));
    auto kernel = sample_kernel<DT, TX>;
    if (smem > 30 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl_smem(kernel, dim3(static_cast<unsigned>(a.B)), dim3(TX), smem, s, a);
}

template <int DT> cudaError_t launch_sample(SampleArgs a, int sms, cudaStream_t s) {
    const int64_t slots = (a.N * DType<DT>::bytes + 15) / 16 + 1;
    a.bits = 62;
    for (int64_t n = a.N; n > 1; n = (n + 1) / 2) --a.bits;
    if (a.bits > 44) a.bits = 44;
    if (slots <= 256) return launch_sample_rows<DT, 32>(a, s);
    if (slots <= 2048) return launch_sample_rows<DT, 128>(a, s);
    if (a.B >= 4 * sms || slots <= 8192) return launch_sample_rows<DT, 256>(a, s);
    return launch_sample_rows<DT, 1024>(a, s);
}

}  // namespace
}  // namespace lse
