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
// in 32 bits would give another token than the formula in one row of a few hundred.  Exact
// weights are therefore whole numbers of 2^-S (S about 44): 2^z with z the distance to the
// maximum in octaves, taken apart as 2^(k/64) 2^r with the remainder r formed without rounding
// the product and a cubic for 2^r - 1; off by at most about 2^-30 of itself.  Sums of whole
// numbers do not depend on their order.  That takes about 40 instructions, four times what the
// memory's rate leaves for a bf16 element, so passes over a row use fast weights, of ex2 with the
// rounding error of its argument carried along.  Such a sum is that of w (1 + e), |e| <= E:
//
//     1.46e-7      of ex2.approx (-1.44e-7 to 1.46e-7 over every f32 in [-110, 110])
//     n 2^-24      of the additions that an element passes through: log2 of the 32 elements (of f32,
//                  16) that a lane adds by halves at a time, and the chunk's
//
// in the worst case, which a row of one or two heavy elements comes near.  Weights are relative to 0
// where the maximum is -64 to 100 octaves (x log2 e / T) from it, else to a maximum.  Distances from that are
// rounded where elements are of 16 bits (f32 ones carry what that loses along): by 2^-24 of
// (m - x) / T, whose mean over the weights is at most log(N / sum of w), the entropy of N equal ones
// less what w has (and log 2 more in first_pass(), whose shifts lie up to an octave below the
// elements).
// What is compared is a part of a sum with u (or top_p) times the whole.  The difference is off by
// 1 - u times the sum of w e over the part, less u times that over the rest; a share L of the part
// that has been summed exactly counts with u, in the whole only.  So it is off by at most
//
//     E (2 u (1 - u) + max(0, 2 u - 1) L) + 2^-24 log(2 N / sum) max(u, 1 - u)
//
// of the whole, the second term only with rounded distances (Doubt).  Where a comparison is closer, the
// row is done again with exact weights.
//
// Threshold.  Every lane's maximum in every chunk is kept in shared memory.  They bound the
// threshold from below (the k-th largest of them is at most the k-th largest element; the same
// for sums), and later passes read only the vectors of lanes and chunks that reach the bound:
// few for peaked rows.  Where what they find fits a list in shared memory, the list is put in
// order and cut, put in column order and drawn from, and the row is not read again.  Otherwise
// (flat rows) a histogram of counts over the values brackets the threshold, since within a bin all
// weights are within a few percent of each other; the bracket's elements go to the list, what
// lies above is summed, and one more pass sums what is kept by chunks.  A range that a histogram hardly
// narrows (a run of equal values so heavy that the widths of bins hide where the sum passes) is
// bisected, a pass for each half.
//
// Measured (us): 2048 x 128256 bf16, nothing cut off 237 (2.2 TB/s; the pass alone, without weights,
// 126, bound by loads at 42 % of the warps; without rows too close to tell 195), top_k 50 and top_p
// 0.95 280, top_p 0.9 of rows from peaked to flat 2680 (instructions: three to four passes of 10 to 15
// per element); one such row 16, 28 and 55; 65536 x 261 f32 top_p 0.9 150 (68 % of the issue slots).
// Putting the lanes' sums together by shuffles in f32 instead takes 12 us less for the 2048 rows, and more
// of them are too close to tell.  Counters of several
// threads are the slowest part: 26 ns for each addition with a result to one of them, so places in a
// list are handed out per warp; histograms by the bits of f32, which have two bins for all
// values within a factor of two, took 11 ms where bins linear in the value take 3.
//
// Rows of up to 256 vectors take a warp each and stay in registers; sums are f32 there, and a
// row in which one of them lies too close to a border to tell is done by the warp as above.
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

constexpr int kBatch = 4;    // vectors of a lane in flight
constexpr int kChunk = 128;  // vectors of a chunk, at least
// Histogram bins and list entries of a row's threads.
template <int TX> __host__ __device__ constexpr int bins_log2() { return TX == 32 ? 7 : 10; }
template <int TX> __host__ __device__ constexpr int list_size() { return TX == 32 ? 64 : 2048; }
constexpr float kInf = __builtin_inff();
// Octaves above and below 0 within which fast weights are relative to it: sums stay below 2^127, and
// 60 octaves below a maximum are still f32 numbers.
constexpr float kNearAbove = 100.0f, kNearBelow = -64.0f;

// What a comparison of a part of a fast sum with a share u of the whole may be off by (see above).
template <int DT> __host__ __device__ constexpr float fast_error() { return 1.46e-7f + (DT == kF32 ? 5 : 6) * 0x1p-24f + 4e-9f; }
struct Doubt {
    uint64_t any;    // of a sum alone, and at any share; 0: sums are exact
    uint64_t fixed;
    float exact;     // times the part's elements that were summed exactly
    __device__ __forceinline__ Doubt() : any(0), fixed(0), exact(0.0f) {}
    // each: fast_error().  (Chunks' sums are rounded to whole numbers, a half each.)
    __device__ __forceinline__ Doubt(uint64_t total, float u, float each, bool whole_distances, int N, int S) {
        u = fminf(fmaxf(u, 0.0f), 1.0f);
        const float all = static_cast<float>(total);
        const float far = whole_distances ? 0.0f : 0x1p-24f * fmaxf(0.0f, __logf(2.0f * static_cast<float>(N) / (all * __int_as_float((127 - S) << 23))));
        any = static_cast<uint64_t>(all * (each + far)) + 300;
        fixed = static_cast<uint64_t>(all * (each * 2.0f * u * (1.0f - u) + far * fmaxf(u, 1.0f - u) + 2e-9f)) + 300;
        exact = each * fmaxf(0.0f, 2.0f * u - 1.0f);
    }
    __device__ __forceinline__ uint64_t at(uint64_t summed) const { return any ? fixed + static_cast<uint64_t>(exact * static_cast<float>(summed)) : 0; }
    // Whether a target between two sums, the second with `summed` of it exact, is next to neither.
    __device__ __forceinline__ bool sure(uint64_t before, uint64_t target, uint64_t with, uint64_t summed) const {
        const uint64_t e = at(summed);
        return target - before > e && with - target > e;
    }
};

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

// 2^(j / 32) as the sum of two floats.
__constant__ float kHigh[32] = {
    0x1.0000000000000p+0f, 0x1.059b0e0000000p+0f, 0x1.0b55860000000p+0f, 0x1.11301e0000000p+0f,
    0x1.172b840000000p+0f, 0x1.1d48740000000p+0f, 0x1.2387a60000000p+0f, 0x1.29e9e00000000p+0f,
    0x1.306fe00000000p+0f, 0x1.371a740000000p+0f, 0x1.3dea640000000p+0f, 0x1.44e0860000000p+0f,
    0x1.4bfdae0000000p+0f, 0x1.5342b60000000p+0f, 0x1.5ab07e0000000p+0f, 0x1.6247ec0000000p+0f,
    0x1.6a09e60000000p+0f, 0x1.71f75e0000000p+0f, 0x1.7a11480000000p+0f, 0x1.82589a0000000p+0f,
    0x1.8ace540000000p+0f, 0x1.93737c0000000p+0f, 0x1.9c49180000000p+0f, 0x1.a5503c0000000p+0f,
    0x1.ae89fa0000000p+0f, 0x1.b7f7700000000p+0f, 0x1.c199be0000000p+0f, 0x1.cb720e0000000p+0f,
    0x1.d5818e0000000p+0f, 0x1.dfc9740000000p+0f, 0x1.ea4afa0000000p+0f, 0x1.f507660000000p+0f,
};
__constant__ float kLow[32] = {
    0x0.0p+0f, -0x1.9d4f520000000p-25f, 0x1.9f31220000000p-25f, -0x1.fdb4960000000p-25f,
    -0x1.c157420000000p-27f, -0x1.d2e8ca0000000p-25f, 0x1.ceac480000000p-25f, -0x1.5c04240000000p-25f,
    0x1.4636e20000000p-25f, -0x1.18aac60000000p-25f, 0x1.8246840000000p-25f, 0x1.8624b40000000p-30f,
    -0x1.593abc0000000p-25f, -0x1.2c56100000000p-25f, -0x1.5bd5ec0000000p-27f, -0x1.f8b5500000000p-25f,
    0x1.9fcef40000000p-26f, 0x1.1d8bee0000000p-25f, -0x1.829fd00000000p-25f, -0x1.accc7c0000000p-26f,
    0x1.15506e0000000p-27f, -0x1.e647440000000p-25f, 0x1.51f8480000000p-27f, -0x1.b83b540000000p-25f,
    -0x1.a94b140000000p-26f, -0x1.a094380000000p-25f, -0x1.3d56b20000000p-27f, -0x1.8837cc0000000p-27f,
    -0x1.822dbc0000000p-27f, -0x1.908c940000000p-25f, 0x1.52486c0000000p-27f, -0x1.246eb00000000p-26f,
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

// What a row's threads share.
template <int TX> struct SampleShared {
    static constexpr int W = TX / 32, kBins = 1 << bins_log2<TX>(), kList = list_size<TX>();
    uint32_t bins[kBins];
    uint64_t list[kList];      // keys
    static constexpr int kPart = TX == 32 ? 64 : 1024;  // of the list, put in order
    union {
        uint64_t work[kBins + kPart];                     // sums of weights by bins, and a bin's keys
        unsigned short entries[4 * (kBins + kPart)];      // lanes and chunks that reach a bound
    };
    uint64_t warp64[W + 1];
    float warpf[W];
    uint64_t r64[4];
    uint32_t r32[4];
};

template <int DT, int TX> struct Sampler {
    static constexpr int W = TX / 32, EB = DType<DT>::bytes, E = 16 / EB;
    static constexpr int kBins = SampleShared<TX>::kBins, kList = SampleShared<TX>::kList, kPart = SampleShared<TX>::kPart;
    SampleShared<TX>& sh;
    const uint32_t* powers;  // kPowers in shared memory
    // the row
    const char* base;  // the 16-byte boundary at or before its first element
    int off, end;      // its first and last bytes (end: in the last vector, from its start)
    int slots;         // vectors that cover it
    int N;
    int chunk, chunks_per_warp, chunks;  // vectors of a chunk; chunks of a warp (one after the other), in all
    // per chunk
    float* maxima;     // [chunks, 32]
    uint64_t* sums;    // [chunks + 1]: sums, then sums before
    uint64_t* added;   // [chunks], in the place of the first pass's sums
    // weights
    float m, ch, cl;   // maximum; log2 e / T in two floats
    float far;         // the distance from which weights are 0
    int S;             // fractional bits of a weight
    bool lost = false; // a threshold or a column was not found: the row is marked, not drawn without it
    int lane, warp, tid;  // in the row's group of threads

    __device__ __forceinline__ Sampler(SampleShared<TX>& s)
        : sh(s), lane(threadIdx.x & 31), warp(TX == 32 ? 0 : threadIdx.x >> 5), tid(TX == 32 ? lane : threadIdx.x) {}

    // -----------------------------------------------------------------------
    // Elements
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void load(int slot, uint32_t (&w)[4]) const {
        const uint4 v = ldg_stream16(base + static_cast<int64_t>(slot) * 16);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    // Elements outside the row to -inf.  Apart from load(): a use of the words next to each load
    // would keep the next load waiting for it.
    __device__ __forceinline__ void mask(int slot, uint32_t (&w)[4]) const {
        if ((slot == 0 && off != 0) || slot == slots - 1)
            mask_words<DT>(w, 0, slot == 0 ? off : 0, slot == slots - 1 ? end : 16);
    }
    // Whether any of the vectors [a, b) holds elements outside the row.
    __device__ __forceinline__ bool has_edge(int a, int b) const { return (a == 0 && off != 0) || b >= slots; }
    __device__ __forceinline__ int column(int slot, int e) const { return slot * E + e - off / EB; }
    __device__ __forceinline__ int chunk_begin(int c) const { return c * chunk; }
    __device__ __forceinline__ int chunk_end(int c) const { return min(c * chunk + chunk, slots); }

    // 2^((x - m) log2 e / T) for x <= m and distances d ch of less than 2^15 octaves, as
    // p 2^(e - 30).
    __device__ __forceinline__ void power(float x, float d, uint32_t* p, int* e) const {
        const float a = d + m, b = d - a, dl = (x - a) + (-m - b);  // x - m = d + dl
        const float kf = fmaf(d, ch * 64.0f, 12582912.0f);
        const int k = __float_as_int(kf) - 0x4b400000;
        float r = fmaf(d, ch, (kf - 12582912.0f) * -0.015625f);
        r = fmaf(d, cl, r);
        r = fmaf(dl, ch, r);
        const float q = r * fmaf(r, fmaf(r, 0.0555041087f, 0.240226507f), 0.693147181f);
        const uint32_t t = powers[k & 63];
        *p = t + __float2int_rn(static_cast<float>(t) * q);
        *e = k >> 6;
    }
    // The weight of an element, a whole number of 2^-S (0 from S + 2 octaves on).
    __device__ __forceinline__ uint64_t weight(float x) const {
        const float d = x - m;
        uint32_t p;
        int e;
        power(d > far ? x : m + far, fmaxf(d, far), &p, &e);
        const int s = S - 30 + e;
        return s >= 0 ? static_cast<uint64_t>(p) << s : (static_cast<uint64_t>(p) + (1ull << (-s - 1))) >> -s;
    }
    __device__ __forceinline__ double factor(float x) const {
        const float d = x - m;
        if (!(d * ch >= -900.0f)) return 0.0;
        uint32_t p;
        int e;
        power(x, d, &p, &e);
        return static_cast<double>(p) * __hiloint2double((1023 - 30 + e) << 20, 0);
    }

    // f(words, vector, mask of its elements) for the elements of at least `low`, by the lanes'
    // maxima: the lanes and chunks that reach it are listed and their vectors handed out to all
    // threads, a warp's lanes in step.  false: they are more than the list holds (f has not been
    // called).
    template <class F> __device__ __forceinline__ bool sparse(float low, F&& f) {
        constexpr uint32_t kEntries = 4 * (kBins + kPart);
        row_sync<TX>();
        if (tid == 0) sh.r32[2] = 0;
        row_sync<TX>();
        for (int i0 = 0; i0 < chunks * 32; i0 += 16 * TX) {
            uint32_t mask = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = i0 + j * TX + tid;
                if (i < chunks * 32 && !(maxima[i] < low)) mask |= 1u << j;
            }
            uint32_t at = places(&sh.r32[2], __popc(mask));
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (mask >> j & 1) {
                    if (at < kEntries) sh.entries[at] = static_cast<unsigned short>(i0 + j * TX + tid);
                    ++at;
                }
        }
        row_sync<TX>();
        const uint32_t n = sh.r32[2];
        if (n > kEntries) return false;
        const uint32_t vectors = chunk / 32;  // a power of two
        const int shift = __ffs(vectors) - 1;
        for (uint32_t t0 = 0; t0 < n * vectors; t0 += TX) {  // (all lanes in step)
            const uint32_t t = t0 + tid;
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = neg_inf_word<DT>();
            int s = -1;
            if (t < n * vectors) {
                const int i = sh.entries[t >> shift], c = i >> 5;
                s = chunk_begin(c) + (i & 31) + 32 * static_cast<int>(t & (vectors - 1));
                if (s < chunk_end(c)) load(s, w), mask(s, w);
                else s = -1;
            }
            uint32_t mask = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (s >= 0 && !(word_elem<DT>(w, e) < low) && static_cast<unsigned>(column(s, e)) < static_cast<unsigned>(N)) mask |= 1u << e;
            f(w, s, mask);
        }
        row_sync<TX>();
        return true;
    }
    // The first of `n` places of this lane behind a shared counter: one addition per warp (one
    // per element made every thread wait 26 ns for each).
    __device__ __forceinline__ uint32_t places(uint32_t* counter, uint32_t n) const {
        uint32_t s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t b = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += b;
        }
        uint32_t first = 0;
        if (lane == 31 && s != 0) first = atomicAdd(counter, s);
        return __shfl_sync(0xffffffffu, first, 31) + s - n;
    }
    // f(words, first vector) for every batch of the row's chunks, the words of lanes whose
    // maximum is below `low` as -inf; done(c) after a chunk.
    template <class F, class G> __device__ __forceinline__ void dense(float low, F&& f, G&& done) {
        for (int i = 0; i < chunks_per_warp; ++i) {
            const int c = warp * chunks_per_warp + i, stop = chunk_end(c);
            const bool some = !(maxima[c * 32 + lane] < low);
            if (__any_sync(0xffffffffu, some)) {
                for (int s0 = chunk_begin(c) + lane; s0 - lane < stop; s0 += 32 * kBatch) {
                    uint32_t w[kBatch][4];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) w[j][q] = neg_inf_word<DT>();
                        if (some && s0 + 32 * j < stop) load(s0 + 32 * j, w[j]);
                    }
                    if (has_edge(s0 - lane, s0 - lane + 32 * kBatch)) {
#pragma unroll
                        for (int j = 0; j < kBatch; ++j)
                            if (some && s0 + 32 * j < stop) mask(s0 + 32 * j, w[j]);
                    }
                    f(w, s0);
                }
            }
            __syncwarp();
            done(c);
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
    // The counts over the chunks of the elements that keep(x, column) names, all of them at
    // least `low`.
    template <class F> __device__ __noinline__ uint64_t count_chunks(float low, F keep) {
        row_sync<TX>();
        uint64_t s = 0;
        dense(low, [&](const uint32_t (&w)[kBatch][4], int s0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) s += keep(word_elem<DT>(w[j], e), column(s0 + 32 * j, e)) ? 1 : 0;
        }, [&](int c) {
            s = warp_sum(s);
            if (lane == 0) sums[c] = s;
            s = 0;
        });
        return scan_chunks();
    }
    // The exact weights of a pair, added to sums of pairs (hi + lo): as power(), in f32 pairs, with
    // the table's entries in the lanes of the warp (all of which take part): 2^z = (high + low)
    // 2^r 2^e.  -inf adds nothing that counts (2^-60).
    __device__ __forceinline__ void add_exact_pair(uint64_t& hi, uint64_t& lo, uint64_t x, float high, float low, float dmin) const {
        const uint64_t m2 = f2_pack(m, m), ch2 = f2_pack(ch, ch), cl2 = f2_pack(cl, cl);
        uint64_t d = f2_sub(x, m2);
        const uint64_t a = f2_add(d, m2), b = f2_sub(d, a);
        uint64_t dl = f2_add(f2_sub(x, a), f2_sub(f2_pack(-m, -m), b));  // x - m = d + dl
        float d0, d1, l0, l1;
        f2_unpack(d, d0, d1);
        f2_unpack(dl, l0, l1);
        dl = f2_pack(d0 > dmin ? l0 : 0.0f, d1 > dmin ? l1 : 0.0f);
        d = f2_pack(fmaxf(d0, dmin), fmaxf(d1, dmin));
        const float magic = 12582912.0f;
        const uint64_t kf = f2_fma(d, f2_pack(ch * 32.0f, ch * 32.0f), f2_pack(magic, magic));
        const uint64_t nf = f2_sub(kf, f2_pack(magic, magic));
        uint64_t r = f2_fma(d, ch2, f2_mul(nf, f2_pack(-0.03125f, -0.03125f)));
        r = f2_fma(d, cl2, r);
        r = f2_fma(dl, ch2, r);
        uint64_t q = f2_fma(r, f2_pack(0.00961812911f, 0.00961812911f), f2_pack(0.0555041087f, 0.0555041087f));
        q = f2_fma(r, q, f2_pack(0.240226507f, 0.240226507f));
        q = f2_fma(r, q, f2_pack(0.693147181f, 0.693147181f));
        q = f2_mul(r, q);
        float k0, k1;
        f2_unpack(kf, k0, k1);
        const int i0 = __float_as_int(k0) - 0x4b400000, i1 = __float_as_int(k1) - 0x4b400000;
        const uint64_t t = f2_pack(__shfl_sync(0xffffffffu, high, i0 & 31), __shfl_sync(0xffffffffu, high, i1 & 31));
        const uint64_t u = f2_pack(__shfl_sync(0xffffffffu, low, i0 & 31), __shfl_sync(0xffffffffu, low, i1 & 31));
        const uint64_t e = f2_pack(__int_as_float((127 + (i0 >> 5)) << 23), __int_as_float((127 + (i1 >> 5)) << 23));
        const uint64_t v = f2_mul(t, e);
        const uint64_t n = f2_add(hi, v), aa = f2_sub(n, v), bb = f2_sub(n, aa);  // hi + v = n + what it loses
        lo = f2_add(lo, f2_add(f2_sub(hi, aa), f2_sub(v, bb)));
        lo = f2_add(lo, f2_mul(f2_fma(t, q, u), e));
        hi = n;
    }
    // The exact sums over the chunks of the weights of the elements that keep(x, column) names,
    // all of them at least `low`.
    template <class F> __device__ __noinline__ uint64_t exact_chunks(float low, F keep) {
        row_sync<TX>();
        const float high = kHigh[lane], rest = kLow[lane], dmin = -60.0f / ch;
        uint64_t hi = 0, lo = 0;
        dense(low, [&](const uint32_t (&w)[kBatch][4], int s0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    float x0, x1;
                    f2_unpack(pair_of(w[j], e), x0, x1);
                    x0 = keep(x0, column(s0 + 32 * j, 2 * e)) ? x0 : -kInf;
                    x1 = keep(x1, column(s0 + 32 * j, 2 * e + 1)) ? x1 : -kInf;
                    add_exact_pair(hi, lo, f2_pack(x0, x1), high, rest, dmin);
                }
        }, [&](int c) {
            const uint64_t s = exact_sum(hi, lo);
            if (lane == 0) sums[c] = s;
            hi = lo = 0;
        });
        return scan_chunks();
    }
    // The warp's sum of pairs of sums, as a weight.
    __device__ __forceinline__ uint64_t exact_sum(uint64_t hi, uint64_t lo) const {
        float h0, h1, l0, l1;
        f2_unpack(hi, h0, h1);
        f2_unpack(lo, l0, l1);
        const double v = (static_cast<double>(h0) + static_cast<double>(h1)) + (static_cast<double>(l0) + static_cast<double>(l1));
        return warp_sum(__double2ull_rn(v * __hiloint2double((1023 + S) << 20, 0)));
    }
    // The first column at which the running sum of f passes `target`; sums are scanned.
    // Sets the sums before it and with it, and what of the latter is the chunk's own (which is summed
    // here, by f); false if there is none in the chunk that the chunks' sums name (they may be
    // approximate).
    template <class F>
    __device__ __forceinline__ bool locate(uint64_t target, bool clamp, F&& f, int* col, float* value, uint64_t* before, uint64_t* with, uint64_t* inside) {
        int c, s0, s1;
        uint64_t own, first, rest;
        bool back = false;
        // (One round, unless `clamp` meets chunks of nothing but elements below 2^-45 of the largest:
        // each alone weighs nothing, while their exact sum may.  The next chunk that weighs takes
        // their place, or the one before if there is none behind.)
        for (int round = 0;; ++round) {
            if (tid == 0) sh.r32[1] = 0;
            row_sync<TX>();
            for (int i = tid; i < chunks; i += TX)
                if (sums[i] <= target && target < sums[i + 1]) sh.r32[0] = i, sh.r32[1] = 1;
            row_sync<TX>();
            const bool any = sh.r32[1] != 0;
            c = sh.r32[0];
            row_sync<TX>();
            if (tid == 0) sh.r32[1] = 0;
            if (!any) {
                row_sync<TX>();
                return false;
            }
            const int b = chunk_begin(c), n = chunk_end(c) - b;
            const int per = (n + TX - 1) / TX;
            s0 = b + tid * per;
            s1 = min(s0 + per, b + n);
            own = 0;
            for (int s = s0; s < s1; ++s) {
                uint32_t w[4];
                load(s, w);
                mask(s, w);
#pragma unroll
                for (int e = 0; e < E; ++e) own += f(word_elem<DT>(w, e), column(s, e));
            }
            first = row_before(own);
            // (Chunks' sums are good to about 2^-32; what is left of the target beyond the chunk's
            // own sum by that is its last element's.)
            rest = target - sums[c];
            if (!clamp) break;
            const uint64_t all = row_sum(own);
            if (all > 0) {
                if (back || rest >= all) rest = all - 1;
                break;
            }
            if (!back && sums[c + 1] >= sums[chunks]) back = true;
            if (round > 2 * chunks || (back && sums[c] == 0)) break;
            target = back ? sums[c] - 1 : sums[c + 1];
        }
        row_sync<TX>();
        if (first <= rest && rest < first + own) {
            uint64_t run = first;
            bool found = false;
            for (int s = s0; s < s1 && !found; ++s) {
                uint32_t w[4];
                load(s, w);
                mask(s, w);
                for (int e = 0; e < E && !found; ++e) {
                    const float x = word_elem<DT>(w, e);
                    const uint64_t v = f(x, column(s, e));
                    if (run + v > rest) {
                        sh.r32[0] = column(s, e);
                        sh.r32[1] = 1;
                        sh.r32[2] = __float_as_uint(x);
                        sh.r64[0] = sums[c] + run;
                        sh.r64[1] = sums[c] + run + v;
                        sh.r64[2] = run + v;
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
        *inside = sh.r64[2];
        row_sync<TX>();
        return ok;
    }

    // -----------------------------------------------------------------------
    // Pass over the row: maxima, and sums of fast weights relative to a shift of the chunk's
    // (chunks are the same whatever the number of threads, and so are a row's sums in any batch)
    // -----------------------------------------------------------------------
    // The fast weights of a pair, w (1 - e log 2): w is 2^t, and e what t has too much of.
    __device__ __forceinline__ uint64_t pair_weights(uint64_t x, float mu, float dmin, uint64_t* lost) const {
        const uint64_t mu2 = f2_pack(mu, mu), ch2 = f2_pack(ch, ch), nch2 = f2_pack(-ch, -ch), ncl2 = f2_pack(-cl, -cl);
        uint64_t d = f2_sub(x, mu2);
        uint64_t dl = 0;
        float d0, d1;
        f2_unpack(d, d0, d1);
        if constexpr (DT == kF32) {  // what the difference of two f32 loses
            const uint64_t a = f2_add(d, mu2), b = f2_sub(d, a);
            dl = f2_add(f2_sub(x, a), f2_sub(f2_pack(-mu, -mu), b));
            float l0, l1;
            f2_unpack(dl, l0, l1);
            dl = f2_pack(d0 > dmin ? l0 : 0.0f, d1 > dmin ? l1 : 0.0f);
        }
        // A weight of 2^-200 is 0; an infinite distance would give inf - inf below.  (A NaN stays.)
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(d0) : "f"(dmin));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(d1) : "f"(dmin));
        d = f2_pack(d0, d1);
        const uint64_t t = f2_mul(d, ch2);
        uint64_t e = f2_fma(d, nch2, t);  // minus what the product lost
        e = f2_fma(d, ncl2, e);
        if constexpr (DT == kF32) e = f2_fma(dl, nch2, e);
        *lost = e;
        return f2_ex2(t);
    }
    // Pairs A .. A + L - 1 of a batch, the words of which f(i) gives, by halves (log L roundings); w e
    // is added to `over`.
    template <int A, int L, class F>
    __device__ __forceinline__ uint64_t sum_pairs(const F& f, uint64_t& over, float mu, float dmin) const {
        if constexpr (L == 1) {
            uint64_t e;
            const uint64_t w = pair_weights(f(A), mu, dmin, &e);
            over = f2_fma(w, e, over);
            return w;
        } else {
            const uint64_t s = sum_pairs<A, L / 2>(f, over, mu, dmin);
            return f2_add(s, sum_pairs<A + L / 2, L / 2>(f, over, mu, dmin));
        }
    }
    template <class F> __device__ __forceinline__ void add_pairs(float& hi, float& lo, const F& f, float mu, float dmin) const {
        uint64_t over = 0;
        const uint64_t s = sum_pairs<0, kBatch * E / 2>(f, over, mu, dmin);
        add_sums(hi, lo, s, over);
    }
    __device__ __forceinline__ static uint64_t pair_of(const uint32_t (&w)[4], int i) {  // i < E / 2
        if constexpr (DT == kF32) return f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return f2_pack(word_lo<DT>(w[i]), word_hi<DT>(w[i]));
    }
    // A batch's sums to the lane's, hi + lo.
    __device__ __forceinline__ static void add_sums(float& hi, float& lo, uint64_t acc, uint64_t over) {
        float a, b, c, d;
        f2_unpack(acc, a, b);
        f2_unpack(over, c, d);
        add_exact(hi, lo, a + b);
        lo = fmaf(c + d, -kLn2, lo);
    }
    // The lanes' sums hi + lo (|lo| a 2^-17th of hi at most) put together as whole numbers, of 2^-38
    // of the largest, and rounded once; NaN if one is no number.
    __device__ __forceinline__ static float over_lanes(float hi, float lo) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(hi));
        if (top == 0) return 0.0f;
        if (top >= 0x7f800000u) return kInf - kInf;
        constexpr float magic = 12582912.0f;  // 1.5 2^23: added to it, a number is rounded to a whole one
        const uint32_t e = max(top >> 23, 23u);
        const float up = __uint_as_float((275u - e) << 23), down = __uint_as_float((e - 21u) << 23);  // the largest to 2^21 .. 2^22
        const float t = fmaf(hi, up, magic), r = fmaf(lo, up, fmaf(hi, up, -(t - magic)));
        const int a = __reduce_add_sync(0xffffffffu, __float_as_int(t) - 0x4b400000);
        const int b = __reduce_add_sync(0xffffffffu, __float_as_int(fmaf(r, 65536.0f, magic)) - 0x4b400000);
        return __ll2float_rn((static_cast<long long>(a) << 16) + b) * 0x1p-16f * down;
    }
    // What fast weights are relative to, for elements of at most v: 0, which no distance is rounded
    // from, where 2^(v log2 e / T) and what counts below it are f32 numbers.
    __device__ __forceinline__ float shift_of(float v) const { return v * ch <= kNearAbove && v * ch >= kNearBelow ? 0.0f : v; }
    // Whether that makes no difference or holds for all elements that count (one of a chunk that lies
    // below it weighs less than 2^-48 of the row).
    __device__ __forceinline__ bool whole_distances() const { return DT == kF32 || (m * ch <= kNearAbove && m * ch >= kNearBelow + 48.0f); }
    // From sums relative to shift_of(m) to weights.
    __device__ __forceinline__ double in_weights() const {
        return factor(shift_of(m)) * __hiloint2double((1023 + S) << 20, 0);
    }
    // hi + lo + v without loss.
    __device__ __forceinline__ static void add_exact(float& hi, float& lo, float v) {
        const float n = hi + v, a = n - v, b = n - a;
        lo += (hi - a) + (v - b);
        hi = n;
    }

    // Leaves (sum, shift) of every chunk in `fast`; returns the lane's maximum.
    __device__ __forceinline__ float first_pass(float2* fast, bool with_sums) {
        float top = -kInf;
        const float dmin = -200.0f / ch;
        const int batches = chunk / (32 * kBatch);  // of a chunk
        const int first = chunk_begin(warp * chunks_per_warp);
        const int stop = min(first + chunks_per_warp * chunk, slots);
        float cm = -kInf, hi = 0.0f, lo = 0.0f, mu = 0.0f, lim = -kInf;
        int c = warp * chunks_per_warp, left = batches;
        const int all = chunks_per_warp * batches;
        for (int i = 0; i < all; i += 2) {
            uint32_t v[2][kBatch][4];  // two batches in flight
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int s = first + (i + h) * (32 * kBatch) + lane + 32 * j;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[h][j][q] = neg_inf_word<DT>();
                    if (s < stop) load(s, v[h][j]);
                }
            const int at = first + i * (32 * kBatch);
            if (has_edge(at, at + 64 * kBatch)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int s = at + h * (32 * kBatch) + lane + 32 * j;
                        if (s < stop) mask(s, v[h][j]);
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (i + h >= all) continue;
                const auto& w = v[h];
                float bm = words_max<DT, 4>(w[0]);
#pragma unroll
                for (int j = 1; j < kBatch; ++j) bm = fmaxf(bm, words_max<DT, 4>(w[j]));
                cm = fmaxf(cm, bm);
                if (!with_sums) {  // maxima ignore NaN: leave one in the sum
                    bool nan = false;
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
#pragma unroll
                        for (int e = 0; e < E; ++e) nan |= word_elem<DT>(w[j], e) != word_elem<DT>(w[j], e);
                    if (nan) hi = kInf - kInf;
                } else {
                    if (__any_sync(0xffffffffu, bm > lim)) {  // the shift goes up
                        float to = 0.0f, wm = 0.0f;
                        if (!__all_sync(0xffffffffu, bm * ch <= kNearAbove) || !__any_sync(0xffffffffu, bm * ch >= kNearBelow)) {
                            wm = bm;
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
                            to = wm;  // (not near 0)
                        }
                        if (wm < kInf) {
                            if (hi != 0.0f) {  // sums relative to the old one (rare: a step of an octave within a chunk)
                                Sampler t = *this;
                                t.m = to;
                                const double sum = (static_cast<double>(hi) + static_cast<double>(lo)) * t.factor(mu);
                                hi = static_cast<float>(sum);
                                lo = static_cast<float>(sum - static_cast<double>(hi));
                            }
                            mu = to;
                            lim = to == 0.0f ? kNearAbove / ch : to + 1.0f / ch;
                            if (!(lim > to)) lim = to;
                        }
                    }
                    add_pairs(hi, lo, [&](int i) { return pair_of(w[i / (E / 2)], i % (E / 2)); }, mu, dmin);
                }
                if (--left == 0) {  // the chunk is complete
                    const float s = over_lanes(hi, lo);
                    maxima[c * 32 + lane] = cm;
                    if (lane == 0) fast[c] = make_float2(s, mu);
                    top = fmaxf(top, cm);
                    cm = -kInf, hi = lo = mu = 0.0f, lim = -kInf;
                    left = batches;
                    ++c;
                }
            }
        }
        return top;
    }
    // The sums over the chunks of the fast weights of the elements that keep(x, column) names,
    // all of them at least `low`; the rest counts as -inf, so that no lane waits for another.
    template <class F> __device__ __forceinline__ uint64_t fast_chunks(float low, F&& keep) {
        row_sync<TX>();
        const float dmin = -200.0f / ch, mu = shift_of(m);
        const double unit = in_weights();
        float hi = 0.0f, lo = 0.0f;
        dense(low, [&](const uint32_t (&w)[kBatch][4], int s0) {
            add_pairs(hi, lo, [&](int i) {
                const int j = i / (E / 2), e = i % (E / 2);
                float x0, x1;
                f2_unpack(pair_of(w[j], e), x0, x1);
                x0 = keep(x0, column(s0 + 32 * j, 2 * e)) ? x0 : -kInf;
                x1 = keep(x1, column(s0 + 32 * j, 2 * e + 1)) ? x1 : -kInf;
                return f2_pack(x0, x1);
            }, mu, dmin);
        }, [&](int c) {
            const float s = over_lanes(hi, lo);
            if (lane == 0) sums[c] = __double2ull_rn(static_cast<double>(s) * unit);
            hi = lo = 0.0f;
        });
        return scan_chunks();
    }

    // The sum of the weights but the maximum's, of the elements that keep(x, column) names, where
    // `total` (the scanned sums', of fast weights) is well below two: so one maximum counts, the
    // first, and the sum of its chunk, whose f32 roundings are as large as the digits of a small
    // rest, is taken again without it.  x: the element of column `col`, which is kept.
    template <class F> __device__ __forceinline__ uint64_t rest_of(uint64_t total, float x, int col, F&& keep) {
        if (x != m) {
            if (tid == 0) sh.r32[0] = 0xffffffffu;
            row_sync<TX>();
            for (int i = tid; i < chunks * 32; i += TX)
                if (maxima[i] == m) atomicMin(&sh.r32[0], static_cast<uint32_t>(i >> 5));
            row_sync<TX>();
        }
        const int c = x != m ? sh.r32[0] : (col + off / EB) / E / chunk;
        const float dmin = -200.0f / ch;
        uint64_t acc = 0, over = 0;
        for (int s = chunk_begin(c) + tid; s < chunk_end(c); s += TX) {
            uint32_t w[4];
            load(s, w);
            mask(s, w);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                float x0, x1;
                f2_unpack(pair_of(w, e), x0, x1);
                x0 = x0 != m && keep(x0, column(s, 2 * e)) ? x0 : -kInf;
                x1 = x1 != m && keep(x1, column(s, 2 * e + 1)) ? x1 : -kInf;
                uint64_t lost;
                const uint64_t v = pair_weights(f2_pack(x0, x1), m, dmin, &lost);
                acc = f2_add(acc, v);
                over = f2_fma(v, lost, over);
            }
        }
        float a = 0.0f, b = 0.0f;
        add_sums(a, b, acc, over);
        const uint64_t own = __double2ull_rn(static_cast<double>(a + b) * __hiloint2double((1023 + S) << 20, 0));
        return row_sum(own) + (total - (sums[c + 1] - sums[c]));
    }

    // -----------------------------------------------------------------------
    // Threshold keys
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void clear_bins() {
        row_sync<TX>();
        for (int i = tid; i < kBins; i += TX) sh.bins[i] = 0;
        row_sync<TX>();
    }
    // Bins of the values from hi down to lo: equal parts of their distance where that is
    // finite, else of the ordered bits.  A larger value never has a larger bin; what lies
    // below lo is in the last one.  (Bits alone would put all values within a factor of two
    // into two bins, whose counters every thread would wait for.)
    struct Bins {
        float hi, scale;
        uint32_t ohi;
        int shift;
        bool linear;
        __device__ __forceinline__ Bins(uint32_t lo, uint32_t top) {
            ohi = top;
            hi = order_value(top);
            const float span = hi - order_value(lo);
            scale = kBins * 0.9999f / span;
            linear = span > 0.0f && scale > 0.0f && scale < 1e30f && span < 1e30f;
            const uint32_t bits = top - lo;
            shift = bits < kBins ? 0 : 32 - __clz(bits) - bins_log2<TX>();
        }
        // The value at which bin b begins (for `more` above 0: at which the one before ends), moved
        // down by `more` bins where bins are rounded.
        __device__ __forceinline__ float edge(int b, float more) const {
            if (linear) return hi - (static_cast<float>(b) + more) / scale;
            const int64_t o = static_cast<int64_t>(ohi) - (static_cast<int64_t>(b) << shift) + (more > 0.0f ? 1 : 0);
            // (ordered bits below those of -inf and above those of the largest value are no numbers)
            return o <= 0x007fffff ? -kInf : order_value(static_cast<uint32_t>(min(o, static_cast<int64_t>(0xff7fffffu))));
        }
        __device__ __forceinline__ int of(float x) const {
            if (linear) return static_cast<int>(fminf(fmaxf(hi - x, 0.0f) * scale, static_cast<float>(kBins - 1)));
            return min((ohi - order_bits(x)) >> shift, static_cast<uint32_t>(kBins - 1));
        }
    };
    // From the top: the first bin at which the sum of the bins reaches `need`, and the sum
    // before it; kBins if none does.
    __device__ __forceinline__ int find_bin(uint64_t need, uint64_t* before) {
        constexpr int P = kBins > TX ? kBins / TX : 1;
        row_sync<TX>();
        if (tid == 0) sh.r32[0] = kBins;
        uint64_t own = 0;
        if (tid * P < kBins) {
#pragma unroll
            for (int i = 0; i < P; ++i) own += sh.bins[tid * P + i];
        }
        uint64_t run = row_before(own);
        row_sync<TX>();
        if (run < need && need <= run + own) {
            for (int i = 0; i < P; ++i) {
                const uint64_t n = run + sh.bins[tid * P + i];
                if (n >= need) {
                    sh.r32[0] = tid * P + i;
                    sh.r64[0] = run;
                    break;
                }
                run = n;
            }
        }
        row_sync<TX>();
        const int at = sh.r32[0];
        *before = sh.r64[0];
        row_sync<TX>();
        return at;
    }
    // Elements below this weigh nothing.
    __device__ __forceinline__ uint32_t weightless() const {
        const float x = m - (S + 2) / ch;
        return x > -kInf ? min(order_bits(x), order_bits(m)) : 0;
    }
    // Elements below this all together weigh less than `rest`: N times such a weight is less.
    __device__ __forceinline__ uint32_t light(uint64_t rest) const {
        if (rest == 0) return weightless();
        const float z = __log2f(static_cast<float>(rest) / static_cast<float>(N)) - static_cast<float>(S) - 0.01f;
        const float x = m + z / ch;  // (z < 0; rounded below by the hundredth and by a step of m)
        const uint32_t o = order_bits(x - 4e-7f * fabsf(m));
        return x > -kInf && z < 0.0f ? max(weightless(), min(o, order_bits(m))) : weightless();
    }
    // Raises *lo to a value that the threshold cannot lie below, from the lanes' maxima: they
    // are elements, so as many of them, or as much of their weights, as is needed is enough.
    // false: they do not reach (lo is left).
    __device__ __forceinline__ bool bound(bool by_mass, uint64_t need, uint64_t total, uint32_t* lo) {
        const int hs = max(0, 33 - __clzll(static_cast<long long>(total)));  // total in 31 bits
        uint32_t mlo = max(*lo, weightless()), mhi = order_bits(m);
        uint64_t left = by_mass ? (need >> hs) + 1 : need;
        bool reached = false;
        for (int round = 0; round < 4; ++round) {
            const Bins bins(mlo, mhi);
            const float low = order_value(mlo), top = order_value(mhi);
            clear_bins();
            for (int i = tid; i < chunks * 32; i += TX) {
                const float x = maxima[i];
                if (x < low || x > top) continue;  // (low may be no number: then nothing is below it)
                if (by_mass) atomicAdd(&sh.bins[bins.of(x)], static_cast<uint32_t>(weight(x) >> hs));
                else atomicAdd(&sh.bins[bins.of(x)], 1u);
            }
            uint64_t before;
            const int b = find_bin(left, &before);
            if (b == kBins) {
                // Counts may need elements that weigh nothing.
                if (reached || by_mass || mlo <= *lo) break;
                mlo = *lo;
                continue;
            }
            const bool enough = by_mass ? round >= 1 : sh.bins[b] * 4ull <= need + 32;
            row_sync<TX>();
            // The bin's ends, moved out by a hundredth of its width.
            const uint32_t a = max(mlo, b == kBins - 1 ? 0u : order_bits(bins.edge(b + 1, 0.01f)));
            const uint32_t z = min(mhi, order_bits(bins.edge(b, -0.01f)));
            if (a == mlo && z == mhi) {
                *lo = a;
                return true;
            }
            // Elements above z were counted; those between the bin's end and z are counted again.
            mlo = a;
            mhi = z;
            reached = true;
            *lo = mlo;
            if (enough || mlo >= mhi) break;
            // (what was counted above z: at most `before`)
            uint64_t over = 0;
            const float zv = order_value(z);
            for (int i = tid; i < chunks * 32; i += TX)
                if (maxima[i] > zv) over += by_mass ? weight(maxima[i]) >> hs : 1;
            over = row_sum(over);
            left = (by_mass ? (need >> hs) + 1 : need) - min(over, by_mass ? need >> hs : need - 1);
        }
        return reached;
    }
    // All elements of at least `lo` to the list; returns how many there are, also where they
    // are more than it holds.
    __device__ __forceinline__ uint32_t gather(uint32_t lo) {
        if (tid == 0) sh.r32[3] = 0;
        const bool done = sparse(order_value(lo), [&](const uint32_t (&w)[4], int s, uint32_t mask) {
            uint32_t at = places(&sh.r32[3], __popc(mask));
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (mask >> e & 1) {
                    if (at < kList) sh.list[at] = key(word_elem<DT>(w, e), column(s, e));
                    ++at;
                }
        });
        const uint32_t n = sh.r32[3];
        row_sync<TX>();
        return done ? n : 0xffffffffu;
    }
    // The first n entries in descending order (bitonic; exchanges over less than 64 entries stay
    // within a warp).
    __device__ __forceinline__ void sort_list(uint64_t* v, uint32_t n) {
        uint32_t size = 2;
        while (size < n) size <<= 1;
        for (uint32_t i = n + tid; i < size; i += TX) v[i] = 0;
        row_sync<TX>();
        for (uint32_t k = 2; k <= size; k <<= 1) {
            for (uint32_t j = k >> 1; j > 0; j >>= 1) {
                for (uint32_t t = tid; t < size / 2; t += TX) {
                    const uint32_t a = 2 * t - (t & (j - 1)), b = a + j;
                    const uint64_t x = v[a], y = v[b];
                    if ((x < y) == ((a & k) == 0)) v[a] = y, v[b] = x;
                }
                if (j >= 64 || (j == 1 && k >= 64)) row_sync<TX>();
                else __syncwarp();
            }
        }
        row_sync<TX>();
    }
    // In keys v[0 .. n) in order: the first at which `before` and the running sum (of ones or
    // weights) reach `need`, and the sums before and with it.  false: they do not.
    __device__ __forceinline__ bool reach(const uint64_t* v, uint32_t n, bool by_mass, uint64_t before, uint64_t need, uint64_t* at,
                                          uint64_t* under, uint64_t* with) {
        const uint32_t per = (n + TX - 1) / TX, b = min(tid * per, n), e = min(b + per, n);
        const auto one = [&](uint32_t i) -> uint64_t { return by_mass ? weight(order_value(static_cast<uint32_t>(v[i] >> 32))) : 1; };
        uint64_t own = 0;
        for (uint32_t i = b; i < e; ++i) own += one(i);
        if (tid == 0) sh.r32[0] = 0;
        uint64_t run = before + row_before(own);
        row_sync<TX>();
        if (run < need && need <= run + own) {
            for (uint32_t i = b; i < e; ++i) {
                const uint64_t w = one(i);
                if (need <= run + w) {
                    sh.r32[0] = 1;
                    sh.r64[0] = v[i];
                    sh.r64[1] = run;
                    sh.r64[2] = run + w;
                    break;
                }
                run += w;
            }
        }
        row_sync<TX>();
        const bool ok = sh.r32[0] != 0;
        *at = sh.r64[0];
        *under = sh.r64[1];
        *with = sh.r64[2];
        row_sync<TX>();
        return ok;
    }
    // The same for the first n entries of the list with keys >= base, in whatever order they are:
    // sums by bins of their values, and the keys of the bin that reaches put in order.
    __device__ __noinline__ bool list_cut(bool by_mass, uint32_t n, uint64_t base_key, uint64_t before, uint64_t need, uint64_t* at,
                                          uint64_t* under, uint64_t* with) {
        uint64_t* const part = sh.work + kBins;
        if (n > 32) {
            uint32_t a = 0xffffffffu;
            for (uint32_t i = tid; i < n; i += TX)
                if (sh.list[i] >= base_key) a = min(a, static_cast<uint32_t>(sh.list[i] >> 32));
            a = __reduce_min_sync(0xffffffffu, a);
            if (tid == 0) sh.r32[1] = 0xffffffffu, sh.r32[2] = 0;
            row_sync<TX>();
            if (lane == 0) atomicMin(&sh.r32[1], a);
            for (int i = tid; i < kBins; i += TX) sh.work[i] = 0;
            row_sync<TX>();
            const uint32_t top = order_bits(m);
            const Bins bins(min(sh.r32[1], top), top);
            for (uint32_t i = tid; i < n; i += TX) {
                const uint64_t k = sh.list[i];
                const float x = order_value(static_cast<uint32_t>(k >> 32));
                if (k >= base_key) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.work[bins.of(x)]), by_mass ? weight(x) : 1ull);
            }
            row_sync<TX>();
            constexpr int P = kBins > TX ? kBins / TX : 1;
            uint64_t own = 0;
            if (tid * P < kBins) {
#pragma unroll
                for (int i = 0; i < P; ++i) own += sh.work[tid * P + i];
            }
            if (tid == 0) sh.r32[0] = kBins;
            uint64_t run = before + row_before(own);
            row_sync<TX>();
            if (run < need && need <= run + own) {
                for (int i = 0; i < P; ++i) {
                    const uint64_t w = sh.work[tid * P + i];
                    if (need <= run + w) {
                        sh.r32[0] = tid * P + i;
                        sh.r64[0] = run;
                        break;
                    }
                    run += w;
                }
            }
            row_sync<TX>();
            const int bin = sh.r32[0];
            const uint64_t above = sh.r64[0];
            if (bin == kBins) {
                row_sync<TX>();
                return false;
            }
            for (uint32_t i0 = 0; i0 < n; i0 += TX) {
                const uint32_t i = i0 + tid;
                const bool in = i < n && sh.list[i] >= base_key && bins.of(list_value(i)) == bin;
                const uint32_t to = places(&sh.r32[2], in ? 1 : 0);
                if (in && to < kPart) part[to] = sh.list[i];
            }
            row_sync<TX>();
            const uint32_t c = sh.r32[2];
            row_sync<TX>();
            if (c <= kPart) {
                sort_list(part, c);
                return reach(part, c, by_mass, above, need, at, under, with);
            }
        }
        sort_list(sh.list, n);  // few, or nearly all of one value
        uint32_t kept = 0;      // (keys below base come last)
        for (uint32_t i = tid; i < n; i += TX) kept += sh.list[i] >= base_key;
        kept = static_cast<uint32_t>(row_sum(kept));
        return reach(sh.list, kept, by_mass, before, need, at, under, with);
    }
    __device__ __forceinline__ float list_value(uint32_t i) const { return order_value(static_cast<uint32_t>(sh.list[i] >> 32)); }
    // The sum of the weights of the list's entries with keys >= base.
    __device__ __forceinline__ uint64_t list_sum(uint32_t n, uint64_t base_key) {
        uint64_t s = 0;
        for (uint32_t i = tid; i < n; i += TX) s += sh.list[i] >= base_key ? weight(list_value(i)) : 0;
        return row_sum(s);
    }
    // Adds the same by chunks: to sums of chunks that have not been scanned.
    __device__ __forceinline__ void list_chunks(uint32_t n, uint64_t base_key) {
        for (uint32_t i = tid; i < n; i += TX) {
            const uint64_t k = sh.list[i];
            if (k < base_key) continue;
            const int col = static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
            atomicAdd(reinterpret_cast<unsigned long long*>(&sums[(col + off / EB) / E / chunk]), weight(list_value(i)));
        }
    }

    // The least sum that is not less than the share p of the whole (at least 1).
    static __device__ __forceinline__ uint64_t mass_needed(uint64_t whole, float p) {
        bool exact;
        const uint64_t n = part_of(whole, p, &exact);
        return !exact || n == 0 ? n + 1 : n;
    }
    // A range of values that a threshold lies in, and how many elements reach its lower end.
    struct Range {
        float lo, hi;
        uint64_t through;
    };
    // The range that holds the threshold of top-p, from a sample: each lane's first vector in every
    // so many chunks.
    // What lies below the threshold has a known sum, `rest`, made of many light elements, so the
    // sample's light elements give its place to within a few percent of that, whatever a few heavy
    // elements hold; split() shows whether the threshold is in the range.
    __device__ __noinline__ bool guess(uint64_t rest, bool part_of_row, uint32_t lo_bits, Range* out) {
        constexpr int P = kBins > TX ? kBins / TX : 1;
        const uint32_t hi_bits = order_bits(m);
        const Bins bins(lo_bits, hi_bits);
        const float low = order_value(lo_bits);
        clear_bins();
        // (of every `step`-th chunk: about 2^15 elements, one vector in chunk / 32 of such a chunk)
        int step = 1;
        while (chunks / (2 * step) * 32 * E >= (1 << 15)) step *= 2;
        float light = 0.0f;  // the sample's weights below lo
        for (int c = warp * step; c < chunks; c += W * step) {
            const int s = chunk_begin(c) + lane;
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = neg_inf_word<DT>();
            if (s < chunk_end(c)) load(s, w), mask(s, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = word_elem<DT>(w, e);
                if (x >= low) atomicAdd(&sh.bins[bins.of(x)], 1u);
                else if (!part_of_row) light += ex2((x - m) * ch);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) light += __shfl_xor_sync(0xffffffffu, light, o);
        if (lane == 0) sh.warpf[warp] = light;
        row_sync<TX>();
        light = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) light += sh.warpf[i];
        // From the bottom: estimates of the sums below each bin, and of their variance.
        const float scale = static_cast<float>(chunk / 32 * step);
        const float want = static_cast<float>(rest) * __int_as_float((127 - S) << 23);
        float own = 0.0f, var = 0.0f;
        float mid[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = kBins - 1 - (tid * P + i);
            mid[i] = 0.0f;
            if (b >= 0) mid[i] = ex2((fminf(bins.edge(b, 0.5f), m) - m) * ch);
            const float c = b >= 0 ? static_cast<float>(sh.bins[b]) : 0.0f;
            own += c * mid[i];
            var += c * mid[i] * mid[i];
        }
        float s = own, v = var;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float p = __shfl_up_sync(0xffffffffu, s, o), q = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) s += p, v += q;
        }
        row_sync<TX>();
        if (lane == 31) sh.work[warp] = static_cast<uint64_t>(__float_as_uint(s)) << 32 | __float_as_uint(v);
        if (tid == 0) sh.r32[0] = 0xffffffffu, sh.r32[1] = 0xffffffffu;
        row_sync<TX>();
        float run = s - own + light, spread = v - var;
        for (int i = 0; i < warp; ++i) {
            run += __uint_as_float(static_cast<uint32_t>(sh.work[i] >> 32));
            spread += __uint_as_float(static_cast<uint32_t>(sh.work[i]));
        }
        // Four deviations (a sum of independent draws, one in `scale` elements) and a little for
        // the bins' widths.  The first bin from below whose upper end may reach, and the first
        // whose lower end certainly has passed.
        uint32_t first = 0xffffffffu, last = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int b = kBins - 1 - (tid * P + i);
            if (b < 0) continue;
            const float c = static_cast<float>(sh.bins[b]);
            run += c * mid[i];
            spread += c * mid[i] * mid[i];
            const float est = run * scale, off = 4.0f * scale * sqrtf(spread + mid[i] * mid[i]) + 0.003f * est;
            if (est + off >= want) first = min(first, static_cast<uint32_t>(tid * P + i));
            if (est - off >= want) last = min(last, static_cast<uint32_t>(tid * P + i));
        }
        first = __reduce_min_sync(0xffffffffu, first);
        last = __reduce_min_sync(0xffffffffu, last);
        if (lane == 0) atomicMin(&sh.r32[0], first), atomicMin(&sh.r32[1], last);
        row_sync<TX>();
        first = sh.r32[0];
        last = sh.r32[1];
        row_sync<TX>();
        if (first == 0xffffffffu) return false;
        const int b1 = kBins - 1 - static_cast<int>(first);  // the lower bin of the range
        const int b0 = last == 0xffffffffu ? 0 : kBins - 1 - static_cast<int>(last);
        out->lo = b1 == kBins - 1 ? low : bins.edge(b1 + 1, 0.01f);
        out->hi = b0 == 0 ? m : fminf(m, bins.edge(b0, -0.01f));
        return out->lo <= out->hi;
    }
    // Counts the elements with keys >= base from lo to hi and brackets the threshold at which
    // their count, or the sum of their weights, reaches `left` (to within err).  false: they do
    // not reach.  `guide`: where the bins end.
    __device__ __noinline__ bool bracket(bool by_mass, uint64_t left, uint64_t err, uint64_t base_key, uint32_t lo, uint32_t guide,
                                         uint32_t hi, Range* out) {
        constexpr int P = kBins > TX ? kBins / TX : 1;
        const Bins bins(guide, hi);
        const float low = order_value(lo), top = order_value(hi);
        clear_bins();
        dense(low, [&](const uint32_t (&w)[kBatch][4], int s0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = word_elem<DT>(w[j], e);
                    const int b = bins.of(x);
                    const bool in = !(x < low) && x <= top && (base_key == 0 || key(x, column(s0 + 32 * j, e)) >= base_key) &&
                                    static_cast<unsigned>(column(s0 + 32 * j, e)) < static_cast<unsigned>(N);
                    if (in) atomicAdd(&sh.bins[b], 1u);
                }
        }, [](int) {});
        int b0, b1;
        if (!by_mass) {
            uint64_t before;
            b0 = b1 = find_bin(left, &before);
            out->through = b0 < kBins ? before + sh.bins[b0] : 0;
            row_sync<TX>();
        } else {
            // A bin's weights lie between those of its ends (moved out by a hundredth of its
            // width, far more than the roundings of a bin's number); the last bin has no lower end.
            row_sync<TX>();
            if (tid == 0) sh.r32[0] = kBins, sh.r32[1] = kBins;
            uint64_t up = 0, down = 0, n = 0;
            uint64_t ups[P], downs[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = tid * P + i;
                ups[i] = downs[i] = 0;
                if (b < kBins) {
                    const uint64_t c = sh.bins[b];
                    const float x1 = fminf(bins.edge(b, -0.01f), m), x0 = b == kBins - 1 ? -kInf : fminf(bins.edge(b + 1, 0.01f), m);
                    ups[i] = c * weight(x1);
                    downs[i] = c * weight(x0);
                    n += c;
                }
                up += ups[i];
                down += downs[i];
            }
            uint64_t u = row_before(up), d = row_before(down), before = row_before(n);
            const uint64_t small = left > err ? left - err : 1, large = left + err;
            row_sync<TX>();
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = tid * P + i;
                if (b >= kBins) continue;
                before += sh.bins[b];
                if (u < small && small <= u + ups[i]) sh.r32[0] = b;
                if (d < large && large <= d + downs[i]) sh.r32[1] = b, sh.r64[0] = before;
                if (b == kBins - 1) sh.r64[1] = before;
                u += ups[i];
                d += downs[i];
            }
            row_sync<TX>();
            b0 = sh.r32[0];
            out->through = sh.r32[1] < kBins ? sh.r64[0] : sh.r64[1];
            b1 = min(sh.r32[1], static_cast<uint32_t>(kBins - 1));
            row_sync<TX>();
        }
        if (b0 >= kBins) return false;
        out->hi = fminf(top, b0 == 0 ? top : bins.edge(b0, -0.01f));
        const float edge = b1 == kBins - 1 ? low : bins.edge(b1 + 1, 0.01f);
        out->lo = edge > low ? edge : low;  // (low may be no number)
        return true;
    }
    // Weights of pairs A .. A + L - 1 of a batch above the range, and of those below it, by halves.
    template <int A, int L>
    __device__ __forceinline__ uint64_t split_pairs(const uint32_t (&w)[kBatch][4], const Range& at, float mu, float dmin, uint64_t& over_above,
                                                    uint64_t& over_below, uint64_t* below) const {
        if constexpr (L == 1) {
            float x0, x1, w0, w1;
            uint64_t lost;
            f2_unpack(pair_of(w[A / (E / 2)], A % (E / 2)), x0, x1);
            f2_unpack(pair_weights(f2_pack(x0, x1), mu, dmin, &lost), w0, w1);
            const uint64_t u = f2_pack(x0 > at.hi ? w0 : 0.0f, x1 > at.hi ? w1 : 0.0f);
            *below = f2_pack(x0 < at.lo ? w0 : 0.0f, x1 < at.lo ? w1 : 0.0f);
            over_above = f2_fma(u, lost, over_above);
            over_below = f2_fma(*below, lost, over_below);
            return u;
        } else {
            uint64_t b0, b1;
            const uint64_t s = split_pairs<A, L / 2>(w, at, mu, dmin, over_above, over_below, &b0);
            const uint64_t r = split_pairs<A + L / 2, L / 2>(w, at, mu, dmin, over_above, over_below, &b1);
            *below = f2_add(b0, b1);
            return f2_add(s, r);
        }
    }
    // Sums what lies above a range by chunks (left in `added`, not scanned), and puts the range's
    // elements to the list; returns the sum of all chunks and, in *n, how many elements are in the range.
    // Of fast weights also what lies below the range, *under.
    template <bool EXACT, bool MASS>
    __device__ __noinline__ uint64_t split(Range at, uint32_t* n, uint32_t* least, uint32_t* most, uint64_t* under) {
        row_sync<TX>();
        if (tid == 0) sh.r32[3] = 0, sh.r32[0] = 0xffffffffu, sh.r32[1] = 0;
        row_sync<TX>();
        uint32_t a = 0xffffffffu, z = 0;
        const float dmin = -200.0f / ch, mu = shift_of(m);
        const double unit = in_weights();
        float hi = 0.0f, lo = 0.0f, under_hi = 0.0f, under_lo = 0.0f;
        uint64_t exact = 0, ehi = 0, elo = 0;
        const float high = kHigh[lane], rest = kLow[lane], far60 = -60.0f / ch;
        const bool beyond = !(at.lo > -kInf);  // elements outside the row are -inf
        dense(EXACT ? at.lo : -kInf, [&](const uint32_t (&w)[kBatch][4], int s0) {
            uint32_t mask = 0;  // of the range's elements, at most 32
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = word_elem<DT>(w[j], e);
                    if (!(x < at.lo) && x <= at.hi) mask |= 1u << (j * E + e);
                    if constexpr (!MASS) exact += x > at.hi ? 1 : 0;
                }
            if constexpr (MASS && EXACT) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        float x0, x1;
                        f2_unpack(pair_of(w[j], e), x0, x1);
                        add_exact_pair(ehi, elo, f2_pack(x0 > at.hi ? x0 : -kInf, x1 > at.hi ? x1 : -kInf), high, rest, far60);
                    }
            }
            if constexpr (!EXACT) {
                uint64_t over_above = 0, over_below = 0, below;
                const uint64_t above = split_pairs<0, kBatch * E / 2>(w, at, mu, dmin, over_above, over_below, &below);
                add_sums(hi, lo, above, over_above);
                add_sums(under_hi, under_lo, below, over_below);
            }
            if (beyond) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (static_cast<unsigned>(column(s0 + 32 * j, e)) >= static_cast<unsigned>(N)) mask &= ~(1u << (j * E + e));
            }
            if (__any_sync(0xffffffffu, mask != 0)) {
                uint32_t to = places(&sh.r32[3], __popc(mask));
                while (mask) {  // (few: read again, so that no register is indexed)
                    const int i = __ffs(mask) - 1;
                    mask &= mask - 1;
                    const int col = column(s0 + 32 * (i / E), i % E);
                    const uint64_t k = key(load_elem<DT>(base + off, col), col);
                    a = min(a, static_cast<uint32_t>(k >> 32));
                    z = max(z, static_cast<uint32_t>(k >> 32));
                    if (to < kList) sh.list[to] = k;
                    ++to;
                }
                __syncwarp();
            }
        }, [&](int c) {
            if constexpr (EXACT) {
                const uint64_t v = MASS ? exact_sum(ehi, elo) : warp_sum(exact);
                if (lane == 0) sums[c] = added[c] = v;
                exact = ehi = elo = 0;
            } else {
                const float s = over_lanes(hi, lo);
                if (lane == 0) sums[c] = added[c] = __double2ull_rn(static_cast<double>(s) * unit);
                hi = lo = 0.0f;
            }
        });
        const uint64_t sum = scan_chunks();
        if constexpr (!EXACT)
            *under = row_sum(__double2ull_rn((static_cast<double>(under_hi) + static_cast<double>(under_lo)) * unit));
        a = __reduce_min_sync(0xffffffffu, a);
        z = __reduce_max_sync(0xffffffffu, z);
        if (lane == 0) atomicMin(&sh.r32[0], a), atomicMax(&sh.r32[1], z);
        row_sync<TX>();
        *n = sh.r32[3];
        *least = sh.r32[0];
        *most = sh.r32[1];
        row_sync<TX>();
        return sum;
    }
    // The threshold key of the shortest prefix (of the elements with keys >= base) whose count
    // or sum of weights reaches `need` (>= 1), given to within `doubt` (0: exact weights are used
    // throughout); `base_key` where all of them do not.  It lies above lo (ordered bits).
    // *sure is false where the doubt left it open; *listed: the threshold is in the list of *listed
    // entries, and what lies above those is summed in `added` (0: it is not).
    __device__ __noinline__ uint64_t select(bool by_mass, uint64_t need, uint64_t total, float share, Doubt doubt, uint64_t base_key,
                                            uint32_t lo, uint32_t guide, bool* sure, uint32_t* listed) {
        const uint64_t err = doubt.any;
        uint64_t left = need;
        uint32_t hi = order_bits(m);
        const uint32_t lowest = lo, first_guide = guide;
        bool tentative = false;
        *sure = err == 0;
        *listed = 0;
        // (Each round leaves half of the ordered bits of its range or a quarter of its length: a few
        // rounds as a rule, and less than 128 from any range.)
        for (int round = 0; round < 128; ++round) {
            Range at;
            const bool sampled = round == 0 && by_mass && total > need && chunks >= 16 && guess(total - need, base_key != 0, lo, &at);
            if (!sampled && !bracket(by_mass, left, err, base_key, lo, guide, hi, &at)) {
                // (Exact sums and the weights of single elements differ by 2^-30, so that a range can
                // fall short of what it has to reach by that: all of it is kept then.)
                if (!tentative) {
                    if (!by_mass) lost = true;  // (fewer than the count: lo was no bound)
                    return err == 0 && by_mass ? max(base_key, static_cast<uint64_t>(lo) << 32) : base_key;
                }
                tentative = false;  // the sample was wrong
                lo = lowest, guide = first_guide, hi = order_bits(m), left = need;
                continue;
            }
            uint32_t n, least, most;
            uint64_t k, under = 0, with;
            const uint64_t above = !by_mass ? split<true, false>(at, &n, &least, &most, &under)
                                   : err ? split<false, true>(at, &n, &least, &most, &under) : split<true, true>(at, &n, &least, &most, &under);
            // Of fast weights the same pass sums the whole, so that what is above has the same errors in
            // both (those of an addition depend on what else is added, and differ from pass to pass).
            const uint64_t whole = above + under;
            const uint64_t border = err && n <= kList ? mass_needed(whole + list_sum(n, 0), share) : need;
            if (above < border && n <= kList && list_cut(by_mass, n, base_key, above, border, &k, &under, &with)) {
                *sure = err == 0 || doubt.sure(under, border, with, 0);
                *listed = by_mass ? n : 0;
                return k;
            }
            if (sampled) {
                if (above >= need || n <= kList) continue;  // not in the range: histograms find it
                tentative = true;
                left = need - above;
                lo = guide = least;
                hi = most;
                continue;
            }
            if (tentative && (n <= kList || above >= need)) {  // the sample was wrong
                tentative = false;
                lo = lowest, guide = first_guide, hi = order_bits(m), left = need;
                continue;
            }
            if (n <= kList || above >= need) {
                if (err) return base_key;  // not sure
                if (!by_mass) return lost = true, base_key;
                // Off by the 2^-30 again: the range's first element, or all of it.
                if (n <= kList) {
                    const uint64_t in = list_sum(n, base_key);
                    if (in == 0) return max(base_key, (static_cast<uint64_t>(order_bits(at.hi)) + 1) << 32);
                    const uint64_t reached = min(max(need, above + 1), above + in);
                    if (!list_cut(true, n, base_key, above, reached, &k, &under, &with)) return lost = true, base_key;
                    *listed = n;
                    return k;
                }
            }
            left = need > above ? need - above : 1;
            const float was = order_value(hi) - order_value(lo), now = order_value(most) - order_value(least);
            const bool poor = most - least > (hi - lo) / 2 && !(was < kInf && now <= 0.25f * was);
            if (err && (least == most || poor)) return base_key;  // not sure
            if (by_mass && poor && least < most) {
                // Heavy equal values: the widths of bins leave more open than lies between the sums.
                const uint32_t mid = least + (most - least) / 2;
                const float pivot = order_value(mid);
                const uint64_t half = exact_chunks(pivot, [=](float v, int) -> bool { return v > pivot; });
                if (half >= need) {
                    lo = guide = mid + 1;
                    hi = most;
                } else {
                    lo = guide = least;
                    hi = mid;
                    left = need - half;
                }
                continue;
            }
            if (least == most) {  // equal values: a count of columns
                const uint64_t one = by_mass ? weight(order_value(least)) : 1;
                uint64_t count = one ? (left + one - 1) / one : 1;
                const auto same = [=](float v, int col) -> uint64_t {
                    return order_bits(v) == least && static_cast<unsigned>(col) < static_cast<unsigned>(N) && key(v, col) >= base_key;
                };
                const uint64_t all = count_chunks(order_value(least), same);
                if (count > all && tentative) {  // the sample was wrong
                    tentative = false;
                    lo = lowest, guide = first_guide, hi = order_bits(m), left = need;
                    continue;
                }
                if (all == 0) return lost = true, base_key;
                if (count > all) count = all;
                int col = 0;
                float value;
                uint64_t b, w;
                uint64_t inside;
                if (!locate(count - 1, false, same, &col, &value, &b, &w, &inside)) lost = true;
                return (static_cast<uint64_t>(least) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
            }
            lo = guide = least;
            hi = most;
        }
        lost = err == 0;  // (else it is not sure)
        return base_key;
    }
};

// A row's settings.
struct RowSettings {
    float temperature, top_p, min_p, u;
    int64_t top_k;
    float ch, cl;  // log2 e / T in two floats
    bool greedy, use_k, use_p, use_min, valid;
    __device__ __forceinline__ RowSettings(const SampleArgs& a, int64_t row) {
        temperature = a.temperature ? a.temperature[row] : a.temperature_all;
        top_k = a.top_k ? a.top_k[row] : a.top_k_all;
        top_p = a.top_p ? a.top_p[row] : a.top_p_all;
        min_p = a.min_p ? a.min_p[row] : a.min_p_all;
        u = a.u[row];
        greedy = temperature < kSampleGreedy;
        use_k = top_k > 0 && top_k < a.N && !greedy;
        use_p = top_p < 1.0f && !greedy;
        use_min = min_p > 0.0f && !greedy;
        valid = temperature >= 0.0f && temperature <= kSampleHottest && top_p >= 0.0f && min_p >= 0.0f;  // (NaN: none)
        // the quotient of the first 24 bits, and what the remainder and the next bits add
        const float t = greedy ? 1.0f : temperature;
        ch = __fdiv_rn(kLog2e, t);
        cl = __fdiv_rn(fmaf(-ch, t, kLog2e) + 1.92596299e-8f, t);
    }
};

__device__ __forceinline__ void put_token(const SampleArgs& a, int64_t row, int64_t token, float logprob) {
    a.token[row] = token;
    if (a.logprob) a.logprob[row] = logprob;
}

// One row by the TX threads of its group.  `dynamic`: chunks + 1 sums, chunks pairs, and the
// lanes' maxima.
template <int DT, int TX>
__device__ void sample_row(SampleShared<TX>& sh, const uint32_t* powers, unsigned char* dynamic, const SampleArgs& a, int64_t row) {
    using R = Sampler<DT, TX>;
    const RowSettings g(a, row);
    R r(sh);
    r.powers = powers;
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
    r.sums = reinterpret_cast<uint64_t*>(dynamic);
    float2* fast = reinterpret_cast<float2*>(r.sums + r.chunks + 1);
    r.added = reinterpret_cast<uint64_t*>(fast);
    r.maxima = reinterpret_cast<float*>(fast + r.chunks);
    r.ch = g.ch;
    r.cl = g.cl;
    r.S = a.bits;
    r.far = -static_cast<float>(a.bits + 3) / g.ch;
    row_sync<TX>();
    // A greedy row needs no sums, nor does one whose top_k cuts the rest off before any sum.
    const bool with_sums = !(g.greedy || g.use_k);
    r.m = r.row_max(r.first_pass(fast, with_sums));
    row_sync<TX>();
    // Chunks' sums relative to the maximum, in whole numbers.
    const bool bad = !g.valid || !(fabsf(r.m) < kInf);
    int nan = 0;
    for (int c = r.tid; c < r.chunks; c += TX) {
        const float2 f = fast[c];
        nan |= f.x != f.x;
        if (with_sums) {
            const double v = f.x > 0.0f && !bad ? static_cast<double>(f.x) * r.factor(f.y) : 0.0;
            r.sums[c] = v < kInf ? __double2ull_rn(v * __hiloint2double((1023 + r.S) << 20, 0)) : 0;
        }
    }
    if constexpr (TX == 32) nan = __any_sync(0xffffffffu, nan);
    else nan = __syncthreads_or(nan);
    const auto mark = [&]() {
        if (r.tid == 0) put_token(a, row, -1, __int_as_float(0x7fc00000));
    };
    if (bad || nan) return mark();
    const uint32_t top = order_bits(r.m);
    if (g.greedy) {
        if (r.tid == 0) sh.r32[0] = 0xffffffffu;
        row_sync<TX>();
        uint32_t best = 0xffffffffu;
        const auto lower = [&](const uint32_t (&w)[4], int s, uint32_t) {
            for (int e = R::E - 1; e >= 0; --e)
                if (s >= 0 && word_elem<DT>(w, e) == r.m) best = min(best, static_cast<uint32_t>(r.column(s, e)));
        };
        if (!r.sparse(r.m, lower))  // the maximum nearly everywhere
            r.dense(r.m, [&](const uint32_t (&w)[kBatch][4], int s0) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) lower(w[j], s0 + 32 * j, 0);
            }, [](int) {});
        best = __reduce_min_sync(0xffffffffu, best);
        if (r.lane == 0) atomicMin(&sh.r32[0], best);
        row_sync<TX>();
        if (r.tid == 0) put_token(a, row, sh.r32[0], 0.0f);
        return;
    }
    // The maximum is kept and weighs 1: log(1 + rest) keeps the digits of a small rest.
    const uint64_t one = 1ull << r.S;
    const auto finish = [&](int64_t token, float x, uint64_t rest) {
        put_token(a, row, token, (x - r.m) / g.temperature - log1pf(static_cast<float>(rest) * __int_as_float((127 - r.S) << 23)));
    };
    const auto drawn = [&](uint64_t total) -> uint64_t {
        bool whole;
        return g.u >= 1.0f ? total - 1 : part_of(total, g.u, &whole);
    };
    const auto all_weights = [&](float x, int) -> uint64_t { return r.weight(x); };
    uint64_t total = 0;
    bool rough = with_sums;  // the sums are of fast weights
    if (with_sums) total = r.scan_chunks();
    // Whether sums leave no doubt.  (Most are farther from a border than any doubt, which is less than
    // 2^-18 of the whole.)
    const auto sure = [&](float share, uint64_t before, uint64_t target, uint64_t with, uint64_t summed) {
        const uint64_t wide = total >> 18;
        if (target - before > wide && with - target > wide && total > 1ull << 40) return true;
        return Doubt(total, share, fast_error<DT>(), r.whole_distances(), r.N, r.S).sure(before, target, with, summed);
    };
    const auto doubt = [&](float share) { return rough ? Doubt(total, share, fast_error<DT>(), r.whole_distances(), r.N, r.S) : Doubt(); };
    uint32_t floor_bits = 0;  // of min_p
    if (g.use_min) {
        // x - m >= T log(min_p) in 64 bits, as a comparison of x in 32.
        if (r.tid == 0) {
            const double v = static_cast<double>(r.m) + static_cast<double>(g.temperature) * log(static_cast<double>(fminf(g.min_p, 1.0f)));
            sh.r32[0] = min(order_bits(__double2float_ru(v)), top);
        }
        row_sync<TX>();
        floor_bits = sh.r32[0];
        row_sync<TX>();
    }
    uint64_t threshold = 0;
    bool exact = false;   // sums are
    uint32_t listed = 0;  // entries of the list, if what is kept is those and what `added` sums
    if (g.use_k || g.use_p || g.use_min) {
        // Everything that can be kept in a list, if it fits.  lo: a bound that all of it reaches.
        const uint64_t need = g.use_k ? static_cast<uint64_t>(g.top_k) : g.use_p ? R::mass_needed(total, g.top_p) : 0;
        const bool by_mass = !g.use_k;
        uint32_t lo = 0, guide = 0, n = 0;
        bool fits;
        if (need) {
            const uint64_t err = by_mass ? doubt(g.top_p).any : 0;
            if (by_mass) lo = r.light(total > need + 2 * err ? total - need - 2 * err : 0);
            guide = lo;
            fits = r.bound(by_mass, need + err, total, &lo);
            if (fits) guide = lo;
            else if (!by_mass) r.bound(false, r.chunks * 24, 0, &guide);  // where three quarters of the maxima lie above
        } else {
            fits = true;
        }
        if (g.use_min && by_mass && floor_bits >= lo) lo = guide = floor_bits, fits = true;
        if (a.N <= R::kList) fits = true;
        if (fits) {
            n = r.gather(lo);
            fits = n <= R::kList;
        }
        if (!fits && need && !by_mass && need <= R::kList) {
            typename R::Range at;
            if (r.bracket(false, need, 0, 0, lo, guide, top, &at) && at.through <= R::kList) {
                n = r.gather(order_bits(at.lo));
                fits = n <= R::kList;
            }
        }
        if (fits) {
            uint64_t cut = 0, under, with;
            if (g.use_k && !r.list_cut(false, n, 0, 0, static_cast<uint64_t>(g.top_k), &cut, &under, &with)) return mark();
            if (g.use_p) {
                const uint64_t base = cut;
                for (;;) {
                    const uint64_t mass = R::mass_needed(g.use_k ? r.list_sum(n, base) : total, g.top_p);
                    const Doubt e = g.use_k ? Doubt() : doubt(g.top_p);
                    uint64_t k;
                    const bool found = r.list_cut(true, n, base, 0, mass, &k, &under, &with);
                    cut = found ? k : max(cut, static_cast<uint64_t>(lo) << 32);
                    // (Not reached: the cut lies below what min_p keeps.)
                    if (!e.any || (found ? e.sure(under, mass, with, with) : g.use_min && mass - r.list_sum(n, base) > e.any)) break;
                    total = r.exact_chunks(-kInf, [](float, int) -> bool { return true; });  // too close to tell
                    rough = false;
                }
            }
            threshold = max(cut, static_cast<uint64_t>(floor_bits) << 32);
            row_sync<TX>();
            for (int c = r.tid; c < r.chunks; c += TX) r.sums[c] = 0;
            row_sync<TX>();
            r.list_chunks(n, threshold);
            total = r.scan_chunks();
            const auto kept = [&](float v, int c) -> uint64_t { return R::key(v, c) >= threshold ? r.weight(v) : 0; };
            int col;
            float x;
            uint64_t before, inside;
            if (!r.locate(drawn(total), false, kept, &col, &x, &before, &with, &inside)) return mark();
            if (r.tid == 0) finish(col, x, total - one);
            return;
        }
        if (g.use_k) {
            bool sure;
            threshold = r.select(false, static_cast<uint64_t>(g.top_k), 0, 0.0f, Doubt(), 0, lo, guide, &sure, &listed);
            if (r.lost) return mark();
        }
        if (g.use_p) {
            const uint64_t base = threshold;
            if (g.use_k) {
                total = r.exact_chunks(order_value(static_cast<uint32_t>(base >> 32)), [&](float x, int col) -> bool { return R::key(x, col) >= base; });
                rough = false;
            }
            for (;;) {
                bool sure;
                const uint64_t mass = R::mass_needed(total, g.top_p);
                const Doubt e = doubt(g.top_p);
                const uint32_t from = max(static_cast<uint32_t>(base >> 32), r.light(total > mass + 2 * e.any ? total - mass - 2 * e.any : 0));
                const uint64_t t = r.select(true, mass, total, g.top_p, e, base, from, from, &sure, &listed);
                if (r.lost) return mark();
                if (sure || !rough) {
                    threshold = max(threshold, t);
                    exact = !rough;
                    break;
                }
                total = r.exact_chunks(-kInf, [](float, int) -> bool { return true; });  // too close to tell
                rough = false;
            }
        }
        const uint64_t t = static_cast<uint64_t>(floor_bits) << 32;
        if (t > threshold) threshold = t, listed = 0;
    }
    int col = 0;
    float x = 0.0f;
    uint64_t before = 0, with = 0, inside = 0, rest = 0;
    // Where f32 sums hold the maximum's weight, they are good to 1e-7 of that.
    const auto rest_from = [&](const auto& keep) { return rough && total < one + one / 4 * 3 ? r.rest_of(total, x, col, keep) : total > one ? total - one : 0; };
    if (threshold == 0) {  // nothing is cut off
        if (!with_sums || g.use_p) {  // (the sums of chunks are not there, or select() has used their place)
            total = r.exact_chunks(-kInf, [](float, int) -> bool { return true; });
            rough = false;
        }
        for (;;) {
            const uint64_t target = drawn(total);
            const bool found = r.locate(target, !rough, all_weights, &col, &x, &before, &with, &inside);
            if (!rough && !found) return mark();
            if (!rough || (found && sure(g.u, before, target, with, inside))) break;
            total = r.exact_chunks(-kInf, [](float, int) -> bool { return true; });  // too close to tell
            rough = false;
        }
        rest = rest_from([](float, int) -> bool { return true; });
    } else {
        const uint32_t bits = static_cast<uint32_t>(threshold >> 32);
        const float low = order_value(bits);
        const uint32_t place = static_cast<uint32_t>(threshold);
        const int last = place == 0 ? INT_MAX : static_cast<int>(0xffffffffu - place);  // column, at the value `low`
        const auto kept = [&](float v, int c) -> uint64_t { return R::key(v, c) >= threshold ? r.weight(v) : 0; };
        if (listed) {
            row_sync<TX>();
            for (int c = r.tid; c < r.chunks; c += TX) r.sums[c] = r.added[c];
            row_sync<TX>();
            r.list_chunks(listed, threshold);
            total = r.scan_chunks();
            rough = !exact;
        } else {
            total = r.fast_chunks(low, [&](float v, int c) -> bool { return v > low || (v == low && c <= last); });
            rough = true;
        }
        const uint64_t target = drawn(total);
        const bool found = r.locate(target, !rough, kept, &col, &x, &before, &with, &inside);
        if (rough && !(found && sure(g.u, before, target, with, inside))) {  // too close to tell
            total = r.exact_chunks(low, [&](float v, int c) -> bool { return v > low || (v == low && c <= last); });
            if (!r.locate(drawn(total), true, kept, &col, &x, &before, &with, &inside)) return mark();
            rough = false;
        } else if (!found) {
            return mark();
        }
        rest = rest_from([&](float v, int c) -> bool { return v > low || (v == low && c <= last); });
    }
    if (r.tid == 0) finish(col, x, rest);
}

template <int TX> __host__ __device__ constexpr int sample_ctas() { return TX == 128 ? 8 : TX == 256 ? 4 : 1; }
template <int DT, int TX> __global__ void __launch_bounds__(TX, sample_ctas<TX>()) sample_kernel(SampleArgs a) {
    __shared__ SampleShared<TX> sh;
    __shared__ uint32_t powers[64];
    extern __shared__ __align__(16) unsigned char dynamic[];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < 64; i += TX) powers[i] = kPowers[i];
    sample_row<DT, TX>(sh, powers, dynamic, a, blockIdx.x);
}

// Vectors of a chunk, by the row's length alone: whole batches, and as many chunks as 32 KB
// of maxima hold.
void plan_chunks(SampleArgs* a, int EB, int W) {
    const int64_t slots = (a->N * EB + 15) / 16 + 1;  // one more for rows off a boundary
    int64_t chunk = kChunk;
    while ((slots + chunk - 1) / chunk > 256) chunk *= 2;
    a->chunk = static_cast<int>(chunk);
    a->chunks_per_warp = static_cast<int>(((slots + chunk - 1) / chunk + W - 1) / W);
}
__host__ __device__ constexpr size_t chunk_bytes(int chunks) {
    return (chunks + 1) * sizeof(uint64_t) + chunks * (sizeof(float2) + 32 * sizeof(float));
}

constexpr int kMostDynamic = 64 * 1024;  // chunk_bytes(256 + 16) is 43 KB

template <int DT, int TX> cudaError_t launch_sample_rows(SampleArgs a, cudaStream_t s) {
    plan_chunks(&a, DType<DT>::bytes, TX / 32);
    const size_t smem = chunk_bytes(a.chunks_per_warp * (TX / 32));
    auto kernel = sample_kernel<DT, TX>;
    // (The same value in every call: calls of other threads do not lower it in between.)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(kernel, dim3(static_cast<unsigned>(a.B)), dim3(TX), smem, s, a);
}

// ---------------------------------------------------------------------------
// Rows of up to 256 vectors: a warp each, V vectors per lane in registers, sums in f32.
// ---------------------------------------------------------------------------
constexpr int kShortWarps = 4;
constexpr int kShortBins = 1 << bins_log2<32>();

template <int DT> struct ShortShared {
    SampleShared<32> row;
    uint64_t dynamic[(chunk_bytes(2) + 7) / 8];
    uint64_t keys[32];
};

template <int DT, int V> struct ShortRow {
    static constexpr int EB = DType<DT>::bytes, E = 16 / EB, M = V * E;
    uint32_t raw[V][4];
    float w[M];  // weights; element j of the lane: vector j / E of its V, lanes next to each other
    int col0, lane;
    float m, ch, cl;
    __device__ __forceinline__ float x(int j) const { return word_elem<DT>(raw[j / E], j % E); }
    __device__ __forceinline__ int column(int j) const { return (j / E * 32 + lane) * E + j % E - col0; }
    __device__ __forceinline__ float weight(float v) const {
        const float d = v - m, t = d * ch, e = fmaf(d, cl, fmaf(d, ch, -t));  // e: what t lost (NaN for -inf)
        return t > -126.0f ? fmaf(ex2(t), e * kLn2, ex2(t)) : 0.0f;
    }
    // What a comparison of a part with a share u of the whole may be off by, of the whole.  Both add
    // the same weights, whose errors count half at most (ex2's 1.46e-7 and a rounding) or once (2^-24
    // of (m - x) / T, at most log 2048 = 7.6 over the weights): 5.6e-7.  The part of a cut passes
    // through M + 12 additions at most, that of a draw through 2 E + V + 7, and the whole, of which the
    // share is taken, through log M + 5 (11 at most) or E + V + 4.
    static __device__ __forceinline__ float cut_error(float u) { return fmaf(fminf(u, 1.0f), 11 * 6e-8f, (M + 12) * 6e-8f + 5.6e-7f); }
    static __device__ __forceinline__ float draw_error(float u) {
        return fmaf(fminf(u, 1.0f), (E + V + 4) * 6e-8f, (2 * E + V + 7) * 6e-8f + 5.6e-7f);
    }
    // By halves: the largest weight passes through log M roundings instead of M.
    template <int A, int L> __device__ __forceinline__ float part() const {
        if constexpr (L == 1) return w[A];
        else return part<A, L / 2>() + part<A + L / 2, L - L / 2>();
    }
    __device__ __forceinline__ float sum() const {
        float s = part<0, M>();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
    // Cuts off what lies behind the shortest prefix (of the elements with a positive weight, or
    // of all for a count) that reaches `need`; false where f32 sums cannot tell.
    __device__ __forceinline__ bool cut(bool by_mass, float need, float total, float err, uint64_t* keys, uint32_t* bins) {
        uint32_t ohi = order_bits(m), olo;
        {
            float low = kInf;
#pragma unroll
            for (int j = 0; j < M; ++j)
                if (by_mass ? w[j] > 0.0f : column(j) >= 0) low = fminf(low, x(j));
            olo = __reduce_min_sync(0xffffffffu, order_bits(low));
            olo = olo > 0 ? olo - 1 : 0;
        }
        float above = 0.0f;
        // First a histogram of counts: over the values from the largest down to where the rest is
        // lighter than what lies behind the threshold, or to the smallest of the lanes' maxima
        // (of which there are 32), and as far again.
        float low = m;
        if (by_mass) {
            const float z = __log2f(fmaxf(total - need, 1e-7f * total) / static_cast<float>(32 * M)) - 0.01f;
            low = m + z / ch;
        } else {
            float top = x(0);
#pragma unroll
            for (int j = 1; j < M; ++j) top = fmaxf(top, x(j));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fminf(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = need <= 32.0f ? top : m - 2.0f * (m - top);
        }
        const float scale = kShortBins * 0.9999f / (m - low);
        // (Of 12 elements or fewer a lane, bisection takes fewer instructions for sums.)
        if ((!by_mass || M > 12) && scale > 0.0f && scale < 1e30f && m - low < 1e30f) {
            constexpr int P = kShortBins / 32;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < P; ++i) bins[lane * P + i] = 0;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < M; ++j)
                if (x(j) >= low && (!by_mass || w[j] > 0.0f)) atomicAdd(&bins[static_cast<int>((m - x(j)) * scale)], 1u);
            __syncwarp();
            // By the weights of a bin's ends where they count.
            float up = 0.0f, down = 0.0f, ups[P], downs[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int b = lane * P + i;
                const float c = static_cast<float>(bins[b]);
                ups[i] = downs[i] = c;
                if (by_mass) {
                    ups[i] *= weight(fminf(m, m - (static_cast<float>(b) - 0.01f) / scale));
                    downs[i] *= weight(m - (static_cast<float>(b) + 1.01f) / scale);
                }
                up += ups[i];
                down += downs[i];
            }
            float su = up, sd = down;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float p = __shfl_up_sync(0xffffffffu, su, o), q = __shfl_up_sync(0xffffffffu, sd, o);
                if (lane >= o) su += p, sd += q;
            }
            su -= up;
            sd -= down;
            int b0 = INT_MAX, b1 = INT_MAX;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                su += ups[i];
                sd += downs[i];
                if (su >= need - err && b0 == INT_MAX) b0 = lane * P + i;
                if (sd >= need + err && b1 == INT_MAX) b1 = lane * P + i;
            }
            b0 = __reduce_min_sync(0xffffffffu, b0);
            b1 = __reduce_min_sync(0xffffffffu, b1);
            if (b0 != INT_MAX && b1 != INT_MAX) {
                const float hi = b0 == 0 ? m : fminf(m, m - (static_cast<float>(b0) - 0.01f) / scale);
                const float lo = m - (static_cast<float>(b1) + 1.01f) / scale;
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < M; ++j) s += x(j) > hi ? (by_mass ? w[j] : 1.0f) : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                above = s;
                ohi = order_bits(hi);
                olo = max(olo, order_bits(lo));
            }
        } else if (by_mass && low < m) {
            olo = max(olo, order_bits(low));
        }
        // Bisection to at most 32 elements in (lo, hi] that hold the last kept one: values for
        // sums, whose relevant elements lie within a few octaves; bits of ordered values for counts.
        const auto beyond = [&](float v) -> int {  // elements above v
            int c = 0;
#pragma unroll
            for (int j = 0; j < M; ++j) c += !(x(j) <= v) ? 1 : 0;
            return __reduce_add_sync(0xffffffffu, c);
        };
        int from_lo = beyond(order_value(olo)), from_hi = beyond(order_value(ohi));
        bool settled = from_lo - from_hi <= 32;
        for (int step = 0; step < 64 && !settled; ++step) {
            if (ohi - olo < 2) return false;  // more than 32 equal values
            uint32_t mid = olo + (ohi - olo) / 2;
            if (by_mass) {
                const uint32_t v = order_bits(0.5f * order_value(olo) + 0.5f * order_value(ohi));
                if (v > olo && v < ohi) mid = v;
            }
            const float pivot = order_value(mid);
            float s = 0.0f;
            int c = 0;
#pragma unroll
            for (int j = 0; j < M; ++j)
                if (x(j) > pivot) s += by_mass ? w[j] : 1.0f, ++c;
            if (by_mass) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (!by_mass) s = static_cast<float>(c);
            if (by_mass && fabsf(s - need) <= err) return false;
            if (s >= need) {
                olo = mid;
                from_lo = c;
            } else {
                ohi = mid;
                above = s;
                from_hi = c;
            }
            settled = from_lo - from_hi <= 32;
        }
        if (!settled) return false;
        // One element per lane, in order.
        const float lo = order_value(olo), hi = order_value(ohi);
        uint32_t at = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const bool in = !(x(j) <= lo) && x(j) <= hi && (by_mass ? w[j] > 0.0f : column(j) >= 0);
            const uint32_t b = __ballot_sync(0xffffffffu, in);
            if (in) keys[at + __popc(b & ((1u << lane) - 1u))] = topk_key(x(j), static_cast<uint32_t>(column(j)));
            at += __popc(b);
        }
        __syncwarp();
        const uint64_t key = list_sort(lane < static_cast<int>(at) ? keys[lane] : 0, lane);
        const bool real = lane < static_cast<int>(at);
        float s = !real ? 0.0f : by_mass ? weight(key_value(key)) : 1.0f;
        const float own = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float b = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += b;
        }
        s += above;
        const uint32_t reach = __ballot_sync(0xffffffffu, real && s >= need);
        if (reach == 0) return false;
        const int last = __ffs(reach) - 1;
        const float over = __shfl_sync(0xffffffffu, s - need, last), under = __shfl_sync(0xffffffffu, need - (s - own), last);
        if (by_mass && (over <= err || under <= err)) return false;
        const uint64_t threshold = __shfl_sync(0xffffffffu, key, last);
        const float tx = key_value(threshold);
        const int tc = static_cast<int>(key_column(threshold));
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (!(x(j) > tx || (x(j) == tx && column(j) <= tc))) w[j] = 0.0f;
        return true;
    }
};

// false: the row is left to sample_row.
template <int DT, int V> __device__ __forceinline__ bool sample_short(const SampleArgs& a, int64_t row, int lane, uint64_t* keys, uint32_t* bins) {
    using R = ShortRow<DT, V>;
    constexpr int E = R::E, M = R::M;
    const RowSettings g(a, row);
    const char* x0 = static_cast<const char*>(a.x) + row * a.row_stride * R::EB;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15);
    const char* base = x0 - off;
    const int end = off + static_cast<int>(a.N) * R::EB, slots = a.N == 0 ? 0 : (end + 15) / 16;
    R r;
    r.lane = lane;
    r.col0 = off / R::EB;
    r.ch = g.ch;
    r.cl = g.cl;
    auto& w = r.raw;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int s = v * 32 + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[v][i] = neg_inf_word<DT>();
        if (s < slots) {
            const uint4 q = ldg_stream16(base + s * 16);
            w[v][0] = q.x, w[v][1] = q.y, w[v][2] = q.z, w[v][3] = q.w;
            if (s == 0 || s == slots - 1) mask_words<DT>(w[v], s * 16, off, end);
        }
    }
    float m = -kInf;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        nan |= r.x(j) != r.x(j);
        m = fmaxf(m, r.x(j));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    r.m = m;
    if (!g.valid || !(fabsf(m) < kInf) || __any_sync(0xffffffffu, nan)) {
        if (lane == 0) put_token(a, row, -1, __int_as_float(0x7fc00000));
        return true;
    }
    if (g.greedy) {
        int c = INT_MAX;
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (r.x(j) == m) c = min(c, r.column(j));
        c = __reduce_min_sync(0xffffffffu, c);
        if (lane == 0) put_token(a, row, c, 0.0f);
        return true;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) r.w[j] = r.weight(r.x(j));
    if (g.use_k && !r.cut(false, static_cast<float>(g.top_k), 0.0f, 0.0f, keys, bins)) return false;
    if (g.use_p) {
        const float all = r.sum();
        if (!r.cut(true, g.top_p * all, all, R::cut_error(g.top_p) * all, keys, bins)) return false;
    }
    if (g.use_min) {
        // In octaves; the border is good to 2^-21 of the distance and of the logarithm.
        const float z = __log2f(fminf(g.min_p, 1.0f));
        bool open = false;
        const float near = 4e-6f * (1.0f - z);
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const float t = (r.x(j) - m) * r.ch;
            open |= fabsf(t - z) <= near && t != 0.0f;
            if (t < z) r.w[j] = 0.0f;
        }
        if (__any_sync(0xffffffffu, open)) return false;
    }
    const auto over_lanes = [](float s) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
    float sums[V], total = 0.0f;  // of vectors
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += r.w[v * E + e];
        sums[v] = over_lanes(s);
        total += sums[v];
    }
    // Without the maximum's weight a small rest keeps its digits.  (Less than two: there is one such
    // weight, and one vector's sum of 1 or more, which holds it.)
    float rest = total - 1.0f;
    if (total < 2.0f) {
        rest = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (sums[v] >= 1.0f) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) s += r.w[v * E + e] == 1.0f ? 0.0f : r.w[v * E + e];
                rest += over_lanes(s);
            } else {
                rest += sums[v];
            }
        }
    }
    // The vector, the lane and the element at which the running sum passes the target.
    const float u = fminf(fmaxf(g.u, 0.0f), 1.0f);  // (fmaxf: NaN counts as 0)
    const float err = R::draw_error(u) * total;
    float target = u * total;
    float before = 0.0f, run = 0.0f;
    float mine[E];
    int at = -1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (at < 0 && target < run + sums[v]) {
            at = v;
            before = run;
#pragma unroll
            for (int e = 0; e < E; ++e) mine[e] = r.w[v * E + e];
        }
        run += sums[v];
    }
    if (at < 0) return false;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += mine[e];
    const float own = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float b = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += b;
    }
    s += before;
    const uint32_t reach = __ballot_sync(0xffffffffu, target < s);
    if (reach == 0) return false;
    const int who = __ffs(reach) - 1;
    run = s - own;
    int e_at = -1;
    float lower = 0.0f, upper = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float n = run + mine[e];
        if (e_at < 0 && target < n) e_at = e, lower = run, upper = n;
        run = n;
    }
    e_at = __shfl_sync(0xffffffffu, e_at, who);
    lower = __shfl_sync(0xffffffffu, lower, who);
    upper = __shfl_sync(0xffffffffu, upper, who);
    if (e_at < 0 || target - lower <= err || upper - target <= err) return false;
    if (lane == who) {
        const int c = (at * 32 + lane) * E + e_at - r.col0;
        // x from its weight's own element: the registers are indexed by constants only
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (j == at * E + e_at) v = r.x(j);
        put_token(a, row, c, (v - m) / g.temperature - log1pf(rest));
    }
    return true;
}

// (Not inlined: one row in a thousand comes here, and its registers are not the others'.)
template <int DT> __device__ __noinline__ void sample_long_way(SampleShared<32>& sh, const uint32_t* powers, unsigned char* dynamic, SampleArgs a, int64_t row) {
    sample_row<DT, 32>(sh, powers, dynamic, a, row);
}

template <int DT, int V> __global__ void __launch_bounds__(32 * kShortWarps, V <= 4 ? 6 : 3) sample_short_kernel(SampleArgs a) {
    __shared__ ShortShared<DT> sh[kShortWarps];
    __shared__ uint32_t powers[64];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < 64; i += 32 * kShortWarps) powers[i] = kPowers[i];
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kShortWarps + warp;
    if (row >= a.B) return;
    if (sample_short<DT, V>(a, row, lane, sh[warp].keys, sh[warp].row.bins)) return;
    sample_long_way<DT>(sh[warp].row, powers, reinterpret_cast<unsigned char*>(sh[warp].dynamic), a, row);
}

template <int DT, int V> cudaError_t launch_sample_short(SampleArgs a, cudaStream_t s) {
    plan_chunks(&a, DType<DT>::bytes, 1);
    return launch_pdl(sample_short_kernel<DT, V>, dim3(static_cast<unsigned>((a.B + kShortWarps - 1) / kShortWarps)),
                      dim3(32 * kShortWarps), s, a);
}

template <int DT> cudaError_t launch_sample(SampleArgs a, int sms, cudaStream_t s) {
    const int64_t slots = (a.N * DType<DT>::bytes + 15) / 16 + 1;
    a.bits = 62;
    for (int64_t n = a.N; n > 1; n = (n + 1) / 2) --a.bits;
    if (a.bits > 44) a.bits = 44;
    if (slots <= 32) return launch_sample_short<DT, 1>(a, s);
    if (slots <= 64) return launch_sample_short<DT, 2>(a, s);
    if (slots <= 96) return launch_sample_short<DT, 3>(a, s);
    if (slots <= 128) return launch_sample_short<DT, 4>(a, s);
    if (slots <= 256) return launch_sample_short<DT, 8>(a, s);
    if (slots <= 2048) return launch_sample_rows<DT, 128>(a, s);
    if (a.B >= 4 * sms || slots <= 4096) return launch_sample_rows<DT, 256>(a, s);
    return launch_sample_rows<DT, 512>(a, s);
}

}  // namespace
}  // namespace lse
