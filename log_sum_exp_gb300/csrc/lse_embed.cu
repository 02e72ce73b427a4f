// lse_embed.cu -- embedding rows for given tokens, and the table's gradient
// (sm_103a).
//
//     out[t, :]    = scale * table[ids[t], :]
//     dtable[v, :] = scale * sum_{t : ids[t] = v} grad[t, :]
//
// The gradient sorts the tokens by id, stably (least significant digit first), so
// that each table row's sum runs over its tokens in their order.  The sorted tokens
// are cut into tiles of equal length, whatever their ids, so a frequent token's rows
// are summed by many CTAs at once: a run of one id inside a tile is summed and written
// by it, a run that crosses tiles leaves one partial sum per tile, which a second
// kernel adds up in order.  Nothing is added through floating-point atomics: a repeated
// call gives equal bits (tile lengths follow the sizes and the alignment).  Up to a few
// thousand tokens are put in order by counting instead.  Rows are zeroed by further CTAs
// of all these kernels: of the sort's first ones (and of the counting) whether they have
// tokens or not, later by a bitmap of the ids that occur.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda_runtime.h>

#include "lse_device.cuh"
#include "lse_elem.cuh"
#include "lse_internal.h"

namespace lse {
namespace {

constexpr int kEmbedThreads = 256;

// The 4 or 8 elements of a 16-byte vector as f32 and back.
template <int DT>
__device__ __forceinline__ void unpack_vector(uint4 v, float (&x)[16 / DType<DT>::bytes]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = word_lo<DT>(w[i]);
            x[2 * i + 1] = word_hi<DT>(w[i]);
        }
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack_vector(const float (&x)[16 / DType<DT>::bytes]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == kF32) w[i] = __float_as_uint(x[i]);
        else w[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A slot is what a thread moves at a time: SB = 16 bytes where every row of both sides
// starts on a 16-byte boundary and is a whole number of vectors, 4 bytes where two
// 16-bit elements can go together, or an element.  Small slots make up with more of
// them in flight.
template <int DT, int SB> struct Slot {
    static constexpr int elems = SB / DType<DT>::bytes;
    static constexpr int in_flight = SB == 16 ? 8 : SB == 4 ? 16 : 24;
    using Raw = typename std::conditional<SB == 16, uint4, uint32_t>::type;
    static __device__ __forceinline__ Raw load(const char* p) {
        if constexpr (SB == 16) return ldg_stream16(p);
        else if constexpr (SB == 4) return __ldg(reinterpret_cast<const uint32_t*>(p));
        else return __ldg(reinterpret_cast<const unsigned short*>(p));
    }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[elems]) {
        if constexpr (SB == 16) {
            unpack_vector<DT>(r, x);
        } else if constexpr (DT == kF32) {
            x[0] = __uint_as_float(r);
        } else {
            x[0] = word_lo<DT>(r);
            if constexpr (SB == 4) x[1] = word_hi<DT>(r);
        }
    }
    static __device__ __forceinline__ void store(char* p, const float (&x)[elems]) {
        if constexpr (SB == 16) *reinterpret_cast<uint4*>(p) = pack_vector<DT>(x);
        else if constexpr (DT == kF32) *reinterpret_cast<float*>(p) = x[0];
        else if constexpr (SB == 4) *reinterpret_cast<uint32_t*>(p) = pack2<DT>(x[0], x[1]);
        else *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(pack2<DT>(x[0], 0.0f));
    }
};

// ---------------------------------------------------------------------------
// Lookup: a warp, or a part of one, per token and segment of its row.
// ---------------------------------------------------------------------------
struct EmbedArgs {
    const char* table;
    int64_t V, D, table_stride;
    const int64_t* ids;
    int64_t T;
    float scale;
    char* out;
    int64_t out_stride;
    int64_t segments;  // per row, of G * U slots
};

// G lanes per row, U slots per lane.  Bound by the rows' bytes when they are many: 20000 rows of 1001 f32 (no
// 16-byte alignment, so 4-byte slots, 16 in flight) in 20.8 us, 7.7 TB/s with what repeats
// coming from L2; 64 rows of 2048 bf16 in 2.3 us, a launch and two dependent loads.
// Few lanes for a short row keep more rows in flight: 65536 rows of 64 bf16 in 3.9 us,
// 14.6 with a warp each.
template <int DT, int SB, int U, int G>
__global__ void __launch_bounds__(kEmbedThreads)
embed_kernel(const __grid_constant__ EmbedArgs a) {
    using S = Slot<DT, SB>;
    constexpr int EB = DType<DT>::bytes;
    const int lane = threadIdx.x & (G - 1);
    const int64_t slots = a.D / S::elems;
    pdl_trigger();
    pdl_wait();
    const int64_t units = a.T * a.segments;
    for (int64_t unit = (static_cast<int64_t>(blockIdx.x) * kEmbedThreads + threadIdx.x) / G; unit < units;
         unit += static_cast<int64_t>(gridDim.x) * (kEmbedThreads / G)) {
        const int64_t t = unit / a.segments;
        const int64_t k0 = (unit - t * a.segments) * (G * U) + lane;
        const int64_t id = __ldg(a.ids + t);
        const bool in = id >= 0 && id < a.V;
        const char* from = a.table + (in ? id : 0) * a.table_stride * EB;
        char* to = a.out + t * a.out_stride * EB;
        typename S::Raw v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (in && k0 + G * j < slots) v[j] = S::load(from + (k0 + G * j) * SB);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + G * j >= slots) continue;
            float x[S::elems];
            if (in) S::unpack(v[j], x);
#pragma unroll
            for (int i = 0; i < S::elems; ++i) x[i] = in ? x[i] * a.scale : __int_as_float(0x7fc00000);
            S::store(to + (k0 + G * j) * SB, x);
        }
    }
}

// ---------------------------------------------------------------------------
// Zeroing table rows without a token.  These CTAs ride along with kernels that leave the
// memory idle: the sorting passes (a few CTAs, bound by latency), the sums, the joins.
// The whole CTA takes row after row where a row gives each thread a vector at least
// (gradient of 32768 tokens in 128256 rows of 4 KB: 119 us, 125 with a warp per row);
// a warp takes a shorter one (20000 tokens in 300000 rows of 200 bytes: 53 against 220,
// 65536 tokens in 50000 rows of 1800 bytes: 89 against 104).
// ---------------------------------------------------------------------------
struct ZeroRows {
    char* table;
    int64_t row_bytes, stride_bytes, rows;
    const uint32_t* bitmap;  // null: no row has a token
    int64_t first;           // group of rows of this launch's first CTA
    int64_t groups;          // CTAs of this launch
    int group_rows;          // 8, 16 or 32 (rows of one word of the bitmap)
    int eb;                  // bytes of an element, 4 or 2
    int64_t vectors;         // of a long row, if all rows are whole, aligned 16-byte vectors; else 0
};

__device__ __forceinline__ void put_zero(char* p, int eb) {
    if (eb == 4) *reinterpret_cast<uint32_t*>(p) = 0u;
    else *reinterpret_cast<unsigned short*>(p) = 0;
}

__device__ __forceinline__ void zero_rows(const ZeroRows& z, int64_t cta, int tid, int threads) {
    const int64_t v0 = (z.first + cta) * z.group_rows;
    const uint32_t present = z.bitmap ? z.bitmap[v0 >> 5] >> (v0 & 31) : 0u;
    if (z.vectors > 0) {
        for (int q = 0; q < z.group_rows; ++q) {
            if (v0 + q >= z.rows) return;
            if ((present >> q) & 1u) continue;
            uint4* row = reinterpret_cast<uint4*>(z.table + (v0 + q) * z.stride_bytes);
            for (int64_t k = tid; k < z.vectors; k += threads) __stcs(row + k, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int lane = tid & 31;
    for (int q = tid >> 5; q < z.group_rows; q += threads >> 5) {
        const int64_t v = v0 + q;
        if (v >= z.rows) return;
        if ((present >> q) & 1u) continue;
        char* row = z.table + v * z.stride_bytes;
        // Elements up to a 16-byte boundary, vectors, elements.
        int64_t head = (16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(row) & 15u)) & 15;
        if (head > z.row_bytes) head = z.row_bytes;
        const int64_t vectors = (z.row_bytes - head) >> 4;
        const int64_t tail = z.row_bytes - head - vectors * 16;
#pragma unroll 4
        for (int64_t k = lane; k < vectors; k += 32) __stcs(reinterpret_cast<uint4*>(row + head) + k, make_uint4(0, 0, 0, 0));
        if (head + tail == 0) continue;
        const int64_t b = static_cast<int64_t>(lane) * z.eb;  // one element per lane at either end
        if (b < head) put_zero(row + b, z.eb);
        if (b < tail) put_zero(row + head + vectors * 16 + b, z.eb);
    }
}

// ---------------------------------------------------------------------------
// Sorting the tokens by id.  A block takes per_block tokens; a digit's counts per
// block give every block its places, and a token's place follows from the tokens of
// its digit before it: in earlier blocks, earlier warps of the block, earlier in the
// warp.  The pass that moves the tokens also counts the next digit, for the blocks
// that they arrive in.  Latency (counts, barriers, a trip to memory
// each way), so rows are zeroed meanwhile: 32768 tokens, two digits, and 16, 56 and 56 MB
// of zeros take 6, 16 and 12 us.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortPer = 4;                            // tokens per thread and round
constexpr int kSortRound = kSortThreads * kSortPer;    // tokens of a round
constexpr int kSortMaxBits = 10;
constexpr int kSortMaxBlocks = 256;

struct SortArgs {
    const int64_t* ids;
    int T;
    int64_t V, padding;
    int block_shift;           // log2 of the tokens per block
    int shift, bits;           // this pass's digit
    int next_bits;             // 0: the last pass
    const uint32_t* key_in;    // (passes after the first)
    const uint32_t* at_in;
    uint32_t* key_out;
    uint32_t* at_out;
    uint32_t* counts;          // [blocks][1 << bits]
    uint32_t* next_counts;     // [blocks][1 << next_bits], zero before
    uint32_t* bitmap;          // ids that occur
    int blocks;                // sorting CTAs, before those that zero rows
    ZeroRows zero;
};

// Tokens that add nothing sort last.
__device__ __forceinline__ uint32_t sort_key(int64_t id, int64_t V, int64_t padding) {
    return static_cast<uint32_t>(id >= 0 && id < V && id != padding ? id : V);
}

// The first digit's counts; clears what later passes count into.
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const __grid_constant__ SortArgs a, uint32_t* clear, int64_t clear_words) {
    __shared__ uint32_t count[1 << kSortMaxBits];
    const int bins = 1 << a.bits;
    pdl_trigger();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= a.blocks) {
        zero_rows(a.zero, blockIdx.x - a.blocks, threadIdx.x, kSortThreads);
        return;
    }
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; i < clear_words;
         i += static_cast<int64_t>(a.blocks) * kSortThreads)
        clear[i] = 0;
    for (int i = threadIdx.x; i < bins; i += kSortThreads) count[i] = 0;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) << a.block_shift;
    const int64_t past = first + (1LL << a.block_shift) < a.T ? first + (1LL << a.block_shift) : a.T;
    for (int64_t i = first + threadIdx.x; i < past; i += kSortThreads)
        atomicAdd(&count[sort_key(__ldg(a.ids + i), a.V, a.padding) & (bins - 1)], 1u);
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kSortThreads)
        a.counts[static_cast<int64_t>(blockIdx.x) * bins + i] = count[i];
}

template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
sort_move_kernel(const __grid_constant__ SortArgs a) {
    __shared__ uint32_t place[1 << kSortMaxBits];               // next place of each digit
    __shared__ uint32_t by_warp[kSortWarps][1 << kSortMaxBits];
    __shared__ uint32_t warp_sum[kSortWarps];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int bins = 1 << a.bits, mask = bins - 1;
    pdl_trigger();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= a.blocks) {
        zero_rows(a.zero, blockIdx.x - a.blocks, tid, kSortThreads);
        return;
    }

    // place[d] = the tokens of lower digits, and of this digit in earlier blocks.
    for (int d = tid; d < bins; d += kSortThreads) {
        uint32_t before = 0, all = 0;
        for (int b0 = 0; b0 < a.blocks; b0 += 16) {  // (16 loads in flight)
            uint32_t c[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                c[i] = b0 + i < a.blocks ? a.counts[static_cast<int64_t>(b0 + i) * bins + d] : 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (b0 + i < static_cast<int>(blockIdx.x)) before += c[i];
                all += c[i];
            }
        }
        place[d] = before;
        by_warp[0][d] = all;
    }
    __syncthreads();
    {
        const int per = (bins + kSortThreads - 1) / kSortThreads;  // consecutive digits per thread
        uint32_t mine = 0;
        for (int i = 0; i < per; ++i)
            if (tid * per + i < bins) mine += by_warp[0][tid * per + i];
        uint32_t sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) warp_sum[wid] = sum;
        __syncthreads();
        uint32_t run = sum - mine;
        for (int w = 0; w < wid; ++w) run += warp_sum[w];
        for (int i = 0; i < per; ++i)
            if (tid * per + i < bins) {
                place[tid * per + i] += run;
                run += by_warp[0][tid * per + i];
            }
        __syncthreads();
    }

    const int64_t first = static_cast<int64_t>(blockIdx.x) << a.block_shift;
    const int64_t past = first + (1LL << a.block_shift) < a.T ? first + (1LL << a.block_shift) : a.T;
    for (int64_t start = first; start < past; start += kSortRound) {
        for (int i = tid; i < kSortWarps * bins; i += kSortThreads) by_warp[i >> a.bits][i & mask] = 0;
        __syncthreads();
        uint32_t key[kSortPer], from[kSortPer], rank[kSortPer];
        const int64_t at0 = start + wid * (32 * kSortPer) + lane;
#pragma unroll
        for (int j = 0; j < kSortPer; ++j) {
            const int64_t i = at0 + 32 * j;
            key[j] = 0;
            from[j] = static_cast<uint32_t>(i);
            if (i < past) {
                key[j] = FIRST ? sort_key(__ldg(a.ids + i), a.V, a.padding) : a.key_in[i];
                if (!FIRST) from[j] = a.at_in[i];
            }
        }
#pragma unroll
        for (int j = 0; j < kSortPer; ++j) {
            const bool live = at0 + 32 * j < past;
            const uint32_t d = live ? (key[j] >> a.shift) & mask : 0xffffffffu;
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            uint32_t before = 0;
            if (live) before = by_warp[wid][d];
            __syncwarp();
            if (live && lane == __ffs(same) - 1) by_warp[wid][d] = before + __popc(same);
            __syncwarp();
            rank[j] = before + __popc(same & ((1u << lane) - 1));
        }
        __syncthreads();
        for (int d = tid; d < bins; d += kSortThreads) {
            uint32_t run = place[d];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = by_warp[w][d];
                by_warp[w][d] = run;
                run += c;
            }
            place[d] = run;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortPer; ++j) {
            const int64_t i = at0 + 32 * j;
            if (i >= past) continue;
            const uint32_t to = by_warp[wid][(key[j] >> a.shift) & mask] + rank[j];
            a.key_out[to] = key[j];
            a.at_out[to] = from[j];
            if (a.next_bits > 0)
                atomicAdd(&a.next_counts[((to >> a.block_shift) << a.next_bits) +
                                         ((key[j] >> (a.shift + a.bits)) & ((1u << a.next_bits) - 1))], 1u);
            if (FIRST && key[j] < a.V) {
                // (looked at first, in L1: the bits of frequent ids share few words; a stale
                // look costs one more atomic)
                uint32_t* const word = &a.bitmap[key[j] >> 5];
                const uint32_t bit = 1u << (key[j] & 31);
                if ((__ldca(word) & bit) == 0) atomicOr(word, bit);
            }
        }
        __syncthreads();
    }
}

// Up to kRankMaxTokens tokens: each one's place is the number of smaller keys, and of
// equal ones before it, counted by eight lanes over all keys in shared memory (T^2 / 8
// steps, on all SMs at once).  One launch instead of three (whole gradient, us against
// those of the sorting passes: 4 tokens in 32000 rows of 1024 bf16 12.4 and 16.5; 300 in
// 20000 of 512 13.2 and 21.8; 4000 24.5 and 28.3; 6000 30.1 and 29.2).
constexpr int kRankMaxTokens = 4096;
constexpr int kRankLanes = 8;
constexpr int kRankTokens = kSortThreads / kRankLanes;  // of a CTA

__global__ void __launch_bounds__(kSortThreads)
sort_rank_kernel(const __grid_constant__ SortArgs a, uint32_t* cross_count) {
    __shared__ uint4 keys4[kRankMaxTokens / 4];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= a.blocks) {
        zero_rows(a.zero, blockIdx.x - a.blocks, tid, kSortThreads);
        return;
    }
    uint32_t* const keys = reinterpret_cast<uint32_t*>(keys4);
    if (blockIdx.x == 0 && tid < 2) cross_count[tid] = 0;
    const int padded = (a.T + kRankTokens - 1) / kRankTokens * kRankTokens;
#pragma unroll 8
    for (int i = tid; i < padded; i += kSortThreads)
        keys[i] = i < a.T ? sort_key(__ldg(a.ids + i), a.V, a.padding) : 0xffffffffu;  // (below no key)
    __syncthreads();
    const int t0 = blockIdx.x * kRankTokens, lane = tid % kRankLanes;
    const int i = t0 + tid / kRankLanes;
    const uint32_t key = keys[i];
    uint32_t place = 0;
    // Before the CTA's tokens equal keys count, after them they do not; among them by number.
#pragma unroll 4
    for (int j = lane; j < t0 / 4; j += kRankLanes) {
        const uint4 k = keys4[j];
        place += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
    }
#pragma unroll 4
    for (int j = t0 / 4 + lane; j < padded / 4; j += kRankLanes) {
        const uint4 k = keys4[j];
        place += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
    }
    for (int j = t0 + lane; j < i; j += kRankLanes) place += keys[j] == key;
#pragma unroll
    for (int off = 1; off < kRankLanes; off <<= 1) place += __shfl_xor_sync(0xffffffffu, place, off);
    if (lane == 0 && i < a.T) {
        a.key_out[place] = key;
        a.at_out[place] = static_cast<uint32_t>(i);
    }
}

// ---------------------------------------------------------------------------
// Sums over the sorted tokens.
// ---------------------------------------------------------------------------
constexpr int kLongRun = 7;  // further tiles of a run that counts as long
// Bytes zeroed next to the counting, to each sorting pass and to the joins: about what
// the memory takes while these wait for their own few loads (32768 tokens, 2048 columns:
// 136 us with 4, 24 and 24 MB, 130 with 8, 40 and 40, 127 with these).  Measured at that
// size alone; the waits of other sizes are longer or shorter, and the bytes do not follow.
constexpr int64_t kCountZeroBytes = 16 << 20;
constexpr int64_t kSortZeroBytes = 56 << 20;
// The ranking kernel zeroes all rows alone, without the overlap with the joins: it is
// taken while there are no more bytes than the sorting passes would zero.
constexpr int64_t kRankZeroBytes = kCountZeroBytes + 2 * kSortZeroBytes;
constexpr int64_t kJoinCtas = 608;  // four for each of the 152 SMs
constexpr int64_t kJoinZeroBytes = 40 << 20;
constexpr int64_t kSumCtas = 256;

struct SumArgs {
    const char* grad;
    int64_t D, grad_stride;
    const uint32_t* key;     // sorted ids; V for tokens that add nothing
    const uint32_t* at;
    int T;
    int64_t V;
    float scale;
    char* dtable;
    int64_t dtable_stride;
    bool accumulate;
    uint32_t* cross;         // [tiles]: those whose last run goes on, in any order
    uint32_t* cross_count;   // of long runs, and of others
    float* head;             // [tiles][D]: the sum of a tile's first run, when the run began before
    float* tail;             // [tiles][D]: of its last run, when that begins here and goes on
    int tile_len;            // sorted tokens of a tile
    int tiles;
    int64_t slots;           // per row: 16-byte vectors or elements of grad
    int64_t col_blocks;      // of blockDim.x slots
    int64_t sum_ctas;        // CTAs before those that zero rows
    ZeroRows zero;
};

// A slot's sums, and the same while they are added up (two at a time, packed FP32).
template <int E> struct Sums {
    float v[E];
};
template <int E> struct Total {
    uint64_t pair[E / 2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) pair[i] = 0ull;
    }
    __device__ __forceinline__ void add(const float (&y)[E]) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) pair[i] = f2_add(pair[i], f2_pack(y[2 * i], y[2 * i + 1]));
    }
    __device__ __forceinline__ Sums<E> sums() const {
        Sums<E> s;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) f2_unpack(pair[i], s.v[2 * i], s.v[2 * i + 1]);
        return s;
    }
};
template <> struct Total<1> {
    float v;
    __device__ __forceinline__ void clear() { v = 0.0f; }
    __device__ __forceinline__ void add(const float (&y)[1]) { v += y[0]; }
    __device__ __forceinline__ Sums<1> sums() const { return Sums<1>{{v}}; }
};

// dtable's slot of row v: scale * sum, plus what was there.
template <int DT, int OT, int SB>
__device__ __forceinline__ void put_slot(const SumArgs& a, uint32_t v, int64_t slot, const Sums<Slot<DT, SB>::elems>& s) {
    constexpr int E = Slot<DT, SB>::elems, OB = DType<OT>::bytes;
    // dtable's share of the slot in pieces of at most 16 bytes, of the same alignment.
    constexpr int PB = OT == DT ? SB : (SB == 16 ? 16 : 4), PE = PB / OB;
    using P = Slot<OT, PB>;
    char* to = a.dtable + static_cast<int64_t>(v) * a.dtable_stride * OB + slot * (E * OB);
#pragma unroll
    for (int q = 0; q < E / PE; ++q, to += PB) {
        float x[PE];
        if (a.accumulate) {
            typename P::Raw old;  // (a plain load: the row is written here)
            if constexpr (PB == 2) old = *reinterpret_cast<const unsigned short*>(to);
            else old = *reinterpret_cast<const typename P::Raw*>(to);
            P::unpack(old, x);
        }
#pragma unroll
        for (int i = 0; i < PE; ++i) x[i] = a.accumulate ? fmaf(s.v[q * PE + i], a.scale, x[i]) : s.v[q * PE + i] * a.scale;
        P::store(to, x);
    }
}

template <int E>
__device__ __forceinline__ void put_partial(float* to, const SumArgs& a, int tile, int64_t slot, const Sums<E>& s) {
    float* p = to + static_cast<int64_t>(tile) * a.D + slot * E;
#pragma unroll
    for (int i = 0; i < E; i += E >= 4 ? 4 : 1) {
        if constexpr (E >= 4) *reinterpret_cast<float4*>(p + i) = make_float4(s.v[i], s.v[i + 1], s.v[i + 2], s.v[i + 3]);
        else p[i] = s.v[i];
    }
}

// The end of a run in a tile.  (Inlined at every step of the unrolled sum: as a called
// function it measured 160 against 140 us for 32768 tokens of 2048 columns.)
template <int DT, int OT, int SB>
__device__ __forceinline__ void end_run(const SumArgs& a, uint32_t run, bool began_before, bool goes_on, int tile,
                                     int64_t slot, Sums<Slot<DT, SB>::elems> s) {
    if (began_before) put_partial(a.head, a, tile, slot, s);
    else if (goes_on) put_partial(a.tail, a, tile, slot, s);
    else put_slot<DT, OT, SB>(a, run, slot, s);
}

// blockDim = (slots of a column block, tiles of a CTA).
//
// Bound by memory: 32768 tokens of 2048 bf16 read, their rows written and what is
// left of 128256 zeroed in 69 us, 6.5 TB/s.  A thread owns a column slot of a tile and walks down
// its tokens, U rows in flight; whether a token starts a run is found out once per tile
// and not by every thread, and a batch without a start is added without looking (122 to
// 119 us for the whole gradient).  A second batch in flight meanwhile spills in the loop
// (123); as it is 16-bit rows spill 56 bytes, at the ends of runs (0.8 % of the
// instructions executed are to local memory).
// A tile's tokens in whole batches of U.
__host__ __device__ constexpr int sum_padded(int len, int U) { return (len + U - 1) / U * U; }

template <int DT, int OT, int SB>
__global__ void __launch_bounds__(kEmbedThreads, 4)
embed_sum_kernel(const __grid_constant__ SumArgs a) {
    using S = Slot<DT, SB>;
    constexpr int E = S::elems, U = S::in_flight;
    extern __shared__ uint4 sm[];
    const int tx = threadIdx.x, ty = threadIdx.y, TX = blockDim.x, TY = blockDim.y;
    pdl_trigger();
    pdl_wait();

    if (blockIdx.x >= a.sum_ctas) {
        zero_rows(a.zero, blockIdx.x - a.sum_ctas, ty * TX + tx, TX * TY);
        return;
    }

    const int64_t group = blockIdx.x / a.col_blocks;
    const int64_t slot = (blockIdx.x - group * a.col_blocks) * TX + tx;
    const int64_t tile0 = group * TY;
    // Of each tile: its keys with one neighbour on either side, where the rows of grad are,
    // and (a byte each) whether a token's key differs from the one before it.  In whole
    // batches of U: what is past the tile is a row that may be read.
    const int len = a.tile_len, padded = sum_padded(len, U);
    uint64_t* const from = reinterpret_cast<uint64_t*>(sm) + ty * padded;
    unsigned char* const starts = reinterpret_cast<unsigned char*>(reinterpret_cast<uint64_t*>(sm) + TY * padded) + ty * padded;
    uint32_t* const key = reinterpret_cast<uint32_t*>(reinterpret_cast<unsigned char*>(sm) + TY * padded * 9) + ty * (len + 2);
    const int64_t i0 = (tile0 + ty) * len;
    const uint64_t row_bytes = static_cast<uint64_t>(a.grad_stride) * DType<DT>::bytes;
    for (int e = tx; e < padded; e += TX) {
        const int64_t i = i0 + e;
        const bool in = e < len && i < a.T;
        from[e] = in ? a.at[i] * row_bytes : 0ull;
        starts[e] = in && e > 0 && a.key[i] != a.key[i - 1] ? 1 : 0;
    }
    for (int e = tx; e < len + 2; e += TX) {
        const int64_t i = i0 + e - 1;
        key[e] = i >= 0 && i < a.T ? a.key[i] : 0xffffffffu;  // (no id)
    }
    __syncthreads();
    if (tile0 + ty >= a.tiles || slot >= a.slots) return;
    const int tile = static_cast<int>(tile0 + ty);
    const char* col = a.grad + slot * SB;

    // (tokens that add nothing sort last)
    int n = a.T - i0 < len ? static_cast<int>(a.T - i0) : len;
    while (n > 0 && key[n] >= a.V) --n;
    if (n == 0) return;
    Total<E> s;
    s.clear();
    uint32_t run = key[1];
    bool began_before = key[0] == run;
    for (int e0 = 0; e0 < n; e0 += U) {
        typename S::Raw v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = S::load(col + from[e0 + u]);
        uint64_t start[U / 8], any = 0;
#pragma unroll
        for (int q = 0; q < U / 8; ++q) any |= start[q] = *reinterpret_cast<const uint64_t*>(starts + e0 + 8 * q);
        if (any == 0 && e0 + U <= n) {  // one run all through
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float y[E];
                S::unpack(v[u], y);
                s.add(y);
            }
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (e0 + u >= n) break;
            if ((start[u / 8] >> (8 * (u % 8))) & 0xffu) {
                end_run<DT, OT, SB>(a, run, began_before, false, tile, slot, s.sums());
                s.clear();
                run = key[e0 + u + 1];
                began_before = false;
            }
            float y[E];
            S::unpack(v[u], y);
            s.add(y);
        }
    }
    const bool goes_on = !began_before && key[n + 1] == run;
    end_run<DT, OT, SB>(a, run, began_before, goes_on, tile, slot, s.sums());
    if (goes_on && slot == 0) {  // long runs from the list's front, others from its back
        const int64_t far = i0 + (kLongRun + 1) * len;
        if (far < a.T && a.key[far] == run) a.cross[atomicAdd(a.cross_count, 1u)] = static_cast<uint32_t>(tile);
        else a.cross[a.tiles - 1 - static_cast<int>(atomicAdd(a.cross_count + 1, 1u))] = static_cast<uint32_t>(tile);
    }
}

template <int E>
__device__ __forceinline__ void add_partial(Sums<E>& s, const float* p) {
    if constexpr (E >= 4) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            s.v[i] += v.x;
            s.v[i + 1] += v.y;
            s.v[i + 2] += v.z;
            s.v[i + 3] += v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) s.v[i] += p[i];
    }
}

// The sum of a run that begins in `tile` and goes on up to tile `last`, as far as
// tiles first .. past - 1 (of the later ones) go; with `tail`, the tile's own.
template <int E>
__device__ __forceinline__ void add_run(Sums<E>& s, const SumArgs& a, int64_t slot, int tile, bool tail, int first, int past) {
    if (tail) add_partial<E>(s, a.tail + static_cast<int64_t>(tile) * a.D + slot * E);
#pragma unroll 4
    for (int j = first; j < past; ++j) add_partial<E>(s, a.head + static_cast<int64_t>(j) * a.D + slot * E);
}

// Runs that cross tiles, listed by the tiles where they begin: the tile's own sum and
// the later tiles', in order.  blockDim = (slots of a narrow column block, groups).  For
// a long run the groups take equal parts of the tiles of one narrow block, then their
// sums are added in order; for others each group has a narrow block of its own.  The
// CTAs take (run, column block) pairs in turn; further CTAs zero rows.  Latency: 8 us
// for 32768 tokens (a look at the keys, the longest run's partial sums), next to 40 MB of
// zeros.
template <int DT, int OT, int SB>
__global__ void __launch_bounds__(kEmbedThreads)
embed_join_kernel(const __grid_constant__ SumArgs a) {
    constexpr int E = Slot<DT, SB>::elems;
    __shared__ float part[kEmbedThreads * E];
    const int tx = threadIdx.x, ty = threadIdx.y, TX = blockDim.x, TY = blockDim.y;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x >= a.sum_ctas) {
        zero_rows(a.zero, blockIdx.x - a.sum_ctas, ty * TX + tx, TX * TY);
        return;
    }
    const int t = ty * TX + tx;
    const int64_t wide_blocks = (a.col_blocks + TY - 1) / TY;
    const int64_t longs = static_cast<int64_t>(a.cross_count[0]) * a.col_blocks;
    const int64_t units = longs + static_cast<int64_t>(a.cross_count[1]) * wide_blocks;
    for (int64_t unit = blockIdx.x; unit < units; unit += a.sum_ctas) {
        const bool is_long = unit < longs;
        const int64_t q = is_long ? unit / a.col_blocks : (unit - longs) / wide_blocks;
        const int64_t block = is_long ? unit - q * a.col_blocks : (unit - longs - q * wide_blocks) * TY + ty;
        const int tile = static_cast<int>(a.cross[is_long ? q : a.tiles - 1 - q]);
        const int64_t slot = block * TX + tx;
        const uint32_t run = a.key[static_cast<int64_t>(tile + 1) * a.tile_len];
        // The last tile whose first token is of this run: 32 tiles looked at in one go,
        // then by halves.
        const int look = tile + 2 + (t & 31);
        const bool more = look < a.tiles && a.key[static_cast<int64_t>(look) * a.tile_len] == run;
        const uint32_t ends = ~__ballot_sync(0xffffffffu, more);
        int lo = tile + 1 + (ends == 0 ? 32 : __ffs(ends) - 1);
        if (ends == 0) {
            int hi = a.tiles - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (a.key[static_cast<int64_t>(mid) * a.tile_len] == run) lo = mid;
                else hi = mid - 1;
            }
        }
        Sums<E> s;
#pragma unroll
        for (int i = 0; i < E; ++i) s.v[i] = 0.0f;
        if (!is_long) {
            if (slot < a.slots) {
                add_run<E>(s, a, slot, tile, true, tile + 1, lo + 1);
                put_slot<DT, OT, SB>(a, run, slot, s);
            }
            continue;
        }
        const int each = (lo - tile + TY - 1) / TY;  // of tiles tile + 1 .. lo
        const int j0 = tile + 1 + ty * each;
        const int j1 = j0 + each < lo + 1 ? j0 + each : lo + 1;
        if (slot < a.slots) add_run<E>(s, a, slot, tile, ty == 0, j0, j1);
#pragma unroll
        for (int i = 0; i < E; ++i) part[i * (TX * TY) + t] = s.v[i];
        __syncthreads();
        if (ty == 0 && slot < a.slots) {
            for (int y = 1; y < TY && tile + 1 + y * each <= lo; ++y) {
#pragma unroll
                for (int i = 0; i < E; ++i) s.v[i] += part[i * (TX * TY) + y * TX + tx];
            }
            put_slot<DT, OT, SB>(a, run, slot, s);
        }
        __syncthreads();
    }
}

bool rows_ok(int64_t rows, int64_t D, int64_t stride, int64_t eb) {
    int64_t extent = 0;
    if (rows < 0 || D < 0 || stride < D) return false;
    if (rows > 0 && __builtin_mul_overflow(rows - 1, stride, &extent)) return false;
    return !__builtin_add_overflow(extent, D, &extent) && !__builtin_mul_overflow(extent, eb, &extent);
}

unsigned capped(int64_t n, int64_t most) { return static_cast<unsigned>(n < 1 ? 1 : n < most ? n : most); }

// The slot that rows of D elements on both sides allow.
template <int DT>
int slot_bytes(const void* p, int64_t stride, const void* q, int64_t stride_q, int64_t eb_q, int64_t D) {
    constexpr int64_t eb = DType<DT>::bytes;
    const auto fits = [&](int64_t sb) {
        return reinterpret_cast<uintptr_t>(p) % sb == 0 && stride * eb % sb == 0 && D * eb % sb == 0 &&
               reinterpret_cast<uintptr_t>(q) % sb == 0 && stride_q * eb_q % sb == 0;
    };
    return fits(16) ? 16 : fits(4) ? 4 : static_cast<int>(eb);
}

template <int DT, int SB, int U, int G>
cudaError_t launch_embed_g(EmbedArgs a, cudaStream_t stream) {
    const int64_t slots = a.D / Slot<DT, SB>::elems;
    a.segments = (slots + G * U - 1) / (G * U);
    const int64_t rows = kEmbedThreads / G;
    const int64_t ctas = (a.T * a.segments + rows - 1) / rows;
    return launch_pdl(embed_kernel<DT, SB, U, G>, dim3(capped(ctas, INT_MAX)), dim3(kEmbedThreads), stream, a);
}

// The fewest lanes (4 to 32) that hold a row.
template <int DT, int SB, int U>
cudaError_t launch_embed_u(const EmbedArgs& a, cudaStream_t stream) {
    const int64_t slots = a.D / Slot<DT, SB>::elems;
    return slots <= 4 * U    ? launch_embed_g<DT, SB, U, 4>(a, stream)
           : slots <= 8 * U  ? launch_embed_g<DT, SB, U, 8>(a, stream)
           : slots <= 16 * U ? launch_embed_g<DT, SB, U, 16>(a, stream)
                             : launch_embed_g<DT, SB, U, 32>(a, stream);
}

// One slot per lane for small calls, where latency counts; else about 64 bytes of each
// row in flight per lane.
template <int DT, int SB>
cudaError_t launch_embed_sb(const EmbedArgs& a, cudaStream_t stream) {
    const bool small = a.T * (a.D / Slot<DT, SB>::elems) <= 1 << 17;
    return small ? launch_embed_u<DT, SB, 1>(a, stream) : launch_embed_u<DT, SB, SB == 16 ? 4 : 16>(a, stream);
}

template <int DT>
cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t stream) {
    const int sb = slot_bytes<DT>(a.table, a.table_stride, a.out, a.out_stride, DType<DT>::bytes, a.D);
    if (sb == 16) return launch_embed_sb<DT, 16>(a, stream);
    if (DT == kF32 || sb == 4) return launch_embed_sb<DT, 4>(a, stream);
    return launch_embed_sb<DT, DType<DT>::bytes>(a, stream);
}

template <int DT, int OT, int SB>
cudaError_t launch_sums(SumArgs a, cudaStream_t stream) {
    a.slots = a.D / Slot<DT, SB>::elems;
    const bool join = a.tiles > 1;
    // The rest of the rows to zero: a part for the joining kernel, if there is
    // one, for which it would take about as long as its longest run.
    ZeroRows rest = a.zero;
    const int64_t late = kJoinZeroBytes / (a.zero.row_bytes * a.zero.group_rows);
    a.zero.groups = join ? rest.groups - (rest.groups < late ? rest.groups : late) : rest.groups;
    int TX = 8;
    while (TX < kEmbedThreads && TX < a.slots) TX *= 2;
    const int TY = kEmbedThreads / TX;
    a.col_blocks = (a.slots + TX - 1) / TX;
    a.sum_ctas = (a.tiles + TY - 1) / TY * a.col_blocks;
    const int64_t ctas = a.sum_ctas + a.zero.groups;
    if (ctas > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (ctas > 0)
        e = launch_pdl_smem(embed_sum_kernel<DT, OT, SB>, dim3(static_cast<unsigned>(ctas)), dim3(TX, TY),
                            TY * (9 * sum_padded(a.tile_len, Slot<DT, SB>::in_flight) + 4 * (a.tile_len + 2)), stream, a);
    if (e != cudaSuccess || !join) return e;
    // Narrow column blocks, so that several groups of threads share a long run.
    const int JX = TX < 32 ? TX : 32;
    a.zero.first = rest.first + a.zero.groups;
    a.zero.groups = rest.groups - a.zero.groups;
    a.col_blocks = (a.slots + JX - 1) / JX;
    a.sum_ctas = (a.tiles - 1) * a.col_blocks < kJoinCtas ? (a.tiles - 1) * a.col_blocks : kJoinCtas;
    if (a.sum_ctas + a.zero.groups > INT_MAX) return cudaErrorInvalidValue;
    return launch_pdl(embed_join_kernel<DT, OT, SB>, dim3(static_cast<unsigned>(a.sum_ctas + a.zero.groups)),
                      dim3(JX, kEmbedThreads / JX), stream, a);
}

template <int DT>
int sum_slot_bytes(const SumArgs& a, int64_t ob) {
    return slot_bytes<DT>(a.grad, a.grad_stride, a.dtable, a.dtable_stride, ob, a.D);
}

template <int DT, int OT>
cudaError_t launch_sums_slot(const SumArgs& a, cudaStream_t stream) {
    const int sb = sum_slot_bytes<DT>(a, DType<OT>::bytes);
    if (sb == 16) return launch_sums<DT, OT, 16>(a, stream);
    if (DT == kF32 || sb == 4) return launch_sums<DT, OT, 4>(a, stream);
    return launch_sums<DT, OT, DType<DT>::bytes>(a, stream);
}

template <int DT>
cudaError_t launch_sums_dt(const SumArgs& a, int out_dtype, cudaStream_t stream) {
    if (DT == kF32 || out_dtype == LSE_F32) return launch_sums_slot<DT, kF32>(a, stream);
    return launch_sums_slot<DT, DT>(a, stream);
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The next groups of *from, as many as `bytes` cover, for a kernel to zero.
ZeroRows take_zero_rows(ZeroRows* from, int64_t bytes, const uint32_t* bitmap) {
    ZeroRows z = *from;
    const int64_t groups = bytes / (z.row_bytes * z.group_rows);
    z.groups = groups < z.groups ? groups : z.groups;
    z.bitmap = bitmap;
    from->first += z.groups;
    from->groups -= z.groups;
    return z;
}

lse_status embed_backward(SumArgs a, lse_dtype dtype, lse_dtype out_dtype, const int64_t* ids,
                          int64_t padding, cudaStream_t stream) {
    char* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    const int64_t ob = out_dtype == LSE_F32 ? 4 : 2;
    a.zero.table = a.dtable;
    a.zero.row_bytes = a.D * ob;
    a.zero.stride_bytes = a.dtable_stride * ob;
    a.zero.rows = a.V;
    // (about 16 KB per CTA, or 32 rows: shorter ones would leave the CTA's launch to pay for)
    a.zero.group_rows = a.zero.row_bytes >= 2048 ? 8 : a.zero.row_bytes >= 1024 ? 16 : 32;
    a.zero.groups = a.accumulate ? 0 : (a.V + a.zero.group_rows - 1) / a.zero.group_rows;
    const bool whole = reinterpret_cast<uintptr_t>(a.dtable) % 16 == 0 && a.zero.stride_bytes % 16 == 0 && a.zero.row_bytes % 16 == 0;
    a.zero.vectors = whole && a.zero.row_bytes >= 16 * kEmbedThreads ? a.zero.row_bytes / 16 : 0;
    a.zero.eb = static_cast<int>(ob);
    if (a.T > 0) {
        // Blocks of at least one round of tokens, at most kSortMaxBlocks of them.
        SortArgs s;
        std::memset(&s, 0, sizeof s);
        s.ids = ids;
        s.T = a.T;
        s.V = a.V;
        s.padding = padding;
        s.block_shift = 10;
        static_assert(kSortRound == 1 << 10, "a block holds whole rounds");
        while ((static_cast<int64_t>(a.T) + (1LL << s.block_shift) - 1) >> s.block_shift > kSortMaxBlocks) ++s.block_shift;
        const int blocks = static_cast<int>((static_cast<int64_t>(a.T) + (1LL << s.block_shift) - 1) >> s.block_shift);
        int bits = 1;  // of keys 0 .. V
        while (bits < 31 && (a.V >> bits) != 0) ++bits;
        const bool ranked = a.T <= kRankMaxTokens && a.zero.groups * a.zero.group_rows * a.zero.row_bytes <= kRankZeroBytes;
        const int passes = ranked ? 0 : (bits + kSortMaxBits - 1) / kSortMaxBits;
        const int per = ranked ? 0 : (bits + passes - 1) / passes;

        // Longer tiles leave fewer partial sums, shorter ones more CTAs: the longest of 64
        // that leaves kSumCtas of them (bf16, us, with tiles of 8, 16, 32, 64: 300 tokens of
        // 512 columns 10.9, 12.6, 15.8, 21.6; 8192 of 1024 36.9, 33.1, 35.9, 41.9; 65536 of
        // 896 99, 83, 77, 76; 32768 of 2048 145, 129, 121, 118).
        const int sb = dtype == LSE_F32 ? sum_slot_bytes<kF32>(a, ob) : dtype == LSE_BF16 ? sum_slot_bytes<kBF16>(a, ob) : sum_slot_bytes<kF16>(a, ob);
        const int64_t slots = a.D * (dtype == LSE_F32 ? 4 : 2) / sb;
        a.tile_len = 64;
        while (a.tile_len > (sb == 16 ? 8 : 16) && a.T * slots < kSumCtas * kEmbedThreads * a.tile_len) a.tile_len /= 2;
        const int64_t tiles = (static_cast<int64_t>(a.T) + a.tile_len - 1) / a.tile_len;
        a.tiles = static_cast<int>(tiles);
        const int64_t list = round_up(static_cast<int64_t>(a.T) * 4, 256);
        const int64_t counts = round_up((static_cast<int64_t>(blocks) << per) * 4, 256);
        const int64_t bitmap = ranked ? 0 : round_up((a.V + 31) / 32 * 4, 256);
        const int64_t cross = round_up((tiles + 2) * 4, 256);
        const int64_t partial = round_up(tiles * a.D * 4, 256);
        const lse_status st = take_scratch(reinterpret_cast<void**>(&scratch),
                                           static_cast<size_t>(4 * list + passes * counts + bitmap + cross + 2 * partial), stream);
        if (st != LSE_OK) return st;
        uint32_t* key[2] = {reinterpret_cast<uint32_t*>(scratch), reinterpret_cast<uint32_t*>(scratch + list)};
        uint32_t* at[2] = {reinterpret_cast<uint32_t*>(scratch + 2 * list), reinterpret_cast<uint32_t*>(scratch + 3 * list)};
        char* const count0 = scratch + 4 * list;
        s.bitmap = reinterpret_cast<uint32_t*>(count0 + passes * counts);
        char* const behind = count0 + passes * counts + bitmap;
        a.cross_count = reinterpret_cast<uint32_t*>(behind);
        a.cross = a.cross_count + 2;
        a.head = reinterpret_cast<float*>(behind + cross);
        a.tail = reinterpret_cast<float*>(behind + cross + partial);
        a.zero.bitmap = s.bitmap;
        s.blocks = blocks;

        if (ranked) {
            s.key_out = key[0];
            s.at_out = at[0];
            s.blocks = (a.T + kRankTokens - 1) / kRankTokens;
            s.zero = take_zero_rows(&a.zero, INT64_MAX, nullptr);
            e = launch_pdl(sort_rank_kernel, dim3(static_cast<unsigned>(s.blocks + s.zero.groups)), dim3(kSortThreads),
                           stream, s, a.cross_count);
        } else {
            // Before the bitmap is known, rows are zeroed whether they have tokens or not: the
            // memory would be idle.
            s.bits = per;
            s.counts = reinterpret_cast<uint32_t*>(count0);
            s.zero = take_zero_rows(&a.zero, kCountZeroBytes, nullptr);
            // (behind the first pass's counts: the later passes', the bitmap, the list's lengths)
            e = launch_pdl(sort_count_kernel, dim3(static_cast<unsigned>(blocks + s.zero.groups)), dim3(kSortThreads), stream,
                           s, reinterpret_cast<uint32_t*>(count0 + counts), ((passes - 1) * counts + bitmap) / 4 + 2);
            for (int p = 0; p < passes && e == cudaSuccess; ++p) {
                s.shift = p * per;
                s.next_bits = p + 1 < passes ? per : 0;
                s.counts = reinterpret_cast<uint32_t*>(count0 + p * counts);
                s.next_counts = reinterpret_cast<uint32_t*>(count0 + (p + 1) * counts);
                s.key_in = key[(p + 1) & 1];
                s.at_in = at[(p + 1) & 1];
                s.key_out = key[p & 1];
                s.at_out = at[p & 1];
                s.zero = p == 0 ? take_zero_rows(&a.zero, kSortZeroBytes, nullptr)
                                : take_zero_rows(&a.zero, kSortZeroBytes, s.bitmap);
                const dim3 grid(static_cast<unsigned>(blocks + s.zero.groups));
                e = p == 0 ? launch_pdl(sort_move_kernel<true>, grid, dim3(kSortThreads), stream, s)
                           : launch_pdl(sort_move_kernel<false>, grid, dim3(kSortThreads), stream, s);
            }
        }
        a.key = key[ranked ? 0 : (passes - 1) & 1];
        a.at = at[ranked ? 0 : (passes - 1) & 1];
    }
    if (e == cudaSuccess)
        e = dtype == LSE_F32 ? launch_sums_dt<kF32>(a, out_dtype, stream)
            : dtype == LSE_BF16 ? launch_sums_dt<kBF16>(a, out_dtype, stream)
                                : launch_sums_dt<kF16>(a, out_dtype, stream);
    if (scratch) {
        const cudaError_t ef = cudaFreeAsync(scratch, stream);
        if (e == cudaSuccess) e = ef;
    }
    return cuda_status(e);
}

}  // namespace
}  // namespace lse

using namespace lse;

extern "C" {

lse_status lse_embedding(const void* table, lse_dtype dtype, int64_t V, int64_t D,
                         int64_t table_stride, const int64_t* ids, int64_t T, float scale, void* out,
                         int64_t out_stride, lse_stream_t stream) {
    if (!valid_dtype(dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2;
    if (!rows_ok(V, D, table_stride, eb) || !rows_ok(T, D, out_stride, eb)) return LSE_ERR_INVALID_ARG;
    if (misaligned(table, eb) || misaligned(out, eb) || misaligned(ids, 8)) return LSE_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return LSE_OK;
    if (ids == nullptr || out == nullptr || (V > 0 && table == nullptr)) return LSE_ERR_INVALID_ARG;
    EmbedArgs a{static_cast<const char*>(table), V, D, table_stride, ids, T, scale, static_cast<char*>(out), out_stride, 1};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(dtype == LSE_F32 ? launch_embed<kF32>(a, s)
                       : dtype == LSE_BF16 ? launch_embed<kBF16>(a, s) : launch_embed<kF16>(a, s));
}

lse_status lse_embedding_backward(const void* grad, lse_dtype dtype, int64_t T, int64_t D,
                                  int64_t grad_stride, const int64_t* ids, int64_t V, float scale,
                                  int64_t padding, void* dtable, lse_dtype dtable_dtype,
                                  int64_t dtable_stride, int accumulate, lse_stream_t stream_) {
    if (!valid_dtype(dtype) || !valid_dtype(dtable_dtype)) return LSE_ERR_UNSUPPORTED_DTYPE;
    if (dtable_dtype != dtype && dtable_dtype != LSE_F32) return LSE_ERR_UNSUPPORTED_DTYPE;
    const int64_t eb = dtype == LSE_F32 ? 4 : 2, ob = dtable_dtype == LSE_F32 ? 4 : 2;
    if (!rows_ok(T, D, grad_stride, eb) || !rows_ok(V, D, dtable_stride, ob)) return LSE_ERR_INVALID_ARG;
    if (T > INT32_MAX || V > INT32_MAX) return LSE_ERR_INVALID_ARG;
    if (misaligned(grad, eb) || misaligned(dtable, ob) || misaligned(ids, 8)) return LSE_ERR_INVALID_ARG;
    if (V == 0 || D == 0) return LSE_OK;
    if (dtable == nullptr || (T > 0 && (grad == nullptr || ids == nullptr))) return LSE_ERR_INVALID_ARG;
    SumArgs a;
    std::memset(&a, 0, sizeof a);
    a.grad = static_cast<const char*>(grad);
    a.D = D;
    a.grad_stride = grad_stride;
    a.T = static_cast<int>(T);
    a.V = V;
    a.scale = scale;
    a.dtable = static_cast<char*>(dtable);
    a.dtable_stride = dtable_stride;
    a.accumulate = accumulate != 0;
    return embed_backward(a, dtype, dtable_dtype, ids, padding, reinterpret_cast<cudaStream_t>(stream_));
}

}  // extern "C"
