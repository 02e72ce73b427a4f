// lse_topk.cuh -- ordering keys and warp-wide lists for the largest elements of
// a row (sm_103a).
//
// An element is ranked by a 64-bit key: its value in the high word, mapped so
// that unsigned order is the order of the values, and the complement of its
// column in the low word.  All keys of a row differ, a larger key is a larger
// value or, at equal values, a lower column, and so "the K largest keys" is one
// definite list whatever the order in which they are found.  -0 ranks with +0,
// a NaN of any sign or payload above everything (ties by column again), and key
// 0 is no element.
//
// A list is one key per lane of a warp, sorted in descending order; K <= 32.
#pragma once

#include <cstdint>

#include "lse_device.cuh"

namespace lse {

constexpr int kMaxTopK = 32;

__device__ __forceinline__ uint32_t order_bits(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 -> +0
    return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t topk_key(float x, uint32_t column) {
    return (static_cast<uint64_t>(order_bits(x)) << 32) | (0xffffffffu - column);
}
__device__ __forceinline__ float key_value(uint64_t k) {
    return order_value(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int64_t key_column(uint64_t k) {
    return static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(k));
}

__device__ __forceinline__ uint64_t key_max(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t key_min(uint64_t a, uint64_t b) { return a < b ? a : b; }

// Bitonic merge of 32 keys that rise and then fall (or the reverse).
__device__ __forceinline__ uint64_t list_tidy(uint64_t k, int lane) {
#pragma unroll
    for (int stride = 16; stride > 0; stride >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, k, stride);
        k = (lane & stride) == 0 ? key_max(k, o) : key_min(k, o);
    }
    return k;
}

// Any 32 keys to a list (bitonic sort).
__device__ __forceinline__ uint64_t list_sort(uint64_t k, int lane) {
#pragma unroll
    for (int size = 2; size < 32; size <<= 1) {
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, k, stride);
            k = ((lane & stride) == 0) == ((lane & size) == 0) ? key_max(k, o) : key_min(k, o);
        }
    }
    return list_tidy(k, lane);
}

// The 32 largest keys of two lists: against the second reversed, the larger of
// each pair is among them, and what results rises and falls once.
__device__ __forceinline__ uint64_t list_merge(uint64_t a, uint64_t b, int lane) {
    const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
    return list_tidy(key_max(a, r), lane);
}

}  // namespace lse
