// lse_elem.cuh -- loads and stores of elements that the model operators share (sm_103a).
#pragma once

#include <cstdint>

#include "lse_device.cuh"

namespace lse {

// Two floats -> packed 16-bit pair, nearest-even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (DT == kBF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ldg_stream16 and load_elem for what the kernel itself may write (an output that is the
// input): the read-only path of those is for memory that nothing writes while the kernel
// runs.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
template <int DT> __device__ __forceinline__ float load_own_elem(const void* row, int64_t i) {
    if constexpr (DT == kF32) {
        return static_cast<const float*>(row)[i];
    } else {
        const unsigned short h = static_cast<const unsigned short*>(row)[i];
        if constexpr (DT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
        else return __half2float(__ushort_as_half(h));
    }
}

}  // namespace lse
