// The two 16-bit element types of the prompt side's operators: packed pairs to
// fp32 and back (low half first, one rounding to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace h3a {

template <bool FP16>
struct Half16;

template <>
struct Half16<false> {
    using T = __nv_bfloat16;
    __device__ static __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    // acc + 0 * w by halves: NaN from an infinity or NaN on
    __device__ static __forceinline__ uint32_t add_zero_times(uint32_t w, uint32_t acc) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
        return r;
    }
    // Exponent bits of both halves, and what is added to find one that is all ones.
    static constexpr uint32_t kExponents = 0x7F807F80u, kStep = 0x00800080u;
};

template <>
struct Half16<true> {
    using T = __half;
    __device__ static __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
    }
    __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ uint32_t add_zero_times(uint32_t w, uint32_t acc) {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
        return r;
    }
    static constexpr uint32_t kExponents = 0x7C007C00u, kStep = 0x04000400u;
};

// Bit 15 (31) set where the low (high) half of w is an infinity or NaN: adding
// one to an exponent of all ones carries into the sign's place, which the mask
// has cleared.
template <bool FP16>
__device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w) {
    return ((w & Half16<FP16>::kExponents) + Half16<FP16>::kStep) & 0x80008000u;
}

// w with the halves that are infinities or NaN replaced by zero.
template <bool FP16>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w, uint32_t bad) {
    return w & ~((bad >> 15) * 0xFFFFu);
}

}  // namespace h3a
