// eight_bit.cuh -- 8-bit floats and their block scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "channel.h"
#include "channel_math.cuh"

namespace i8c {

constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126

__host__ __device__ __forceinline__ constexpr float largest_of(bool e5m2) { return e5m2 ? 57344.0f : 448.0f; }

// Four floats as 8-bit values, the first in the lowest byte; to nearest even,
// beyond the largest value to it, NaN kept.
template <bool kE5m2>
__device__ __forceinline__ uint32_t pack_eight_bit(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if constexpr (kE5m2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Two 8-bit values (the lower half of `v`) as two f16, which hold either type's exactly.
template <bool kE5m2>
__device__ __forceinline__ uint32_t unpack_eight_bit(uint16_t v) {
    uint32_t r;
    if constexpr (kE5m2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(v));
    else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// Magnitudes are compared as bit patterns: that orders them, infinity above
// every finite one and NaN above infinity, so that both reach the scale.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A block's scale, and L / a as the sum of two floats, which takes its values
// to [-L, L].  The second makes up for the rounding of the first: with it a
// quotient that 32 bits hold comes out as it is, so that a value halfway
// between two 8-bit ones is seen to be (without it 2 values in 10000 of bf16
// rows went to the odd neighbour).
struct BlockScale {
    float scale, factor, rest;
};
template <bool kE5m2>
__device__ __forceinline__ BlockScale block_scale(uint32_t most) {
    constexpr float L = largest_of(kE5m2);
    const float a = __uint_as_float(most), s = a * (1.0f / L);
    BlockScale b;
    // (a / L by its reciprocal is within 2^-23 of the quotient, which is near
    // enough for the choice but not for the scale itself)
    if (s < kLeastScale) {
        b.scale = kLeastScale, b.factor = 1.0f / kLeastScale, b.rest = 0.0f;
    } else {
        b.scale = __fdiv_rn(a, L), b.factor = __fdiv_rn(L, a);
        // (L - factor * a is exact; an infinite a has a factor of 0)
        b.rest = b.factor > 0.0f ? fmaf(-b.factor, a, L) * (1.0f / L) * b.factor : 0.0f;
    }
    return b;
}
__device__ __forceinline__ Pair quotient(Pair v, Pair factor, Pair rest) { return fma2(v, factor, mul2(v, rest)); }
__device__ __forceinline__ float quotient(float v, const BlockScale &b) { return fmaf(v, b.factor, v * b.rest); }

}  // namespace i8c
