// channel_math.cuh -- element conversions and activations of the channel
// operators, all in 32-bit floats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int8conv.h"

namespace i8c {

// Element i of a typed buffer as a float, and back (rounded to nearest even).
__device__ __forceinline__ float load_as_float(const void *p, int64_t i, int32_t dtype) {
    switch (dtype) {
        case CONV_FLOAT32: return ((const float *)p)[i];
        case CONV_FLOAT16: return __half2float(((const __half *)p)[i]);
        case CONV_BFLOAT16: return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
        default: return (float)((const int32_t *)p)[i];
    }
}

__device__ __forceinline__ void store_from_float(void *p, int64_t i, int32_t dtype, float v) {
    switch (dtype) {
        case CONV_FLOAT32: ((float *)p)[i] = v; break;
        case CONV_FLOAT16: ((__half *)p)[i] = __float2half_rn(v); break;
        default: ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(v); break;
    }
}

// Logistic function and Phi, the standard normal distribution.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678f * z); }

// z/2 (1 + tanh u) = z * logistic(2u): no cancellation where tanh u is near -1.
__device__ __forceinline__ float gelu_tanh_arg2(float z) {
    return 1.5957691216f * (z + 0.044715f * z * z * z);
}

template <int kAct>
__device__ __forceinline__ float activate(float z) {
    if constexpr (kAct == CONV_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (kAct == CONV_ACT_GELU) return z * normal_cdf(z);
    if constexpr (kAct == CONV_ACT_GELU_TANH) return z * logistic(gelu_tanh_arg2(z));
    if constexpr (kAct == CONV_ACT_SILU) return z * logistic(z);
    return z;
}

// Derivative of the activation at z.
template <int kAct>
__device__ __forceinline__ float activation_slope(float z) {
    if constexpr (kAct == CONV_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (kAct == CONV_ACT_GELU) return normal_cdf(z) + z * 0.39894228f * __expf(-0.5f * z * z);
    if constexpr (kAct == CONV_ACT_GELU_TANH) {
        // (z held to +-64 in the second term, which has long vanished there,
        // so that no infinity meets its zero)
        const float s = logistic(gelu_tanh_arg2(z));
        const float zc = fminf(fmaxf(z, -64.0f), 64.0f);
        return s + zc * s * (1.0f - s) * 1.5957691216f * (1.0f + 0.134145f * zc * zc);
    }
    if constexpr (kAct == CONV_ACT_SILU) {
        const float s = logistic(z);
        return s + z * s * (1.0f - s);
    }
    return 1.0f;
}

}  // namespace i8c
