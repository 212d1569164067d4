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

// Two 16-bit values in a word, eight in a 16-byte vector.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int32_t dtype) {
    if (dtype == CONV_FLOAT16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void unpack2(uint32_t w, int32_t dtype, float *lo, float *hi) {
    if (dtype == CONV_FLOAT16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        *lo = f.x, *hi = f.y;
    } else {
        *lo = __uint_as_float(w << 16);
        *hi = __uint_as_float(w & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *v, int32_t dtype) {
    return make_uint4(pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype), pack2(v[4], v[5], dtype),
                      pack2(v[6], v[7], dtype));
}

__device__ __forceinline__ void unpack8(const uint4 &w, int32_t dtype, float *v) {
    unpack2(w.x, dtype, v, v + 1);
    unpack2(w.y, dtype, v + 2, v + 3);
    unpack2(w.z, dtype, v + 4, v + 5);
    unpack2(w.w, dtype, v + 6, v + 7);
}

// Logistic function and Phi, the standard normal distribution.
__device__ __forceinline__ float exp2f_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// Phi(z) by formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions: erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + p x),
// off by at most 1.5e-7 for x >= 0; here x = |z| / sqrt(2) and the halved
// coefficients give Phi(-|z|), off by 7.5e-8.  One exponential and one
// reciprocal per value (erfcf takes about twice the instructions); *density
// is exp(-z^2 / 2), which the slope needs too.
__device__ __forceinline__ float normal_cdf(float z, float *density) {
    const float e = exp2f_fast(-0.72134752f * z * z);
    const float t = __fdividef(1.0f, fmaf(0.23164189f, fabsf(z), 1.0f));
    float h = fmaf(t, 0.5307027145f, -0.7265760135f);
    h = fmaf(t, h, 0.7107068705f);
    h = fmaf(t, h, -0.142248368f);
    h = fmaf(t, h, 0.127414796f);
    h = h * t * e;
    *density = e;
    return z < 0.0f ? h : 1.0f - h;
}

// z/2 (1 + tanh u) = z * logistic(2u): no cancellation where tanh u is near -1.
__device__ __forceinline__ float gelu_tanh_arg2(float z) {
    return 1.5957691216f * (z + 0.044715f * z * z * z);
}

template <int kAct>
__device__ __forceinline__ float activate(float z) {
    if constexpr (kAct == CONV_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (kAct == CONV_ACT_GELU) {
        float e;
        return z * normal_cdf(z, &e);
    }
    if constexpr (kAct == CONV_ACT_GELU_TANH) return z * logistic(gelu_tanh_arg2(z));
    if constexpr (kAct == CONV_ACT_SILU) return z * logistic(z);
    return z;
}

// Derivative of the activation at z.
template <int kAct>
__device__ __forceinline__ float activation_slope(float z) {
    if constexpr (kAct == CONV_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (kAct == CONV_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, &e);
        return fmaf(0.39894228f * z, e, c);
    }
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
