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

// The same with the type known: for loops that branch on it once.
template <bool kHalf>
__device__ __forceinline__ uint4 pack8(const float *v) {
    constexpr int32_t t = kHalf ? CONV_FLOAT16 : CONV_BFLOAT16;
    return make_uint4(pack2(v[0], v[1], t), pack2(v[2], v[3], t), pack2(v[4], v[5], t), pack2(v[6], v[7], t));
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

// ---------------------------------------------------------------- pairs
// The activations work on two values at a time with the packed 32-bit
// instructions, which take half the issue slots of the plain ones.
struct Pair {
    uint64_t v;
};

__device__ __forceinline__ Pair pair(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ Pair pair(float a) { return pair(a, a); }
__device__ __forceinline__ void split(Pair p, float *a, float *b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(p.v)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// -|v| held to -16, max(v, 0): both keep a NaN.
__device__ __forceinline__ float minus_abs16(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0fC1800000;" : "=f"(r) : "f"(-fabsf(v)));
    return r;
}
__device__ __forceinline__ float max0(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ Pair exp2_2(Pair p) {
    float a, b;
    split(p, &a, &b);
    return pair(exp2_approx(a), exp2_approx(b));
}

// Logistic function of u from -u * log2(e): 1 / (1 + 2^arg).
__device__ __forceinline__ Pair logistic_of(Pair arg) {
    const Pair d = add2(exp2_2(arg), pair(1.0f));
    float a, b;
    split(d, &a, &b);
    return pair(rcp_approx(a), rcp_approx(b));
}

// z/2 (1 + tanh u) = z * logistic(2u), without cancellation where tanh u is
// near -1; the logistic's argument is 2u = 2 sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ Pair gelu_tanh_arg(Pair z) {
    const Pair z2 = mul2(z, z);
    return mul2(z, fma2(z2, pair(-0.102943245f), pair(-2.302208198f)));  // times -log2(e)
}

// Phi(x) for x = -min(|z|, 16), as 2^p(x): the logarithm of the normal tail
// is nearly a parabola, so that a polynomial of degree 6 does (fitted to
// minimise the largest error of Phi over [-9, 0], by least squares on
// Chebyshev nodes reweighted towards the maximum): off by 1.4e-7 at most in
// 32-bit arithmetic, and falling below 2^-126 before x = -16.  One
// exponential per value and half the instructions of a polynomial times
// exp(-x^2/2).
// That is the accuracy of 1 + erf in 32 bits, and like it absolute: of Phi
// itself it is 0.24 % at -4, 2.1 % at -5 and 8.8 % at -6.  (Accuracy of 2^-12
// of Phi takes degree 11 and 12 us of the 111 us of 50176 x 512 -> 2048 with a
// pre-activation, 2^-10 degree 8 and 5.5 us.)
__device__ __forceinline__ Pair normal_tail(Pair x) {
    Pair p = fma2(x, pair(1.917647205e-05f), pair(6.586165400e-04f));
    p = fma2(x, p, pair(7.754437625e-03f));
    p = fma2(x, p, pair(5.296542495e-02f));
    p = fma2(x, p, pair(-4.590602517e-01f));
    p = fma2(x, p, pair(1.151122093e+00f));
    p = fma2(x, p, pair(-9.999997020e-01f));
    return exp2_2(p);
}

// Activation of two values, in place.
template <int kAct>
__device__ __forceinline__ void activate(float &a, float &b) {
    if constexpr (kAct == CONV_ACT_RELU) {
        a = max0(a), b = max0(b);
    } else if constexpr (kAct == CONV_ACT_GELU) {
        // z Phi(z) = max(z, 0) + x Phi(x), x = -|z| (0 for z = -inf, its limit)
        const Pair x = pair(minus_abs16(a), minus_abs16(b));
        split(fma2(x, normal_tail(x), pair(max0(a), max0(b))), &a, &b);
    } else if constexpr (kAct == CONV_ACT_GELU_TANH) {
        const Pair z = pair(a, b);
        split(mul2(z, logistic_of(gelu_tanh_arg(z))), &a, &b);
    } else if constexpr (kAct == CONV_ACT_SILU) {
        const Pair z = pair(a, b);
        split(mul2(z, logistic_of(mul2(z, pair(-1.442695041f)))), &a, &b);
    }
}

// Derivative of the activation at two values, in place.
template <int kAct>
__device__ __forceinline__ void activation_slope(float &a, float &b) {
    if constexpr (kAct == CONV_ACT_RELU) {
        a = a > 0.0f ? 1.0f : 0.0f, b = b > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (kAct == CONV_ACT_GELU) {
        // Phi(z) + z phi(z), Phi(z) = 1/2 + sign(z) (1/2 - Phi(x)), z held
        // to +-16 in the second term, where phi has vanished
        const Pair x = pair(minus_abs16(a), minus_abs16(b));
        const Pair e = exp2_2(mul2(mul2(x, x), pair(-0.72134752f)));
        float u, v, xa, xb;
        split(fma2(normal_tail(x), pair(-1.0f), pair(0.5f)), &u, &v);
        split(x, &xa, &xb);
        const Pair zc = pair(copysignf(xa, a), copysignf(xb, b));
        split(fma2(mul2(zc, pair(0.39894228f)), e, add2(pair(copysignf(u, a), copysignf(v, b)), pair(0.5f))), &a, &b);
    } else if constexpr (kAct == CONV_ACT_GELU_TANH) {
        // s + z s (1 - s) (2u)', s = logistic(2u); z held to +-64 in the
        // second term, which has long vanished there, so that no infinity
        // meets its zero
        const Pair s = logistic_of(gelu_tanh_arg(pair(a, b)));
        const Pair z = pair(fminf(fmaxf(a, -64.0f), 64.0f), fminf(fmaxf(b, -64.0f), 64.0f));
        const Pair d = mul2(z, fma2(mul2(z, z), pair(0.2140644488f), pair(1.5957691216f)));
        const Pair q = fma2(mul2(s, pair(-1.0f)), s, s);
        split(fma2(d, q, s), &a, &b);
    } else if constexpr (kAct == CONV_ACT_SILU) {
        // s + z s (1 - s), s = logistic(z); z held to +-128 in the second term,
        // where s is 0 or 1 and the term has vanished, for the same reason
        const Pair s = logistic_of(mul2(pair(a, b), pair(-1.442695041f)));
        const Pair z = pair(fminf(fmaxf(a, -128.0f), 128.0f), fminf(fmaxf(b, -128.0f), 128.0f));
        const Pair q = fma2(mul2(s, pair(-1.0f)), s, s);
        split(fma2(z, q, s), &a, &b);
    } else {
        a = 1.0f, b = 1.0f;
    }
}

}  // namespace i8c
