// The 8-bit checkpoint's format, and the activation functions.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "mica_train.h"

namespace mica {
namespace {

constexpr int kBlock = 32;  // columns that share a step

// The stored exponent (e + 127) of a block whose largest magnitude has the bits `most`: the smallest e with
// max / 2^e < 127.5. With max = m * 2^E, 1 <= m < 2, that is E - 6 for m < 1.9921875 (an m whose first 7 fraction bits
// are not all ones) and E - 5 above: adding 2^16 to the bits carries into E exactly there.
__device__ __forceinline__ uint32_t step_of(uint32_t most, bool half_source) {
    if (most >= 0x7F800000u) return 255u;
    const int e = (int)((most + 0x10000u) >> 23) - 6, least = half_source ? 103 : 1;
    return (uint32_t)(e < least ? least : e);
}
// 2^-e, a normal float for every stored exponent of a finite block (1 .. 249); 0 for a block of NaNs, whose codes are 0
__device__ __forceinline__ float inverse_step(uint32_t step) {
    return step == 255u ? 0.0f : __uint_as_float((254u - step) << 23);
}
// 2^e; NaN for 255
__device__ __forceinline__ float step_value(uint32_t step) {
    return __uint_as_float(step == 255u ? 0x7FC00000u : step << 23);
}
// The largest code: 127, but 63 at the type's top exponent, where 64 steps would be past its largest finite value (2^16
// in binary16, 2^128 in the others).
__device__ __forceinline__ float largest_code(uint32_t step, bool half_source) {
    return step == (half_source ? 137u : 249u) ? 63.0f : 127.0f;
}
// Four codes x / 2^e, to nearest, ties to even: x * inv is exact (unless it underflows to well below 1/2), and adding
// 1.5 * 2^23 rounds it to an integer, whose two's complement is then in the low byte.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d, float inv) {
    const uint32_t p = __float_as_uint(fmaf(a, inv, 12582912.0f)), q = __float_as_uint(fmaf(b, inv, 12582912.0f));
    const uint32_t r = __float_as_uint(fmaf(c, inv, 12582912.0f)), t = __float_as_uint(fmaf(d, inv, 12582912.0f));
    return __byte_perm(__byte_perm(p, q, 0x0040), __byte_perm(r, t, 0x0040), 0x5410);
}
// Byte i of w, a code, as a float: 2^23 + (q + 128) has the bits 0x4B000000 | (q ^ 128).
__device__ __forceinline__ float code_value(uint32_t flipped, int i) {
    return __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7440u | i)) - 8388736.0f;
}

// 1 / (1 + exp(-w)), from the hardware's power of two and reciprocal (some 2^-22 of its value, and |w| 2^-24 in the tail)
__device__ __forceinline__ float logistic(float w) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w * -1.44269504088896341f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// The activation functions and their slopes, in float32. GELU's tanh form is x * logistic(2 u), u = c (x + b x^3), since
// (1 + tanh u) / 2 = logistic(2 u); its slope is h + x h (1 - h) 2 u'. Past |x| = 20, where h is 0 or 1, x^2 is held, so
// that u' stays finite.
template <int kAct>
__device__ __forceinline__ void act_of(float x, float& y, float& slope) {
    if constexpr (kAct == MICA_ACT_GELU_TANH) {
        constexpr float c2 = 2.0f * 0.797884560802865356f, b = 0.044715f;
        const float x2 = fminf(x * x, 400.0f), h = logistic(c2 * x * fmaf(b, x2, 1.0f));
        y = x * h;
        slope = fmaf(y * (1.0f - h), fmaf(3.0f * b * c2, x2, c2), h);
    } else if constexpr (kAct == MICA_ACT_GELU) {
        const float p = normcdff(x);
        y = x * p;
        slope = fmaf(x * 0.398942280401432678f, expf(-0.5f * x * x), p);
    } else if constexpr (kAct == MICA_ACT_SILU) {
        const float h = logistic(x);
        y = x * h;
        slope = fmaf(y, 1.0f - h, h);
    } else if constexpr (kAct == MICA_ACT_RELU) {
        y = x > 0.0f ? x : (x <= 0.0f ? 0.0f : x);  // (a NaN stays one)
        slope = x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
    } else {
        y = x;
        slope = 1.0f;
    }
}

}  // namespace
}  // namespace mica
