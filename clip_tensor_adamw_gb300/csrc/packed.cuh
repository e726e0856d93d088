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
__device__ __forceinline__ uint32_t codes_of(Two a, Two b, float inv) {
    const Two k = two(inv, inv), magic = two(12582912.0f, 12582912.0f);
    const float2 p = each(fma2(a, k, magic)), q = each(fma2(b, k, magic));
    return __byte_perm(__byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x0040),
                       __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040), 0x5410);
}
// Byte i of w, a code, as a float: 2^23 + (q + 128) has the bits 0x4B000000 | (q ^ 128).
__device__ __forceinline__ float code_value(uint32_t flipped, int i) {
    return __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7440u | i)) - 8388736.0f;
}

__device__ __forceinline__ float fast_reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// h = 1 / (1 + 2^t), from the hardware's power of two and reciprocal (some 2^-22 of its value, and |t| 2^-24 in the tail): the
// logistic function of w for t = -log2(e) w; and rest = 1 - h, as 2^t h, since an h near 1 has no digits left of it.
__device__ __forceinline__ void logistic_of(float t, float& h, float& rest) {
    const float e = exp2_fast(t);
    h = fast_reciprocal(1.0f + e);
    rest = fminf(e, 0x1p100f) * h;  // (an infinite e makes h 0; beyond 2^100 what rest is for is multiplied by h too)
}

constexpr float kLog2E = 1.44269504088896341f;
constexpr float kGelu1 = 2.0f * 0.797884560802865356f, kGelu3 = kGelu1 * 0.044715f;  // 2 u = kGelu1 x + kGelu3 x^3

// The activation functions and their slopes, in float32. GELU's tanh form is x * logistic(2 u), u = c (x + b x^3), since
// (1 + tanh u) / 2 = logistic(2 u); its slope is h + x h (1 - h) 2 u'. Past |x| = 20, where h is 0 or 1, x^2 is held, so
// that u' stays finite.
template <int kAct>
__device__ __forceinline__ void act_of(float x, float& y, float& slope) {
    if constexpr (kAct == MICA_ACT_GELU_TANH) {
        const float x2 = fminf(x * x, 400.0f);
        float h, rest;
        logistic_of(x * fmaf(-kLog2E * kGelu3, x2, -kLog2E * kGelu1), h, rest);
        y = x * h;
        slope = fmaf(y * rest, fmaf(3.0f * kGelu3, x2, kGelu1), h);
    } else if constexpr (kAct == MICA_ACT_GELU) {
        const float p = normcdff(x);
        y = x * p;
        slope = fmaf(x * 0.398942280401432678f, expf(-0.5f * x * x), p);
    } else if constexpr (kAct == MICA_ACT_SILU) {
        float h, rest;
        logistic_of(-kLog2E * x, h, rest);
        y = x * h;
        slope = fmaf(y, rest, h);
    } else if constexpr (kAct == MICA_ACT_RELU) {
        y = x > 0.0f ? x : (x <= 0.0f ? 0.0f : x);  // (a NaN stays one)
        slope = x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
    } else {
        y = x;
        slope = 1.0f;
    }
}

// Two of the functions' values at a time.
template <int kAct>
__device__ __forceinline__ Two act_pair(Two x) {
    if constexpr (kAct == MICA_ACT_GELU_TANH || kAct == MICA_ACT_SILU) {
        Two t = two(-kLog2E, -kLog2E);
        if constexpr (kAct == MICA_ACT_GELU_TANH)
            t = fma2(two(-kLog2E * kGelu3, -kLog2E * kGelu3), x * x, two(-kLog2E * kGelu1, -kLog2E * kGelu1));
        const float2 e = each(x * t);
        const float2 d = each(two(exp2_fast(e.x), exp2_fast(e.y)) + two(1.0f, 1.0f));
        return x * two(fast_reciprocal(d.x), fast_reciprocal(d.y));
    } else {
        const float2 v = each(x);
        float a, b, slope;
        act_of<kAct>(v.x, a, slope);
        act_of<kAct>(v.y, b, slope);
        return two(a, b);
    }
}

}  // namespace
}  // namespace mica
