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
// x / 2^e to the nearest integer (the product is exact unless it underflows to well below 1/2); 0 in a block of NaNs
__device__ __forceinline__ int code_of(float x, float inv, float most) {
    return inv == 0.0f ? 0 : (int)fminf(fmaxf(rintf(x * inv), -most), most);
}

// The activation functions and their slopes, in float32.
template <int kAct>
__device__ __forceinline__ void act_of(float x, float& y, float& slope) {
    if constexpr (kAct == MICA_ACT_GELU_TANH) {
        constexpr float c = 0.797884560802865356f, b = 0.044715f;
        const float x2 = x * x, u = tanhf(c * x * fmaf(b, x2, 1.0f)), h = 0.5f + 0.5f * u;
        y = x * h;
        slope = fmaf(0.5f * x * (1.0f - u * u), c * fmaf(3.0f * b, x2, 1.0f), h);
        if (fabsf(x) > 1e18f) slope = h;  // x2 overflows there: 0 * inf
    } else if constexpr (kAct == MICA_ACT_GELU) {
        const float p = normcdff(x);
        y = x * p;
        slope = fmaf(x * 0.398942280401432678f, expf(-0.5f * x * x), p);
    } else if constexpr (kAct == MICA_ACT_SILU) {
        const float e = expf(-x), s = 1.0f / (1.0f + e);
        y = x * s;
        slope = s * fmaf(x, 1.0f - s, 1.0f);
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
