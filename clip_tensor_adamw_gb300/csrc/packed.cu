// 8-bit activation checkpoints: pack (with the activation function), unpack, and the activation's backward pass.
#include <cuda_runtime.h>

#include <cstdint>

#include "packed.cuh"
#include "plan.h"
#include "train.h"

namespace mica {
namespace {

constexpr int kPackThreads = 256;

// One warp packs a block of 32 columns; lane j holds column j.
template <typename T, int kAct, bool kGated>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const T* x, int64_t ld_x, mica_packed p, T* y, int64_t ld_y) {
    const int lane = threadIdx.x & 31;
    const int64_t blocks = (p.cols + kBlock - 1) / kBlock, F = kGated ? p.cols / 2 : p.cols;
    constexpr bool half = std::is_same<T, __half>::value;
    for (int64_t i = (int64_t)blockIdx.x * (kPackThreads / 32) + threadIdx.x / 32; i < p.rows * blocks;
         i += (int64_t)gridDim.x * (kPackThreads / 32)) {
        const int64_t row = i / blocks, b = i % blocks, col = b * kBlock + lane;
        const float v = col < p.cols ? widen(x[row * ld_x + col]) : 0.0f;
        const uint32_t most = __reduce_max_sync(~0u, __float_as_uint(v) & 0x7FFFFFFFu), step = step_of(most, half);
        reinterpret_cast<int8_t*>(p.codes)[row * p.ld + col] = (int8_t)code_of(v, inverse_step(step), largest_code(step, half));
        if (lane == 0) reinterpret_cast<uint8_t*>(p.steps)[row * p.ld_s + b] = (uint8_t)step;
        if (kAct != MICA_ACT_NONE && col < F) {
            float a, slope;
            act_of<kAct>(v, a, slope);
            if (kGated) a *= widen(x[row * ld_x + F + col]);
            y[row * ld_y + col] = narrow<T>(a);
        }
    }
}

__device__ __forceinline__ float value_of(const mica_packed& p, int64_t row, int64_t col) {
    return (float)reinterpret_cast<const int8_t*>(p.codes)[row * p.ld + col] *
           step_value(reinterpret_cast<const uint8_t*>(p.steps)[row * p.ld_s + col / kBlock]);
}

template <typename T>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(mica_packed p, T* x, int64_t ld_x) {
    for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < p.rows * p.cols;
         i += (int64_t)gridDim.x * kPackThreads) {
        const int64_t row = i / p.cols, col = i % p.cols;
        x[row * ld_x + col] = narrow<T>(value_of(p, row, col));
    }
}

template <typename T, int kAct, bool kGated>
__global__ void __launch_bounds__(kPackThreads) act_grad_kernel(mica_packed p, const T* dy, int64_t ld_dy, T* dx,
                                                                int64_t ld_dx) {
    const int64_t F = kGated ? p.cols / 2 : p.cols;
    for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < p.rows * F;
         i += (int64_t)gridDim.x * kPackThreads) {
        const int64_t row = i / F, col = i % F;
        const float g = widen(dy[row * ld_dy + col]);
        float a, slope;
        act_of<kAct>(value_of(p, row, col), a, slope);
        if (kGated) {
            dx[row * ld_dx + col] = narrow<T>(g * value_of(p, row, F + col) * slope);
            dx[row * ld_dx + F + col] = narrow<T>(g * a);
        } else {
            dx[row * ld_dx + col] = narrow<T>(g * slope);
        }
    }
}

unsigned grid_for(int64_t threads) {
    const int64_t g = (threads + kPackThreads - 1) / kPackThreads;
    return (unsigned)(g < 1 ? 1 : g > (1 << 20) ? (1 << 20) : g);
}

template <typename F>
int by_type(int32_t dtype, F f) {
    if (dtype == MICA_F32) f(float{});
    else if (dtype == MICA_F16) f(__half{});
    else f(__nv_bfloat16{});
    count_launches(1);
    return (int)cudaGetLastError();
}

template <int kAct>
struct Act {
    static constexpr int value = kAct;
};

// f(Act<kAct>, gated as a type) for the checked act
template <typename F>
void by_act(int32_t act, F f) {
    switch (act) {
        case MICA_ACT_GELU_TANH: return f(Act<MICA_ACT_GELU_TANH>{});
        case MICA_ACT_GELU: return f(Act<MICA_ACT_GELU>{});
        case MICA_ACT_SILU: return f(Act<MICA_ACT_SILU>{});
        default: return f(Act<MICA_ACT_RELU>{});
    }
}

}  // namespace

int launch_act_pack(const void* x, int64_t ld_x, const mica_packed& p, int32_t act, bool gated, void* y, int64_t ld_y,
                    void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = grid_for(p.rows * ((p.cols + kBlock - 1) / kBlock * kBlock));
    return by_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        const T* in = static_cast<const T*>(x);
        T* out = static_cast<T*>(y);
        if (act == MICA_ACT_NONE) {
            pack_kernel<T, MICA_ACT_NONE, false><<<grid, kPackThreads, 0, st>>>(in, ld_x, p, out, ld_y);
            return;
        }
        by_act(act, [&](auto a) {
            if (gated) pack_kernel<T, decltype(a)::value, true><<<grid, kPackThreads, 0, st>>>(in, ld_x, p, out, ld_y);
            else pack_kernel<T, decltype(a)::value, false><<<grid, kPackThreads, 0, st>>>(in, ld_x, p, out, ld_y);
        });
    });
}

int launch_act_unpack(const mica_packed& p, void* x, int64_t ld_x, void* stream) {
    return by_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        unpack_kernel<T><<<grid_for(p.rows * p.cols), kPackThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            p, static_cast<T*>(x), ld_x);
    });
}

int launch_act_grad(const mica_packed& p, int32_t act, bool gated, const void* dy, int64_t ld_dy, int32_t dtype, void* dx,
                    int64_t ld_dx, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = grid_for(p.rows * (gated ? p.cols / 2 : p.cols));
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        by_act(act, [&](auto a) {
            const T* g = static_cast<const T*>(dy);
            T* d = static_cast<T*>(dx);
            if (gated) act_grad_kernel<T, decltype(a)::value, true><<<grid, kPackThreads, 0, st>>>(p, g, ld_dy, d, ld_dx);
            else act_grad_kernel<T, decltype(a)::value, false><<<grid, kPackThreads, 0, st>>>(p, g, ld_dy, d, ld_dx);
        });
    });
}

}  // namespace mica
