// 8-bit activation checkpoints: pack (with the activation function), unpack, and the activation's backward pass.
//
// All three stream: some 5 bytes an element (2 in, 1 of codes, 2 out in 16-bit types) and a few instructions. A thread takes
// 8 columns at a time, so that a warp's accesses are contiguous, and kItems such places, whose loads are in flight
// together; four neighbouring threads hold a block of 32 columns and agree on its step by two shuffles. A gated unit's
// thread takes its 8 columns of both halves. Rows whose addresses are not 16-byte aligned, and the last columns, go element by
// element.
#include <cuda_runtime.h>

#include <cstdint>

#include "packed.cuh"
#include "plan.h"
#include "stream.cuh"
#include "train.h"

namespace mica {
namespace {

constexpr int kPackThreads = 256, kItems = 4, kTile = kPackThreads * kItems;

// Where a thread's items are: place i of the matrix's rows x (4 per block) places of 8 columns, row by row.
struct Places {
    int64_t row0, rows;
    uint32_t place0, per_row;
    __device__ __forceinline__ Places(int64_t rows_, int64_t cols) : rows(rows_) {
        per_row = (uint32_t)((cols + kBlock - 1) / kBlock) * 4;
        const int64_t first = (int64_t)blockIdx.x * kTile;
        row0 = first / per_row;
        place0 = (uint32_t)(first - row0 * per_row);
    }
    // item u's row (at least rows: none) and first column
    __device__ __forceinline__ void at(int u, int64_t& row, int64_t& col) const {
        const uint32_t p = place0 + threadIdx.x + u * kPackThreads, down = p / per_row;
        row = row0 + down;
        col = (int64_t)(p - down * per_row) * 8;
    }
};

// Eight elements of a row from column col on; 0 past cols. `whole`: the row is aligned and all eight are there.
struct Eight {
    float v[8];
};

template <typename T>
__device__ __forceinline__ Eight load8(const T* p, int64_t there, bool aligned) {
    Eight r;
    if (aligned && there >= 8) {
        if constexpr (sizeof(T) == 4) {
            const uint4 a = ld16_stream(p), b = ld16_stream(p + 4);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = __uint_as_float(w[i]);
        } else {
            const uint4 a = ld16_stream(p);
            const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
            for (int i = 0; i < 8; ++i) r.v[i] = widen(e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = i < there ? widen(p[i]) : 0.0f;
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t there, bool aligned, const Eight& x) {
    if (aligned && there >= 8) {
        alignas(16) T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = narrow<T>(x.v[i]);
        const uint4* w = reinterpret_cast<const uint4*>(e);
        st16(p, w[0]);
        if constexpr (sizeof(T) == 4) st16(p + 4, w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < there) p[i] = narrow<T>(x.v[i]);
    }
}

// Packs a thread's eight columns (its three neighbours hold the block's others) and writes codes and, one of the four, the
// step. Every lane of the warp calls it.
template <bool kHalf>
__device__ __forceinline__ void pack8(const Eight& x, bool there, const mica_packed& p, int64_t row, int64_t col) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x.v[i]) & 0x7FFFFFFFu);
    most = max(most, __shfl_xor_sync(~0u, most, 1));
    most = max(most, __shfl_xor_sync(~0u, most, 2));
    if (!there) return;
    const uint32_t step = step_of(most, kHalf);
    const float inv = inverse_step(step);
    uint2 q;
    if (step == 255u) {
        q = make_uint2(0, 0);
    } else if (largest_code(step, kHalf) != 127.0f) {
        const float top = 63.0f * step_value(step);
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(x.v[i], -top), top);
        q = make_uint2(codes_of(c[0], c[1], c[2], c[3], inv), codes_of(c[4], c[5], c[6], c[7], inv));
    } else {
        q = make_uint2(codes_of(x.v[0], x.v[1], x.v[2], x.v[3], inv), codes_of(x.v[4], x.v[5], x.v[6], x.v[7], inv));
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(p.codes) + row * p.ld + col) = q;
    if (col % kBlock == 0) reinterpret_cast<uint8_t*>(p.steps)[row * p.ld_s + col / kBlock] = (uint8_t)step;
}

struct RawCodes {
    uint2 q;
    uint32_t step;
};
__device__ __forceinline__ RawCodes load_codes(const mica_packed& p, int64_t row, int64_t col) {
    RawCodes r;
    r.q = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const int8_t*>(p.codes) + row * p.ld + col));
    r.step = __ldg(reinterpret_cast<const uint8_t*>(p.steps) + row * p.ld_s + col / kBlock);
    return r;
}
__device__ __forceinline__ Eight decode8(const RawCodes& r) {
    const float s = step_value(r.step);
    const uint32_t a = r.q.x ^ 0x80808080u, b = r.q.y ^ 0x80808080u;
    Eight x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.v[i] = code_value(a, i) * s;
        x.v[i + 4] = code_value(b, i) * s;
    }
    return x;
}

template <typename T>
__device__ __forceinline__ bool aligned16(const T* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
}

template <typename T, int kAct, bool kGated>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const T* x, int64_t ld_x, mica_packed p, T* y, int64_t ld_y) {
    constexpr bool kHalf = std::is_same<T, __half>::value;
    wait_prerequisite();
    allow_dependents();
    const int64_t F = kGated ? p.cols / 2 : p.cols;
    const Places places(p.rows, F);
    const bool in = aligned16(x, ld_x), out = kAct != MICA_ACT_NONE && aligned16(y, ld_y);
    Eight v[kItems], up[kGated ? kItems : 1];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        const T* at = x + row * ld_x + col;
        v[u] = load8(at, row < p.rows ? F - col : 0, in);
        if (kGated) up[u] = load8(at + F, row < p.rows ? F - col : 0, in);  // (F is a multiple of 32)
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        const bool there = row < p.rows;
        pack8<kHalf>(v[u], there, p, row, col);
        if (kGated) pack8<kHalf>(up[u], there, p, row, col + F);
        if (kAct != MICA_ACT_NONE && there) {
            Eight a;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float slope;
                act_of<kAct>(v[u].v[i], a.v[i], slope);
                if (kGated) a.v[i] *= up[u].v[i];
            }
            store8(y + row * ld_y + col, F - col, out, a);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(mica_packed p, T* x, int64_t ld_x) {
    wait_prerequisite();
    allow_dependents();
    const Places places(p.rows, p.cols);
    const bool out = aligned16(x, ld_x);
    RawCodes raw[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        if (row < p.rows) raw[u] = load_codes(p, row, col);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        if (row < p.rows) store8(x + row * ld_x + col, p.cols - col, out, decode8(raw[u]));
    }
}

template <typename T, int kAct, bool kGated>
__global__ void __launch_bounds__(kPackThreads) act_grad_kernel(mica_packed p, const T* dy, int64_t ld_dy, T* dx,
                                                                int64_t ld_dx) {
    wait_prerequisite();
    allow_dependents();
    const int64_t F = kGated ? p.cols / 2 : p.cols;
    const Places places(p.rows, F);
    const bool in = aligned16(dy, ld_dy), out = aligned16(dx, ld_dx);
    RawCodes gate[kItems], up[kGated ? kItems : 1];
    Eight g[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        if (row >= p.rows) continue;
        gate[u] = load_codes(p, row, col);
        if (kGated) up[u] = load_codes(p, row, col + F);
        g[u] = load8(dy + row * ld_dy + col, F - col, in);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        int64_t row, col;
        places.at(u, row, col);
        if (row >= p.rows) continue;
        const Eight x = decode8(gate[u]);
        Eight a, b;
        if (kGated) b = decode8(up[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y, slope;
            act_of<kAct>(x.v[i], y, slope);
            a.v[i] = kGated ? g[u].v[i] * b.v[i] * slope : g[u].v[i] * slope;
            b.v[i] = g[u].v[i] * y;
        }
        T* at = dx + row * ld_dx + col;
        store8(at, F - col, out, a);
        if (kGated) store8(at + F, F - col, out, b);
    }
}

template <typename K, typename... A>
cudaError_t launch_places(K kernel, int64_t rows, int64_t cols, void* stream, A... args) {
    const int64_t places = rows * ((cols + kBlock - 1) / kBlock * 4), ctas = (places + kTile - 1) / kTile;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPackThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// f(a value of the type) for a checked type
template <typename F>
int by_type(int32_t dtype, F f) {
    return (int)(dtype == MICA_F32 ? f(float{}) : dtype == MICA_F16 ? f(__half{}) : f(__nv_bfloat16{}));
}

template <int kAct>
struct Act {
    static constexpr int value = kAct;
};

// f(Act<act>) for a checked activation function
template <typename F>
cudaError_t by_act(int32_t act, F f) {
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
    const int64_t F = gated ? p.cols / 2 : p.cols;
    return by_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        const T* in = static_cast<const T*>(x);
        T* out = static_cast<T*>(y);
        if (act == MICA_ACT_NONE)
            return launch_places(pack_kernel<T, MICA_ACT_NONE, false>, p.rows, F, stream, in, ld_x, p, out, ld_y);
        return by_act(act, [&](auto a) {
            constexpr int k = decltype(a)::value;
            return gated ? launch_places(pack_kernel<T, k, true>, p.rows, F, stream, in, ld_x, p, out, ld_y)
                         : launch_places(pack_kernel<T, k, false>, p.rows, F, stream, in, ld_x, p, out, ld_y);
        });
    });
}

int launch_act_unpack(const mica_packed& p, void* x, int64_t ld_x, void* stream) {
    return by_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_places(unpack_kernel<T>, p.rows, p.cols, stream, p, static_cast<T*>(x), ld_x);
    });
}

int launch_act_grad(const mica_packed& p, int32_t act, bool gated, const void* dy, int64_t ld_dy, int32_t dtype, void* dx,
                    int64_t ld_dx, void* stream) {
    const int64_t F = gated ? p.cols / 2 : p.cols;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const T* g = static_cast<const T*>(dy);
        T* d = static_cast<T*>(dx);
        return by_act(act, [&](auto a) {
            constexpr int k = decltype(a)::value;
            return gated ? launch_places(act_grad_kernel<T, k, true>, p.rows, F, stream, p, g, ld_dy, d, ld_dx)
                         : launch_places(act_grad_kernel<T, k, false>, p.rows, F, stream, p, g, ld_dy, d, ld_dx);
        });
    });
}

}  // namespace mica
