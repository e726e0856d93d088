// 8-bit activation checkpoints: pack (with the activation function), unpack, and the activation's backward pass.
//
// All three stream: some 5 bytes an element (2 in, 1 of codes, 2 out in 16-bit types), which bounds them, and some 15
// instructions, which must not. A thread takes 8 columns of kItems rows, whose loads are in flight together; 2^k
// neighbouring threads share a row, as many as its columns fill (see launch_places), so that indices take shifts and not
// divisions. Four threads hold a block of 32 columns and agree on its step by two shuffles. A gated unit's thread takes its 8
// columns of both halves. Rows whose addresses are not 16-byte aligned, and the last columns, go element by element.
#include <cuda_runtime.h>

#include <cstdint>

#include "packed.cuh"
#include "plan.h"
#include "stream.cuh"
#include "train.h"

namespace mica {
namespace {

constexpr int kPackThreads = 256;

// How a matrix's places (8 columns of a row each) are dealt: 2^log threads a row and `tiles` of them, kItems times.
struct Shape {
    int32_t log, tiles;
};

struct Places {
    int64_t row, rows, col;
    int32_t apart;  // rows between a thread's items
    __device__ __forceinline__ Places(Shape s, int items, int64_t rows_) : rows(rows_) {
        const uint32_t at = blockIdx.x / (uint32_t)s.tiles, tile = blockIdx.x - at * (uint32_t)s.tiles;
        apart = kPackThreads >> s.log;
        row = (int64_t)at * apart * items + (threadIdx.x >> s.log);
        col = (((int64_t)tile << s.log) + (threadIdx.x & ((1 << s.log) - 1))) * 8;
    }
};

// Eight elements of a row as they are stored.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(reinterpret_cast<const uint32_t*>(w)[i]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const uint32_t p = reinterpret_cast<const uint32_t*>(w)[i / 2];
            return __uint_as_float(i % 2 ? p & 0xFFFF0000u : p << 16);
        } else {
            const uint32_t p = reinterpret_cast<const uint32_t*>(w)[i / 2];
            return __half2float(__ushort_as_half((unsigned short)(p >> (16 * (i % 2)))));
        }
    }
    __device__ __forceinline__ Two pair(int i) const { return two(get(2 * i), get(2 * i + 1)); }
    // the bits of the largest magnitude, as a float32's
    __device__ __forceinline__ uint32_t most() const {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(w);
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, p[i] & 0x7FFFFFFFu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(p[i] & 0x7FFF7FFFu));
            m = max(m & 0xFFFFu, m >> 16);
            if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
            else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
        }
    }
};

// Eight elements from p on, of which `there` are in the row; the others 0.
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p, int64_t there, bool aligned) {
    Eight<T> r;
    if (aligned && there >= 8) {
        r.w[0] = ld16_stream(p);
        if constexpr (sizeof(T) == 4) r.w[1] = ld16_stream(p + 4);
    } else {
        alignas(16) T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < there ? p[i] : narrow<T>(0.0f);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(e)[i];
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t there, bool aligned, const float (&x)[8]) {
    if (aligned && there >= 8) {
        if constexpr (sizeof(T) == 4) {
            st16(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
            st16(p + 4, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    const __nv_bfloat162 q = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&q);
                } else {
                    const __half2 q = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&q);
                }
            }
            st16(p, make_uint4(w[0], w[1], w[2], w[3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < there) p[i] = narrow<T>(x[i]);
    }
}

// Packs a thread's eight columns (its three neighbours hold the block's others) and writes codes and, one of the four, the
// step. Every lane of the warp calls it.
template <typename T>
__device__ __forceinline__ void pack8(const Eight<T>& x, bool there, int8_t* codes, uint8_t* steps, bool writes_step) {
    constexpr bool kHalf = std::is_same<T, __half>::value;
    uint32_t most = x.most();
    most = max(most, __shfl_xor_sync(~0u, most, 1));
    most = max(most, __shfl_xor_sync(~0u, most, 2));
    if (!there) return;
    const uint32_t step = step_of(most, kHalf);
    const float inv = inverse_step(step);
    uint2 q = make_uint2(0, 0);
    if (step == 255u || largest_code(step, kHalf) != 127.0f) {
        const float top = 63.0f * step_value(step);
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(x.get(i), -top), top);
        if (step != 255u)
            q = make_uint2(codes_of(two(c[0], c[1]), two(c[2], c[3]), inv), codes_of(two(c[4], c[5]), two(c[6], c[7]), inv));
    } else {
        q = make_uint2(codes_of(x.pair(0), x.pair(1), inv), codes_of(x.pair(2), x.pair(3), inv));
    }
    *reinterpret_cast<uint2*>(codes) = q;
    if (writes_step) *steps = (uint8_t)step;
}

struct RawCodes {
    uint2 q;
    uint32_t step;
};
__device__ __forceinline__ RawCodes load_codes(const int8_t* codes, const uint8_t* steps) {
    return RawCodes{__ldcs(reinterpret_cast<const uint2*>(codes)), __ldg(steps)};
}
__device__ __forceinline__ void decode8(const RawCodes& r, float (&x)[8]) {
    const float s = step_value(r.step);
    const uint32_t a = r.q.x ^ 0x80808080u, b = r.q.y ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = code_value(a, i) * s;
        x[i + 4] = code_value(b, i) * s;
    }
}

template <typename T>
__device__ __forceinline__ bool aligned16(const T* p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)sizeof(T) % 16 == 0;
}

template <typename T, int kAct, bool kGated, int kItems>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(Shape shape, const T* x, int64_t ld_x, mica_packed p, T* y,
                                                            int64_t ld_y) {
    wait_prerequisite();
    allow_dependents();
    const int64_t F = kGated ? p.cols / 2 : p.cols;
    const Places at(shape, kItems, p.rows);
    const int64_t padded = (F + kBlock - 1) / kBlock * kBlock;  // codes past the columns are written too, as 0
    const bool in = aligned16(x, ld_x), out = kAct != MICA_ACT_NONE && aligned16(y, ld_y);
    const T* from = x + at.row * ld_x + at.col;
    T* to = kAct != MICA_ACT_NONE ? y + at.row * ld_y + at.col : nullptr;
    int8_t* codes = reinterpret_cast<int8_t*>(p.codes) + at.row * p.ld + at.col;
    uint8_t* steps = reinterpret_cast<uint8_t*>(p.steps) + at.row * p.ld_s + (at.col >> 5);
    const bool first = at.col % kBlock == 0;
    Eight<T> v[kItems], up[kGated ? kItems : 1];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const T* q = from + u * at.apart * ld_x;
        const int64_t there = at.row + u * at.apart < p.rows ? F - at.col : 0;
        v[u] = load8(q, there, in);
        if (kGated) up[u] = load8(q + F, there, in);  // (F is a multiple of 32)
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        const bool there = at.row + u * at.apart < p.rows && at.col < padded;
        pack8(v[u], there, codes + u * at.apart * p.ld, steps + u * at.apart * p.ld_s, first);
        if (kGated) pack8(up[u], there, codes + u * at.apart * p.ld + F, steps + u * at.apart * p.ld_s + F / kBlock, first);
        if (kAct != MICA_ACT_NONE && there) {
            float a[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Two r = act_pair<kAct>(v[u].pair(i));
                if (kGated) r = r * up[u].pair(i);
                const float2 f = each(r);
                a[2 * i] = f.x;
                a[2 * i + 1] = f.y;
            }
            store8(to + u * at.apart * ld_y, F - at.col, out, a);
        }
    }
}

template <typename T, int kItems>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(Shape shape, mica_packed p, T* x, int64_t ld_x) {
    wait_prerequisite();
    allow_dependents();
    const Places at(shape, kItems, p.rows);
    const bool out = aligned16(x, ld_x);
    if (at.col >= p.cols) return;
    const int8_t* codes = reinterpret_cast<const int8_t*>(p.codes) + at.row * p.ld + at.col;
    const uint8_t* steps = reinterpret_cast<const uint8_t*>(p.steps) + at.row * p.ld_s + (at.col >> 5);
    T* to = x + at.row * ld_x + at.col;
    RawCodes raw[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        if (at.row + u * at.apart < p.rows) raw[u] = load_codes(codes + u * at.apart * p.ld, steps + u * at.apart * p.ld_s);
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
        if (at.row + u * at.apart >= p.rows) return;
        float v[8];
        decode8(raw[u], v);
        store8(to + u * at.apart * ld_x, p.cols - at.col, out, v);
    }
}

template <typename T, int kAct, bool kGated>
__global__ void __launch_bounds__(kPackThreads) act_grad_kernel(Shape shape, mica_packed p, const T* dy, int64_t ld_dy, T* dx,
                                                                int64_t ld_dx) {
    wait_prerequisite();
    allow_dependents();
    const int64_t F = kGated ? p.cols / 2 : p.cols;
    const Places at(shape, 1, p.rows);
    if (at.col >= F || at.row >= p.rows) return;
    auto codes_at = [&](int64_t col) {
        return load_codes(reinterpret_cast<const int8_t*>(p.codes) + at.row * p.ld + col,
                          reinterpret_cast<const uint8_t*>(p.steps) + at.row * p.ld_s + (col >> 5));
    };
    const RawCodes gate = codes_at(at.col), up = codes_at(kGated ? at.col + F : at.col);
    const Eight<T> g = load8(dy + at.row * ld_dy + at.col, F - at.col, aligned16(dy, ld_dy));
    float v[8], a[8], b[8];
    decode8(gate, v);
    if (kGated) decode8(up, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = g.get(i);
        float y, slope;
        act_of<kAct>(v[i], y, slope);
        a[i] = kGated ? d * b[i] * slope : d * slope;
        b[i] = d * y;
    }
    T* to = dx + at.row * ld_dx + at.col;
    const bool out = aligned16(dx, ld_dx);
    store8(to, F - at.col, out, a);
    if (kGated) store8(to + F, F - at.col, out, b);
}

// Threads of a row: the most, at 32 and more, of which a tenth at most has no columns, else what leaves fewest idle.
Shape shape_of(int64_t cols) {
    const int64_t places = (cols + kBlock - 1) / kBlock * 4;
    int log = 2;
    int64_t least = INT64_MAX;
    for (int k = 8; k >= 2; --k) {
        const int64_t all = ((places + (1 << k) - 1) >> k) << k;
        if (all < least) least = all, log = k;
        if (k >= 5 && all * 10 <= places * 11) break;
    }
    return Shape{log, (int32_t)((places + (1 << log) - 1) >> log)};
}

// Items of a thread, the best of 1 to 8. 16,384 x 6,400 bfloat16, packing with GELU and unpacking: 129 us with 4 and 2 (6.5
// TB/s); with GELU one element at a time 140, 156 with 1 and 2, 149 with 4 and 1, 188 with 8 and 16. The backward pass
// takes one: a gated unit's over 16,384 x 8,192 83 us (6.5 TB/s) with 1, 98 with 2, 113 with 4.
constexpr int kPackItems = 4, kUnpackItems = 2;
constexpr int64_t kManyCtas = 152 * 8;

// `one` item a thread, or `many` (`items`) where that still fills the SMs
template <typename A, typename B, typename... Args>
cudaError_t launch_places(A one, B many, int items, int64_t rows, int64_t cols, void* stream, Args... args) {
    const Shape s = shape_of(cols);
    const int64_t per = kPackThreads >> s.log;
    auto ctas = [&](int items) { return (rows + per * items - 1) / (per * items) * s.tiles; };
    const bool big = ctas(items) >= kManyCtas;
    const int64_t grid = ctas(big ? items : 1);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kPackThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, big ? many : one, s, args...);
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
            return launch_places(pack_kernel<T, MICA_ACT_NONE, false, 1>, pack_kernel<T, MICA_ACT_NONE, false, kPackItems>,
                                 kPackItems, p.rows, F, stream, in, ld_x, p, out, ld_y);
        return by_act(act, [&](auto a) {
            constexpr int k = decltype(a)::value;
            return gated ? launch_places(pack_kernel<T, k, true, 1>, pack_kernel<T, k, true, kPackItems / 2>, kPackItems / 2,
                                         p.rows, F, stream, in, ld_x, p, out, ld_y)
                         : launch_places(pack_kernel<T, k, false, 1>, pack_kernel<T, k, false, kPackItems>, kPackItems,
                                         p.rows, F, stream, in, ld_x, p, out, ld_y);
        });
    });
}

int launch_act_unpack(const mica_packed& p, void* x, int64_t ld_x, void* stream) {
    return by_type(p.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_places(unpack_kernel<T, 1>, unpack_kernel<T, kUnpackItems>, kUnpackItems, p.rows, p.cols, stream, p,
                             static_cast<T*>(x), ld_x);
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
            const auto kernel = gated ? act_grad_kernel<T, k, true> : act_grad_kernel<T, k, false>;
            return launch_places(kernel, kernel, 1, p.rows, F, stream, p, g, ld_dy, d, ld_dx);
        });
    });
}

}  // namespace mica
