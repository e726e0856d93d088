// A linear layer's weight gradient from its input's 8-bit checkpoint: dw = add + x^T dy.
#include <cuda_runtime.h>

#include <cstdint>

#include "packed.cuh"
#include "plan.h"
#include "train.h"

namespace mica {
namespace {

constexpr int kTile = 64, kDepth = 16, kSimpleThreads = 256;

// One CTA per 64 x 64 tile of dw, each thread 4 x 4 of it, 16 tokens at a time through shared memory.
template <typename T, typename O>
__global__ void __launch_bounds__(kSimpleThreads) wgrad_simple_kernel(Wgrad w) {
    __shared__ float xs[kDepth][kTile], ys[kDepth][kTile];
    const int64_t i0 = (int64_t)blockIdx.y * kTile, j0 = (int64_t)blockIdx.x * kTile;
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    const T* dy = static_cast<const T*>(w.dy);
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < w.x.rows; t0 += kDepth) {
        for (int k = threadIdx.x; k < kDepth * kTile; k += kSimpleThreads) {
            const int64_t t = t0 + k / kTile, i = i0 + k % kTile, j = j0 + k % kTile;
            float x = 0.0f, y = 0.0f;
            if (t < w.x.rows && i < w.x.cols)
                x = (float)reinterpret_cast<const int8_t*>(w.x.codes)[t * w.x.ld + i] *
                    step_value(reinterpret_cast<const uint8_t*>(w.x.steps)[t * w.x.ld_s + i / kBlock]);
            if (t < w.x.rows && j < w.n) y = widen(dy[t * w.ld_dy + j]);
            xs[k / kTile][k % kTile] = x;
            ys[k / kTile][k % kTile] = y;
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(xs[k][ti + a], ys[k][tj + b], acc[a][b]);
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t i = i0 + ti + a, j = j0 + tj + b;
            if (i >= w.x.cols || j >= w.n) continue;
            float v = acc[a][b];
            if (w.add) v += widen(static_cast<const O*>(w.add)[i * w.ld_add + j]);
            static_cast<O*>(w.dw)[i * w.ld_dw + j] = narrow<O>(v);
        }
}

template <typename T>
void launch_simple(const Wgrad& w, cudaStream_t st) {
    const dim3 grid((unsigned)((w.n + kTile - 1) / kTile), (unsigned)((w.x.cols + kTile - 1) / kTile));
    if (w.dw_dtype == MICA_F32) wgrad_simple_kernel<T, float><<<grid, kSimpleThreads, 0, st>>>(w);
    else if (w.dw_dtype == MICA_F16) wgrad_simple_kernel<T, __half><<<grid, kSimpleThreads, 0, st>>>(w);
    else wgrad_simple_kernel<T, __nv_bfloat16><<<grid, kSimpleThreads, 0, st>>>(w);
}

}  // namespace

int64_t wgrad_workspace(int64_t, int64_t, int64_t, int) { return 0; }

int launch_wgrad(const Wgrad& w, void*, int, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (w.dy_dtype == MICA_F16) launch_simple<__half>(w, st);
    else launch_simple<__nv_bfloat16>(w, st);
    count_launches(1);
    return (int)cudaGetLastError();
}

}  // namespace mica
