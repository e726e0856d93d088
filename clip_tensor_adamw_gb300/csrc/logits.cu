// The losses over logits: log-probabilities, preference and policy losses, and the gradient of the logits.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "mica_optim.h"
#include "plan.h"
#include "train.h"

namespace mica {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFarBelow = -1000.0f;  // an exponent of 2 whose power is 0, and finite (0 * it is 0)

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The running softmax of part of a row, in units of log2: the largest logit, s = sum 2^x and u = sum x 2^x with
// x = (z - m) * inv_t_log2e. A part without a logit above -inf has m == -inf and s == u == 0.
struct Running {
    float m, s, u;
};

// z - m in units of log2; a part that has seen nothing but -inf counts from 0, so that no difference of two infinities
// turns its zero weight into a NaN.
__device__ __forceinline__ float exponent(float z, float m, float a) { return (z - m) * a; }
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

template <bool kEntropy>
__device__ __forceinline__ void add_one(Running& r, float z, float a) {
    if (z > r.m) {  // (never for a NaN)
        const float sh = fmaxf(exponent(r.m, z, a), kFarBelow), f = exp2_fast(sh);
        if (kEntropy) r.u = f * fmaf(r.s, sh, r.u);
        r.s *= f;
        r.m = z;
    }
    const float x = exponent(z, origin(r.m), a), e = exp2_fast(x);
    r.s += e;
    if (kEntropy) r.u = fmaf(e, fmaxf(x, kFarBelow), r.u);
}

template <bool kEntropy>
__device__ __forceinline__ Running join(const Running& p, const Running& q, float a) {
    Running r;
    r.m = fmaxf(p.m, q.m);
    const float o = origin(r.m);
    const float xp = fmaxf(exponent(p.m, o, a), kFarBelow), xq = fmaxf(exponent(q.m, o, a), kFarBelow);
    const float fp = exp2_fast(xp), fq = exp2_fast(xq);
    r.s = fmaf(p.s, fp, q.s * fq);
    r.u = kEntropy ? fmaf(fp, fmaf(p.s, xp, p.u), fq * fmaf(q.s, xq, q.u)) : 0.0f;
    return r;
}

template <bool kEntropy>
__device__ __forceinline__ Running block_join(Running r, float a, Running* shared) {
    for (int d = 16; d > 0; d >>= 1) {
        Running q;
        q.m = __shfl_xor_sync(~0u, r.m, d);
        q.s = __shfl_xor_sync(~0u, r.s, d);
        q.u = kEntropy ? __shfl_xor_sync(~0u, r.u, d) : 0.0f;
        r = join<kEntropy>(r, q, a);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x / 32] = r;
    __syncthreads();
    r = shared[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) r = join<kEntropy>(r, shared[w], a);
    return r;
}

__device__ __forceinline__ int64_t target_of(const LogitRows& L, int64_t row) {
    return L.wide_targets ? reinterpret_cast<const int64_t*>(L.targets)[row]
                          : (int64_t) reinterpret_cast<const int32_t*>(L.targets)[row];
}

// (z_y - zmax) / temperature - log(s); NaN for a target past the vocabulary
template <typename T>
__device__ __forceinline__ float logp_of(const LogitRows& L, const T* z, int64_t y, const Running& r) {
    if (y >= L.vocab) return NAN;
    return (widen(z[y]) - origin(r.m)) * L.inv_t - logf(r.s);
}

template <typename T, bool kEntropy>
__device__ Running row_softmax(const LogitRows& L, const T* z, Running* shared) {
    Running r{-INFINITY, 0.0f, 0.0f};
    for (int j = threadIdx.x; j < L.vocab; j += blockDim.x) add_one<kEntropy>(r, widen(z[j]), L.inv_t_log2e);
    return block_join<kEntropy>(r, L.inv_t_log2e, shared);
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kRowThreads) row_logps_kernel(LogitRows L, float* logps, float* entropy, RowStat* stat) {
    __shared__ Running shared[kRowThreads / 32];
    for (int64_t row = blockIdx.x; row < L.rows; row += gridDim.x) {
        const int64_t y = target_of(L, row);
        if (y < 0) {
            if (threadIdx.x == 0) {
                logps[row] = 0.0f;
                if (kEntropy) entropy[row] = 0.0f;
            }
            continue;
        }
        const T* z = reinterpret_cast<const T*>(L.z) + row * L.ld;
        const Running r = row_softmax<T, kEntropy>(L, z, shared);
        if (threadIdx.x == 0) {
            logps[row] = logp_of(L, z, y, r);
            if (kEntropy) entropy[row] = logf(r.s) - kLn2 * r.u / r.s;
            if (stat) stat[row] = RowStat{r.m, 1.0f / r.s};
        }
    }
}

// dz = c * ((j == y) - p) over the row; c == 0 gives zeros
template <typename T>
__device__ void write_grad(const LogitRows& L, const T* z, int64_t y, float zmax, float inv_sum, float c, T* dz) {
    const float o = origin(zmax), k = -c * inv_sum;
    for (int j = threadIdx.x; j < L.vocab; j += blockDim.x) {
        float d = 0.0f;
        if (c != 0.0f) {
            const float e = exp2_fast(exponent(widen(z[j]), o, L.inv_t_log2e));
            d = j == y ? c * (1.0f - e * inv_sum) : k * e;
        }
        dz[j] = narrow<T>(d);
    }
}

__device__ __forceinline__ float policy_coef(const PolicyTerms& P, int64_t row, float lp) {
    const float A = P.advantages[row], r = expf(lp - P.old_logps[row]);
    const float plain = r * A, held = fminf(fmaxf(r, P.lo), P.hi) * A;
    float slope = held < plain ? 0.0f : -plain;
    if (P.ref_logps) slope += P.kl_coef * -expm1f(P.ref_logps[row] - lp);
    return slope * (P.weights ? P.weights[row] : 1.0f) * P.grad_factor;
}

enum CoefKind { kGiven, kPolicy };

template <typename T, CoefKind kKind>
__global__ void __launch_bounds__(kRowThreads) row_loss_grad_kernel(LogitRows L, PolicyTerms P, const float* coef,
                                                                    float factor, float* logps, T* dz, int64_t ld_d) {
    __shared__ Running shared[kRowThreads / 32];
    for (int64_t row = blockIdx.x; row < L.rows; row += gridDim.x) {
        const int64_t y = target_of(L, row);
        const T* z = reinterpret_cast<const T*>(L.z) + row * L.ld;
        T* d = dz + row * ld_d;
        float c = 0.0f;
        Running r{0.0f, 1.0f, 0.0f};
        if (kKind == kGiven && y >= 0) c = coef[row] * factor;
        if (y >= 0 && (kKind == kPolicy || c != 0.0f)) {
            r = row_softmax<T, false>(L, z, shared);
            const float lp = logp_of(L, z, y, r);
            if (kKind == kPolicy) c = policy_coef(P, row, lp);
            if (y >= L.vocab) c = NAN;
            if (kKind == kPolicy && threadIdx.x == 0) logps[row] = lp;
        } else if (kKind == kPolicy && threadIdx.x == 0) {
            logps[row] = 0.0f;
        }
        __syncthreads();  // in place: every thread has read the target's logit
        write_grad(L, z, y, r.m, 1.0f / r.s, c, d);
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) row_grad_kernel(LogitRows L, const RowStat* stat, const float* coef, T* dz,
                                                               int64_t ld_d) {
    for (int64_t row = blockIdx.x; row < L.rows; row += gridDim.x) {
        const int64_t y = target_of(L, row);
        float c = y < 0 ? 0.0f : coef[row];
        if (y >= L.vocab) c = NAN;
        RowStat s{0.0f, 1.0f};
        if (c != 0.0f) s = stat[row];
        write_grad(L, reinterpret_cast<const T*>(L.z) + row * L.ld, y, s.zmax, s.inv_sum, c, dz + row * ld_d);
    }
}

// ----------------------------------------------------------------------------------------------------------------------
// per-token and per-pair terms
// ----------------------------------------------------------------------------------------------------------------------

constexpr int kSumThreads = 1024;

__device__ __forceinline__ double warp_sum(double x) {
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

__device__ double block_sum_ordered(double x, double* shared) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x / 32] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += shared[w];
    return s;
}

__global__ void __launch_bounds__(kSumThreads) policy_sums_kernel(LogitRows L, PolicyTerms P, const float* logps,
                                                                  float* stats) {
    __shared__ double shared[kSumThreads / 32];
    double sl = 0.0, sk = 0.0, sc = 0.0;
    for (int64_t row = threadIdx.x; row < L.rows; row += blockDim.x) {
        if (target_of(L, row) < 0) continue;
        const float lp = logps[row], A = P.advantages[row], r = expf(lp - P.old_logps[row]);
        const float plain = r * A, held = fminf(fmaxf(r, P.lo), P.hi) * A;
        const double w = P.weights ? P.weights[row] : 1.0;
        sl -= w * (held < plain ? held : plain);
        sc += held < plain ? w : 0.0;
        if (P.ref_logps) {
            const float q = P.ref_logps[row] - lp;
            sk += w * (double)(expm1f(q) - q);
        }
    }
    sl = block_sum_ordered(sl, shared) * P.inv_denom;
    sk = block_sum_ordered(sk, shared) * P.inv_denom;
    sc = block_sum_ordered(sc, shared) * P.inv_denom;
    if (threadIdx.x == 0) {
        stats[0] = (float)(P.ref_logps ? sl + P.kl_coef * sk : sl);
        stats[1] = (float)sl;
        stats[2] = (float)sk;
        stats[3] = (float)sc;
    }
}

__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

__device__ __forceinline__ int64_t clamp_row(int64_t x, int64_t rows) { return x < 0 ? 0 : x > rows ? rows : x; }

// One CTA: each warp sums its sequences; then the threads take the pairs' losses and slopes; then each warp writes its
// sequences' coefficients. sums[s] holds a sequence's sum, then its rows' coefficient.
__global__ void __launch_bounds__(kSumThreads) pairs_kernel(LogitRows L, PairTerms P, const float* logps, double* sums,
                                                            float* loss, float* rewards, float* coef) {
    __shared__ double shared[kSumThreads / 32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, warps = blockDim.x / 32;
    if (coef)
        for (int64_t row = threadIdx.x; row < L.rows; row += blockDim.x) coef[row] = 0.0f;
    auto count_of = [&](int64_t a, int64_t b) {
        int n = 0;
        for (int64_t row = a + lane; row < b; row += 32) n += target_of(L, row) >= 0;
        return __reduce_add_sync(~0u, n);
    };
    for (int s = warp; s < 2 * P.pairs; s += warps) {
        const int64_t a = clamp_row(P.cu_seqlens[s], L.rows), b = clamp_row(P.cu_seqlens[s + 1], L.rows);
        double d = 0.0;
        for (int64_t row = a + lane; row < b; row += 32)
            if (target_of(L, row) >= 0) d += (double)logps[row] - (P.ref_logps ? (double)P.ref_logps[row] : 0.0);
        d = warp_sum(d);
        if (P.length_norm) {
            const int n = count_of(a, b);
            d /= n > 0 ? n : 1;
        }
        if (lane == 0) {
            sums[s] = d;
            if (rewards) rewards[s] = (float)(P.beta * d);
        }
    }
    __syncthreads();
    double mine = 0.0;
    for (int p = threadIdx.x; p < P.pairs; p += blockDim.x) {
        const double d = sums[2 * p] - sums[2 * p + 1], h = P.beta * d;
        double l, slope;  // the pair's loss and its derivative by d
        if (P.kind == MICA_PREF_SIGMOID) {
            l = (1.0 - P.smoothing) * softplus(-h) + (P.smoothing > 0.0 ? P.smoothing * softplus(h) : 0.0);
            slope = P.beta * (-(1.0 - P.smoothing) / (1.0 + exp(h)) + P.smoothing / (1.0 + exp(-h)));
        } else if (P.kind == MICA_PREF_HINGE) {
            l = h < 1.0 ? 1.0 - h : (h >= 1.0 ? 0.0 : h);  // (a NaN stays one)
            slope = h < 1.0 ? -P.beta : (h >= 1.0 ? 0.0 : h);
        } else {
            const double gap = d - 0.5 / P.beta;
            l = gap * gap;
            slope = 2.0 * gap;
        }
        mine += l;
        sums[2 * p] = slope * P.grad_factor;
        sums[2 * p + 1] = -slope * P.grad_factor;
    }
    const double total = block_sum_ordered(mine, shared);
    if (threadIdx.x == 0) *loss = P.pairs ? (float)(total / P.pairs) : 0.0f;
    if (!coef) return;
    for (int s = warp; s < 2 * P.pairs; s += warps) {
        const int64_t a = clamp_row(P.cu_seqlens[s], L.rows), b = clamp_row(P.cu_seqlens[s + 1], L.rows);
        double c = sums[s];
        if (P.length_norm) {
            const int n = count_of(a, b);
            c /= n > 0 ? n : 1;
        }
        for (int64_t row = a + lane; row < b; row += 32) coef[row] = (float)c;
    }
}

unsigned grid_for(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

template <typename F>
int by_type(int32_t dtype, F f) {
    if (dtype == MICA_F32) f(float{});
    else if (dtype == MICA_F16) f(__half{});
    else f(__nv_bfloat16{});
    count_launches(1);
    return (int)cudaGetLastError();
}

}  // namespace

int launch_row_logps(const LogitRows& L, float* logps, float* entropy, RowStat* stat, void* stream) {
    return by_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (entropy) row_logps_kernel<T, true><<<grid_for(L.rows), kRowThreads, 0, st>>>(L, logps, entropy, stat);
        else row_logps_kernel<T, false><<<grid_for(L.rows), kRowThreads, 0, st>>>(L, logps, nullptr, stat);
    });
}

int launch_row_softmax_grad(const LogitRows& L, const float* coef, float factor, void* dz, int64_t ld_d, void* stream) {
    return by_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        row_loss_grad_kernel<T, kGiven><<<grid_for(L.rows), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            L, PolicyTerms{}, coef, factor, nullptr, static_cast<T*>(dz), ld_d);
    });
}

int launch_row_policy_grad(const LogitRows& L, const PolicyTerms& P, float* logps, void* dz, int64_t ld_d, void* stream) {
    return by_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        row_loss_grad_kernel<T, kPolicy><<<grid_for(L.rows), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            L, P, nullptr, 0.0f, logps, static_cast<T*>(dz), ld_d);
    });
}

int launch_row_grad(const LogitRows& L, const RowStat* stat, const float* coef, void* dz, int64_t ld_d, void* stream) {
    return by_type(L.dtype, [&](auto t) {
        using T = decltype(t);
        row_grad_kernel<T><<<grid_for(L.rows), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            L, stat, coef, static_cast<T*>(dz), ld_d);
    });
}

int launch_policy_sums(const LogitRows& L, const PolicyTerms& P, const float* logps, float* stats, void* stream) {
    policy_sums_kernel<<<1, kSumThreads, 0, static_cast<cudaStream_t>(stream)>>>(L, P, logps, stats);
    count_launches(1);
    return (int)cudaGetLastError();
}

int launch_pairs(const LogitRows& L, const PairTerms& P, const float* logps, double* sums, float* loss, float* rewards,
                 float* coef, void* stream) {
    pairs_kernel<<<1, kSumThreads, 0, static_cast<cudaStream_t>(stream)>>>(L, P, logps, sums, loss, rewards, coef);
    count_launches(1);
    return (int)cudaGetLastError();
}

}  // namespace mica
