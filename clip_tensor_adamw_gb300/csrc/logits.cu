// The losses over logits: log-probabilities, preference and policy losses, and the gradient of the logits.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "mica_optim.h"
#include "pipe.cuh"
#include "plan.h"
#include "stream.cuh"
#include "train.h"

namespace mica {
namespace {

constexpr int kRowThreads = 256, kShortThreads = 64;  // of a CTA; of one for short rows
constexpr int kRowResident = 1280;                    // of the CTAs of an SM
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMostCluster = 8;  // CTAs of a portable cluster
constexpr int kBatch = 4;        // vectors of a thread in flight
constexpr int64_t kFewCtas = 608;  // (100 rows of 50,257 logits: 16.3 us a call with 608, 19.2 with 304, 17.1 with 1,216)
constexpr double kLn2 = 0.693147180559945309;
constexpr float kFarBelow = -1000.0f;  // an exponent of 2 whose power is 0, and finite (0 * it is 0)
// How much the hardware's 2^x is low on average, of its value, for x < -1 (-2e-8 from there to 0, +3e-8 above 1, exact for
// whole x): every log-probability of a sequence would be as much too high, and a sequence's sum has hundreds.
constexpr double kLow = 5.0e-8;

// ----------------------------------------------------------------------------------------------------------------------
// rows
// ----------------------------------------------------------------------------------------------------------------------
//
// The softmax of a row of logits and, where the gradient c * ((j == y) - p_j) is wanted, that too: its coefficient c
// depends on nothing but the row, so the row is read again and its gradient written while it is still in L2 (the rows in
// work together are some 60 MB, half of it). Traffic with memory is one read, or one read and one write, which is what
// bounds it. Each thread keeps a running maximum and sum over its vectors of 16 bytes, kBatch of them in flight; a warp
// joins its threads', and one barrier joins the warps'. Where there are few rows, a cluster of CTAs shares each, and its
// CTAs read one another's shared memory.
//
// This serves few rows and short ones; see the ring below for the others. Rows held in the registers of a cluster, read
// once from L2 too, took 295 us where this took 116 (8,192 rows of 50,257 bfloat16 logits): the share of a thread was so
// small that the joins were most of its work.
//
// Vectors start at 16-byte addresses, whatever the row's alignment (an odd vocabulary puts each row elsewhere): the first
// and the last may reach outside the row, and are then read and written element by element, the rest as -inf.

// z[j] - origin in units of log2, 2^that being the weight: a = log2(e) / temperature split in two floats, since the relative
// error of one alone (up to 2^-24) would shift every log-probability of a sequence the same way. a_lo > 0 (the host sees
// to it), so that a banned token's -inf stays -inf.
__device__ __forceinline__ float exponent(const LogitRows& L, float z, float origin) {
    const float d = z - origin;
    return fmaf(d, L.a_hi, d * L.a_lo);
}

// A part that has seen nothing but -inf counts from 0, so that no difference of two infinities makes its zero weight a NaN.
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

// The softmax of part of a row: the logit that the weights are counted from (-inf: nothing above that yet), s = sum 2^x and
// u = sum x 2^x, x the exponents.
struct Running {
    float m, s, u;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
    return x;
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float peer_load(const float* p, uint32_t rank) {
    uint32_t at;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

template <typename T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ float get(int i) const {  // i is a constant after unrolling
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        else return __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (16 * (i % 2)))));
    }
    __device__ __forceinline__ Two pair(int i) const { return two(get(2 * i), get(2 * i + 1)); }
    template <int kCount>
    __device__ __forceinline__ static float max(const Vec (&v)[kCount]) {
        if constexpr (sizeof(T) == 4) {
            float m = v[0].get(0);
#pragma unroll
            for (int i = 1; i < kCount * n; ++i) m = fmaxf(m, v[i / n].get(i % n));
            return m;
        } else {
            using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
            const T2* p = reinterpret_cast<const T2*>(v);
            T2 m = p[0];
#pragma unroll
            for (int i = 1; i < kCount * 4; ++i) m = __hmax2(m, p[i]);
            return fmaxf(widen(m.x), widen(m.y));
        }
    }
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __half2 p = __floats2half2_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    __device__ __forceinline__ static Vec of(const float (&x)[n]) {
        Vec v;
        if constexpr (sizeof(T) == 4)
            v.raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else v.raw = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
        return v;
    }
};

// Where a row's 16-byte vectors lie: vector k holds elements [k * n - lead, k * n - lead + n). Of a CTA's vectors those in
// [lo, hi) lie inside the row; the row's first or last, where it reaches outside, is `edge` of thread 0 or 1 (else -1).
struct RowVectors {
    int lead, lo, hi, edge;
};

template <typename T>
__device__ __forceinline__ RowVectors row_vectors(const T* z, int vocab) {
    constexpr int n = Vec<T>::n;
    const int lead = (int)(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T)), total = (lead + vocab + n - 1) / n;
    const int C = (int)cluster_size(), per = (total + C - 1) / C, first = min((int)cluster_rank() * per, total);
    const int end = min(first + per, total), open = lead > 0, closed = (lead + vocab) / n;  // whole ones: [open, closed)
    int edge = -1;
    if (threadIdx.x == 0 && open && first == 0) edge = 0;
    if (threadIdx.x == 1 && closed < total && first < total && end == total && !(open && total == 1)) edge = total - 1;
    return RowVectors{lead, max(first, open), min(end, closed), edge};
}

// 16 bytes that are read again soon: past L1, and kept in L2
__device__ __forceinline__ uint4 ld16_again(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// An edge vector, from the element j0 (which may be before the row) on; -inf outside the row.
template <typename T>
__device__ __forceinline__ Vec<T> load_edge(const T* z, int j0, int vocab) {
    constexpr int n = Vec<T>::n;
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = j0 + i >= 0 && j0 + i < vocab ? widen(z[j0 + i]) : -INFINITY;
    return Vec<T>::of(x);  // (exact: each element is one of T)
}

template <typename T>
__device__ __forceinline__ void store_some(T* dz, int j0, int vocab, const float (&x)[Vec<T>::n]) {
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i)
        if (j0 + i >= 0 && j0 + i < vocab) dz[j0 + i] = narrow<T>(x[i]);
}

__device__ __forceinline__ int64_t target_of(const LogitRows& L, int64_t row) {
    return L.wide_targets ? reinterpret_cast<const int64_t*>(L.targets)[row]
                          : (int64_t) reinterpret_cast<const int32_t*>(L.targets)[row];
}

// What a launch over rows is for: log-probabilities (with entropies), or the gradient with the coefficient given, or with
// the policy loss's, computed from the log-probability.
enum RowKind { kLogps, kEntropy, kGiven, kPolicy };

struct RowOut {
    float* logps;         // kLogps, kEntropy, kPolicy
    float* rest_logps;    // kLogps, or null: what rounding took from the log-probabilities
    float* entropy;       // kEntropy
    RowStat* stat;        // kLogps, or null
    const float* coef;    // kGiven
    float factor;         // kGiven: the coefficient is coef * factor
    void* dz;
    int64_t ld_d;
};

__device__ __forceinline__ float policy_coef(const PolicyTerms& P, int64_t row, float lp) {
    const float A = P.advantages[row], r = expf(lp - P.old_logps[row]);
    const float plain = r * A, held = fminf(fmaxf(r, P.lo), P.hi) * A;
    float slope = held < plain ? 0.0f : -plain;
    if (P.ref_logps) slope += P.kl_coef * -expm1f(P.ref_logps[row] - lp);
    return slope * (P.weights ? P.weights[row] : 1.0f) * P.grad_factor;
}

// Zeros over the CTA's part of a row. `same`: the row of dz is aligned as that of z is.
template <typename T, int kThreads>
__device__ __forceinline__ void zero_row(const RowVectors& g, int vocab, T* dz, bool same) {
    constexpr int n = Vec<T>::n;
    const float zero[n] = {};
    if (g.edge >= 0) store_some(dz, g.edge * n - g.lead, vocab, zero);
    for (int k = g.lo + (int)threadIdx.x; k < g.hi; k += kThreads) {
        if (same) st16(dz + (k * n - g.lead), make_uint4(0, 0, 0, 0));
        else store_some(dz, k * n - g.lead, vocab, zero);
    }
}

// What the gradient of a row takes: p = inv * 2^exponent, counted from o; c its coefficient.
struct RowGrad {
    float o, c, inv;
    int at;  // the target, or -16
};

// The weights' exponents of two elements, counted from -away, as the statistics were taken with. (One float for log2(e) /
// temperature would put the weight of a row's likeliest token, and so 1 - p, off by up to 2^-24 of its exponent against the
// sum that has it; the rounding to 16 bits hides that, so there one product less is taken.)
template <typename T>
__device__ __forceinline__ Two exponents(const LogitRows& L, Two z, Two away) {
    const Two d = z + away;
    if constexpr (sizeof(T) == 4) return fma2(d, two(L.a_hi, L.a_hi), d * two(L.a_lo, L.a_lo));
    else return d * two(L.a, L.a);
}

// One vector of the gradient c * ((j == y) - p), from the element j0 on.
template <typename T>
__device__ __forceinline__ void grad_values(const LogitRows& L, const Vec<T>& v, const RowGrad& q, int j0,
                                            float (&d)[Vec<T>::n]) {
    constexpr int n = Vec<T>::n;
    const float k = -q.c * q.inv;
    const Two away = two(-q.o, -q.o), kk = two(k, k);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const float2 x = each(exponents<T>(L, v.pair(i), away));
        const float2 e = each(two(exp2_fast(x.x), exp2_fast(x.y)) * kk);
        d[2 * i] = e.x;
        d[2 * i + 1] = e.y;
    }
    if ((unsigned)(q.at - j0) < (unsigned)n) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (j0 + i == q.at) d[i] = q.c * (1.0f - q.inv * exp2_fast(each(exponents<T>(L, two(v.get(i), 0.0f), away)).x));
    }
}

template <typename T>
__device__ __forceinline__ void grad_vector(const LogitRows& L, const Vec<T>& v, const RowGrad& q, int j0, T* dz, bool same) {
    float d[Vec<T>::n];
    grad_values(L, v, q, j0, d);
    if (same) st16(dz + j0, Vec<T>::of(d).raw);
    else store_some(dz, j0, L.vocab, d);
}

// The CTA's part of a row's gradient, the statistics known.
template <typename T, int kThreads>
__device__ __forceinline__ void grad_row(const LogitRows& L, const T* z, const RowVectors& g, const RowGrad& q, T* dz,
                                         bool same) {
    constexpr int n = Vec<T>::n;
    if (g.edge >= 0) {
        const int j0 = g.edge * n - g.lead;
        float d[n];
        grad_values(L, load_edge(z, j0, L.vocab), q, j0, d);
        store_some(dz, j0, L.vocab, d);
    }
    int k = g.lo + (int)threadIdx.x;
    for (; k + (kBatch - 1) * kThreads < g.hi; k += kBatch * kThreads) {
        const int j0 = k * n - g.lead;
        Vec<T> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = Vec<T>{ld16_stream(z + j0 + u * kThreads * n)};
#pragma unroll
        for (int u = 0; u < kBatch; ++u) grad_vector(L, v[u], q, j0 + u * kThreads * n, dz, same);
    }
    for (; k < g.hi; k += kThreads) {
        const int j0 = k * n - g.lead;
        grad_vector(L, Vec<T>{ld16_stream(z + j0)}, q, j0, dz, same);
    }
}

// The sum of some vectors' weights, counted from o, and of their moments. kAnything: with banned tokens among them (whose
// zero weights would make a moment of 0 * -inf).
template <typename T, bool kMoment, bool kAnything, int kCount>
__device__ __forceinline__ void sum_weights(const LogitRows& L, const Vec<T> (&v)[kCount], float o, float& s, float& u) {
    const Two away = two(-o, -o), hi = two(L.a_hi, L.a_hi), lo = two(L.a_lo, L.a_lo);
    Two sv = two(0.0f, 0.0f), uv = two(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kCount; ++j)
#pragma unroll
        for (int i = 0; i < Vec<T>::n / 2; ++i) {
            const Two d = v[j].pair(i) + away;
            Two xx = fma2(d, hi, d * lo);
            float2 x = each(xx);
            const Two e = two(exp2_fast(x.x), exp2_fast(x.y));
            sv = sv + e;
            if (kMoment && kAnything) xx = two(fmaxf(x.x, kFarBelow), fmaxf(x.y, kFarBelow));
            if (kMoment) uv = fma2(e, xx, uv);
        }
    const float2 t = each(sv), w = each(uv);
    s = t.x + t.y;
    u = w.x + w.y;
}

// 2^x for the factor of a part that is counted anew, x <= 0: from the nearest integer, whose power the hardware has exactly,
// and what remains of x, where its error is 1e-8 on average (see kLow) and not the same way for every part.
__device__ __forceinline__ float exp2_factor(float x) {
    const float i = (x + 12582912.0f) - 12582912.0f;  // 1.5 * 2^23
    return exp2_fast(i) * exp2_fast(x - i);
}

// Counts a part from `m` instead, a larger origin.
template <bool kMoment>
__device__ __forceinline__ void raise(const LogitRows& L, Running& r, float m) {
    const float x = fmaxf(exponent(L, r.m, m), kFarBelow), f = exp2_factor(x);
    if (kMoment) r.u = f * fmaf(r.s, x, r.u);
    r.s *= f;
    r.m = m;
}

// Counts a part from m, the largest of some vectors that it is about to take, where that is larger. Log-probabilities with
// entropies are counted so throughout: an entropy is log s, which is then not negative, plus the mean of -x, which is not
// either. Counted from a target far below the maximum it would be the difference of two numbers as large as that distance,
// in float32, and of a confident row little is left (20 nats: 1e-6 off, and below 0). The comparisons cost up to 7% (8,192
// rows of 50,257 bfloat16 logits, of which 6,144 count, with entropies: 104 us, counted from the target 100; 117 with the
// weights counted from the target and the moment from the maximum). Without entropies they are made too, so that the
// log-probabilities are the same bits.
template <bool kMoment>
__device__ __forceinline__ void count_from_highest(const LogitRows& L, float m, Running& r) {
    if (r.s == 0.0f) r.m = fmaxf(r.m, m);  // nothing to scale (a NaN target is in the sum by itself)
    else if (m > r.m) raise<kMoment>(L, r, m);
}

// Adds some vectors to a thread's part. Weights are counted from an origin that need not be the maximum: any will do as long
// as one weight of the row is at least 1 and none comes near 2^128. So for a gradient the target's logit serves, until a sum
// passes 2^60; the elements are compared only then (and where the target is banned, or an infinity or a NaN is among them).
template <typename T, bool kMoment, int kCount>
__device__ __forceinline__ void add_vectors(const LogitRows& L, const Vec<T> (&v)[kCount], Running& r) {
    float s, u;
    sum_weights<T, kMoment, false>(L, v, r.m, s, u);
    if (!(s < 0x1p60f) || (kMoment && !(fabsf(u) < 0x1p100f))) {
        const float m = Vec<T>::max(v);
        if (!(s < 0x1p60f) && m > r.m) raise<kMoment>(L, r, m);
        sum_weights<T, kMoment, true>(L, v, origin(r.m), s, u);
    }
    r.s += s;
    if (kMoment) r.u += u;
}

struct Parts {
    Running warp[kRowWarps];
    Running cta;
};

// The lanes' parts as one, in all lanes alike.
template <bool kMoment>
__device__ __forceinline__ Running join_warp(const LogitRows& L, const Running& p) {
    Running r;
    r.m = warp_max(p.m);
    const float x = fmaxf(exponent(L, p.m, origin(r.m)), kFarBelow), f = exp2_factor(x);
    r.s = warp_add(p.s * f);
    r.u = kMoment ? warp_add(f * fmaf(p.s, x, p.u)) : 0.0f;
    return r;
}

// Joins the parts of all threads of the cluster, in every thread alike. Where the cluster has other CTAs, leave_cluster()
// has to follow before the CTA ends.
template <bool kMoment>
__device__ __forceinline__ Running join_parts(const LogitRows& L, Parts& parts, Running r) {
    const int C = (int)cluster_size(), warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = (int)blockDim.x / 32;
    const Running none{-INFINITY, 0.0f, 0.0f};
    r = join_warp<kMoment>(L, r);
    if (warps > 1) {
        if (lane == 0) parts.warp[warp] = r;
        __syncthreads();
        if (C == 1 || warp == 0) r = join_warp<kMoment>(L, lane < warps ? parts.warp[lane] : none);
    }
    if (C > 1) {
        if (threadIdx.x == 0) parts.cta = r;
        cluster_arrive();
        cluster_wait();
        r = none;
        if (lane < C) r = Running{peer_load(&parts.cta.m, lane), peer_load(&parts.cta.s, lane),
                                  kMoment ? peer_load(&parts.cta.u, lane) : 0.0f};
        cluster_arrive();  // what leave_cluster() waits for: no more reads of the others' shared memory
        r = join_warp<kMoment>(L, r);
    }
    return r;
}

__device__ __forceinline__ void leave_cluster() {
    if (cluster_size() > 1) cluster_wait();
}

// A row that does not count.
template <RowKind kKind>
__device__ __forceinline__ void skip_outputs(const RowOut& out, int64_t row) {
    if (kKind == kGiven || threadIdx.x != 0 || cluster_rank() != 0) return;
    out.logps[row] = 0.0f;
    if (kKind == kLogps && out.rest_logps) out.rest_logps[row] = 0.0f;
    if (kKind == kEntropy) out.entropy[row] = 0.0f;
}

// log(s) to some 2^-25 absolutely: the exponent's part in float64, and that of the fraction, which is below 0.7, in
// float32. (float64's own log took 3 us of a row's 12: this chip has next to no float64.)
__device__ __forceinline__ double wide_log(float s) {
    const uint32_t bits = __float_as_uint(s);
    if (!(s >= 0x1p-126f && s < INFINITY)) return logf(s);
    // (kLow is of the share that is not the largest weight's, which is exactly 1: to within 3e-8)
    return fma((double)((int)(bits >> 23) - 127), kLn2, s < 1.5f ? 0.0 : kLow) +
           logf(__uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u));
}

// Writes a row's results (one thread, `head`) and returns the gradient's coefficient, c itself where it was given, in every
// thread alike. zy: the target's logit.
template <RowKind kKind>
__device__ __forceinline__ float finish_row(const LogitRows& L, const PolicyTerms& P, const RowOut& out, int64_t row,
                                            int64_t y, float zy, const Running& r, float c, bool head) {
    const float o = origin(r.m);
    if constexpr (kKind == kLogps || kKind == kEntropy) {
        if (head) {
            const double log_sum = wide_log(r.s);
            const double lp = y < L.vocab ? ((double)zy - o) * L.wide_inv_t - log_sum : NAN;
            out.logps[row] = (float)lp;
            if (kKind == kLogps && out.rest_logps) out.rest_logps[row] = isfinite(lp) ? (float)(lp - (float)lp) : 0.0f;
            if (kKind == kEntropy) out.entropy[row] = (float)(log_sum - kLn2 * (r.u / r.s));
            if (kKind == kLogps && out.stat) out.stat[row] = RowStat{r.m, 1.0f / r.s};
        }
    }
    if constexpr (kKind == kPolicy) {
        const float lp = y < L.vocab ? fmaf(zy - o, L.inv_t, -logf(r.s)) : NAN;
        c = policy_coef(P, row, lp);
        if (head) out.logps[row] = lp;
    }
    return y < L.vocab ? c : NAN;
}

template <typename T, int kThreads, RowKind kKind>
__global__ void __launch_bounds__(kThreads, kRowResident / kThreads) row_kernel(LogitRows L, PolicyTerms P, RowOut out) {
    constexpr int n = Vec<T>::n;
    constexpr bool kGrad = kKind == kGiven || kKind == kPolicy, kMoment = kKind == kEntropy, kHighest = !kGrad;
    __shared__ Parts parts;
    wait_prerequisite();
    allow_dependents();
    const int64_t row = blockIdx.x / cluster_size();
    const T* z = reinterpret_cast<const T*>(L.z) + row * L.ld;
    T* dz = kGrad ? reinterpret_cast<T*>(out.dz) + row * out.ld_d : nullptr;
    const bool same = kGrad && (reinterpret_cast<uintptr_t>(dz) - reinterpret_cast<uintptr_t>(z)) % 16 == 0;
    const RowVectors g = row_vectors(z, L.vocab);
    const int64_t y = target_of(L, row);
    float c = kKind == kGiven && y >= 0 ? out.coef[row] * out.factor : 0.0f;
    if (y < 0 || (kKind == kGiven && c == 0.0f)) {  // a row that does not count is not read (every CTA of the cluster alike)
        if (kGrad) zero_row<T, kThreads>(g, L.vocab, dz, same);
        skip_outputs<kKind>(out, row);
        return;
    }
    const float zy = y < L.vocab ? widen(z[y]) : -INFINITY;  // (read before the join, after which dz may be written over z)
    Running r{zy, 0.0f, 0.0f};
    int k = g.lo + (int)threadIdx.x;
    for (; k + (kBatch - 1) * kThreads < g.hi; k += kBatch * kThreads) {
        const T* at = z + (k * n - g.lead);
        Vec<T> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            v[u] = Vec<T>{kGrad ? ld16_again(at + u * kThreads * n) : ld16_stream(at + u * kThreads * n)};
        if (kHighest) count_from_highest<kMoment>(L, Vec<T>::max(v), r);
        add_vectors<T, kMoment>(L, v, r);
    }
    if constexpr (kHighest) {  // fewer than a batch are left
        Vec<T> v[kBatch - 1];
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < kBatch - 1; ++u)
            if (k + u * kThreads < g.hi) v[u] = Vec<T>{ld16_stream(z + ((k + u * kThreads) * n - g.lead))};
#pragma unroll
        for (int u = 0; u < kBatch - 1; ++u)
            if (k + u * kThreads < g.hi) m = fmaxf(m, Vec<T>::max({v[u]}));
        count_from_highest<kMoment>(L, m, r);
#pragma unroll
        for (int u = 0; u < kBatch - 1; ++u)
            if (k + u * kThreads < g.hi) add_vectors<T, kMoment>(L, {v[u]}, r);
    } else {
        for (; k < g.hi; k += kThreads) {
            const Vec<T> v[1] = {{ld16_again(z + (k * n - g.lead))}};
            add_vectors<T, kMoment>(L, v, r);
        }
    }
    if (g.edge >= 0) {
        const Vec<T> v[1] = {load_edge(z, g.edge * n - g.lead, L.vocab)};
        if (kHighest) count_from_highest<kMoment>(L, Vec<T>::max(v), r);
        add_vectors<T, kMoment>(L, v, r);
    }
    r = join_parts<kMoment>(L, parts, r);
    c = finish_row<kKind>(L, P, out, row, y, zy, r, c, threadIdx.x == 0 && cluster_rank() == 0);
    if constexpr (kGrad) {
        const RowGrad q{origin(r.m), c, 1.0f / r.s, y < L.vocab ? (int)y : -16};
        if (c == 0.0f) zero_row<T, kThreads>(g, L.vocab, dz, same);
        else grad_row<T, kThreads>(L, z, g, q, dz, same);
    }
    leave_cluster();
}

// ----------------------------------------------------------------------------------------------------------------------
// many long rows: a ring of shared memory
// ----------------------------------------------------------------------------------------------------------------------
//
// Where there are more rows than CTAs, what a CTA per row loses is its start and its joins: the loads stop there. Here a
// CTA takes row after row. One producer thread keeps a ring of stages filled with bulk copies, the row's vectors
// once for the statistics and, for a gradient, once more for it (from L2), and goes on to the next row while the consumers
// join this one's parts: the loads depend on nothing that they compute. The consumer warps take each stage together.
// Rows are handed out by the hardware: the grid has a CTA for each row, and a CTA that is at work cancels one that has not
// begun and takes its row, so that rows that do not count leave no CTA idle. Every wait is bounded.
// A CTA's consumer threads, its ring, and the CTAs of an SM.
template <int kThreads, int kVectors, int kCount, int kCtas>
struct RingShape {
    static constexpr int consumers = kThreads, warps = kThreads / 32, vectors = kVectors, stages = kCount, ctas = kCtas;
    static constexpr int threads = kThreads + 32, stage_bytes = kVectors * 16, bytes = kCount * stage_bytes;
    static constexpr int per_thread = kVectors / kThreads;
};
// Each the best of a dozen shapes. Reading only: many CTAs, so that others compute while one joins a row, and smaller ones the
// shorter the rows. Log-probabilities without and with entropies in us, four CTAs of 192 threads and then six of 128, bfloat16:
// 8,192 rows of 8,192 logits 39 and 43, 31 and 37; of 16,384 52 and 58, 46 and 54; of 32,768 80 and 91, 85 and 89; 6,144 of
// 50,257 92 and 100, 99 and 105. Three CTAs of 256 threads take 95 and 107 for the last, two of 384 112 and 126.
using ShortReadRing = RingShape<128, 1024, 2, 6>;
using ReadRing = RingShape<192, 1536, 2, 4>;
// A gradient reads its row again, which has to be in L2 still: of long rows one at a time on an SM (6,144 rows of 131,072:
// 486 us, 6.2 TB/s, against 535 us with two CTAs and 625 us with three), of others two (6,144 rows of 50,257: 196 us,
// with 256 threads 214 us; 260 us with one CTA).
using GradRing = RingShape<384, 2304, 3, 2>;
using LongGradRing = RingShape<512, 2048, 6, 1>;
// One pass that reads and writes.
using StreamRing = RingShape<512, 2048, 3, 2>;
constexpr int64_t kLongReadBytes = 48 << 10, kLongRowBytes = 160 << 10;
constexpr int kEntries = 2;
constexpr int64_t kRingRows = 300, kShortRingRows = 4096;

// Set (OR-ed) by a kernel whose bounded wait gave up; read and cleared by the host (read_logits_status).
__device__ unsigned int g_logits_status;
std::atomic<bool> g_ring_launched{false};  // in this process; until then nothing can have set it
enum : unsigned int { kStatusRowProducer = 0x20u, kStatusRowConsumer = 0x40u };

// A row handed to the consumers; row < 0: no more.
struct RowEntry {
    int64_t row, y;
    float c;   // the coefficient where it was given
    float zy;  // the target's logit; -inf for a target past the vocabulary
};

template <typename S>
struct Ring {
    alignas(16) uint4 answer;  // of the hardware, about the next row
    uint64_t asked;
    uint64_t full[S::stages], empty[S::stages];
    uint64_t entry_full[kEntries], entry_empty[kEntries];
    uint64_t joined;
    RowEntry entry[kEntries];
    Running part[2][S::warps];  // by the row's parity: a warp is at most one row ahead
};

template <typename S>
__device__ __forceinline__ void ask_next_row(Ring<S>& ring) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last answer has been read
    mbar_arrive_expect_tx(&ring.asked, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(&ring.answer)),
                 "r"(smem_u32(&ring.asked))
                 : "memory");
}

// The row of the CTA that was cancelled, or -1 when every CTA has begun.
template <typename S>
__device__ __forceinline__ int64_t next_row(const Ring<S>& ring) {
    uint32_t got, row;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t"
        "ld.shared.v2.b64 {lo, hi}, [%2];\n\t"
        "mov.b128 r, {lo, hi};\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(row)
        : "r"(smem_u32(&ring.answer))
        : "memory");
    return got ? (int64_t)row : -1;
}

template <typename T>
__device__ __forceinline__ Vec<T> stage_vector(const unsigned char* stage, int i) {
    return Vec<T>{*reinterpret_cast<const uint4*>(stage + i * 16)};
}

// kStream: the gradient with the statistics given (`stat`, out.coef the whole coefficient): no first pass.
template <typename T, RowKind kKind, bool kStream, typename S>
__global__ void __launch_bounds__(S::threads, S::ctas) ring_kernel(LogitRows L, PolicyTerms P, RowOut out) {
    constexpr int n = Vec<T>::n;
    constexpr bool kGrad = kKind == kGiven || kKind == kPolicy, kMoment = kKind == kEntropy, kHighest = !kGrad;
    constexpr int kPasses = kGrad && !kStream ? 2 : 1;
    extern __shared__ __align__(128) unsigned char stages[];
    constexpr int kStages = S::stages, kStageVectors = S::vectors, kStageBytes = S::stage_bytes;
    constexpr int kConsumers = S::consumers, kPerThread = S::per_thread;
    __shared__ Ring<S> ring;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        mbar_init(&ring.asked, 1);
        mbar_init(&ring.joined, kConsumers / 32);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ring.full[i], 1);
            mbar_init(&ring.empty[i], kConsumers / 32);
        }
        for (int i = 0; i < kEntries; ++i) {
            mbar_init(&ring.entry_full[i], 1);
            mbar_init(&ring.entry_empty[i], kConsumers / 32);
        }
        mbar_fence_init();
    }
    __syncthreads();
    wait_prerequisite();
    const T* logits = reinterpret_cast<const T*>(L.z);

    if (warp == kConsumers / 32) {  // the producer
        if (lane != 0) return;
        auto head = [&](int64_t row, int64_t* y, float* c) {
            *y = target_of(L, row);
            *c = kKind == kGiven ? out.coef[row] * out.factor : 1.0f;
        };
        uint64_t keep, drop;
        asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
        // given statistics were taken from the first row on: the rows read last are still in L2
        auto row_of = [&](int64_t cta) { return kStream && cta >= 0 ? L.rows - 1 - cta : cta; };
        int64_t row = row_of(blockIdx.x), y;
        Turn<kStages> turn;
        Turn<kEntries> entries;
        int queued = 0;
        float c;
        head(row, &y, &c);
        ask_next_row(ring);
        bool ok = true, asking = true;  // asking: an answer is on its way
        uint32_t asked = 0;             // its phase
        while (ok) {
            if (!(ok = mbar_wait(&ring.asked, asked))) break;
            asked ^= 1;
            const int64_t next = row_of(next_row(ring));
            int64_t next_y = -1;
            float next_c = 0.0f;
            asking = next >= 0;
            if (asking) {
                ask_next_row(ring);
                head(next, &next_y, &next_c);  // (arrives while this row's copies are queued)
            }
            if (!(ok = mbar_wait(&ring.entry_empty[entries.at], entries.round ^ 1))) break;
            const float zy = !kStream && y >= 0 && y < L.vocab ? widen(logits[row * L.ld + y]) : -INFINITY;
            ring.entry[entries.at] = RowEntry{row, y, c, zy};
            mbar_arrive(&ring.entry_full[entries.at]);
            entries.next();
            if (y >= 0 && c != 0.0f) {
                const T* z = logits + row * L.ld;
                const int lead = (int)(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
                const int lo = lead > 0, hi = (lead + L.vocab) / n;
                for (int pass = 0; pass < kPasses && ok; ++pass)
                    for (int k = lo; k < hi; k += kStageVectors, turn.next()) {
                        const int s = turn.at;
                        if (!(ok = mbar_wait(&ring.empty[s], turn.round ^ 1))) break;
                        if (queued < kStages) ++queued;
                        const uint32_t bytes = (uint32_t)min(kStageVectors, hi - k) * 16;
                        mbar_arrive_expect_tx(&ring.full[s], bytes);
                        unsigned char* to = stages + s * kStageBytes;
                        const T* at = z + (k * n - lead);
                        if (kPasses == 1) bulk_copy_g2s(to, at, bytes, &ring.full[s]);
                        else bulk_copy_g2s_hint(to, at, bytes, &ring.full[s], pass == 0 ? keep : drop);
                    }
            }
            row = next, y = next_y, c = next_c;
            if (row < 0 && ok) {  // the end: an entry of its own
                if (!(ok = mbar_wait(&ring.entry_empty[entries.at], entries.round ^ 1))) break;
                ring.entry[entries.at] = RowEntry{-1, -1, 0.0f, 0.0f};
                mbar_arrive(&ring.entry_full[entries.at]);
                break;
            }
        }
        if (!ok) atomicOr(&g_logits_status, kStatusRowProducer);
        // no copy is left in flight when the CTA ends, and no answer (after a wait that gave up)
        drain(ring.full, turn, queued);
        if (asking) mbar_wait(&ring.asked, asked);
        return;
    }

    Turn<kStages> turn;
    Turn<kEntries> entries;
    uint32_t joins = 0;  // mod 2
    auto give_up = [&] { atomicOr(&g_logits_status, kStatusRowConsumer); };
    for (;; entries.next()) {
        if (!mbar_wait(&ring.entry_full[entries.at], entries.round)) return give_up();
        const RowEntry at = ring.entry[entries.at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.entry_empty[entries.at]);
        const int64_t row = at.row, y = at.y;
        if (row < 0) return;
        const T* z = logits + row * L.ld;
        T* dz = kGrad ? reinterpret_cast<T*>(out.dz) + row * out.ld_d : nullptr;
        const bool same = kGrad && (reinterpret_cast<uintptr_t>(dz) - reinterpret_cast<uintptr_t>(z)) % 16 == 0;
        const RowVectors g = row_vectors(z, L.vocab);
        float c = kKind == kGiven ? at.c : 0.0f;
        if (y < 0 || (kKind == kGiven && c == 0.0f)) {
            if (kGrad) zero_row<T, kConsumers>(g, L.vocab, dz, same);
            skip_outputs<kKind>(out, row);
            continue;
        }
        const float zy = at.zy;
        Running q{zy, 0.0f, 0.0f};
        if constexpr (!kStream) {
            for (int k = g.lo; k < g.hi; k += kStageVectors, turn.next()) {
                const int s = turn.at, left = g.hi - k;
                if (!mbar_wait(&ring.full[s], turn.round)) return give_up();
                const unsigned char* stage = stages + s * kStageBytes;
                if (left >= kStageVectors) {
                    Vec<T> v[kPerThread];
#pragma unroll
                    for (int u = 0; u < kPerThread; ++u) v[u] = stage_vector<T>(stage, (int)threadIdx.x + u * kConsumers);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring.empty[s]);
                    if (kHighest) count_from_highest<kMoment>(L, Vec<T>::max(v), q);
#pragma unroll
                    for (int u = 0; u < kPerThread; u += 2) {
                        const Vec<T> two_of[2] = {v[u], v[u + 1]};
                        add_vectors<T, kMoment>(L, two_of, q);
                    }
                } else {
                    if (kHighest) {
                        float m = q.m;
                        for (int i = (int)threadIdx.x; i < left; i += kConsumers)
                            m = fmaxf(m, Vec<T>::max({stage_vector<T>(stage, i)}));
                        count_from_highest<kMoment>(L, m, q);
                    }
                    for (int i = (int)threadIdx.x; i < left; i += kConsumers) {
                        const Vec<T> v[1] = {stage_vector<T>(stage, i)};
                        add_vectors<T, kMoment>(L, v, q);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring.empty[s]);
                }
            }
            if (g.edge >= 0) {
                const Vec<T> v[1] = {load_edge(z, g.edge * n - g.lead, L.vocab)};
                if (kHighest) count_from_highest<kMoment>(L, Vec<T>::max(v), q);
                add_vectors<T, kMoment>(L, v, q);
            }
            q = join_warp<kMoment>(L, q);
            Running* part = ring.part[joins];
            if (lane == 0) {
                part[warp] = q;
                mbar_arrive(&ring.joined);
            }
            if (!mbar_wait(&ring.joined, joins)) return give_up();
            joins ^= 1;
            if (kGrad || warp == 0) {
                q = join_warp<kMoment>(L, lane < kConsumers / 32 ? part[lane] : Running{-INFINITY, 0.0f, 0.0f});
                c = finish_row<kKind>(L, P, out, row, y, zy, q, c, threadIdx.x == 0);
            }
        } else {
            const RowStat st = out.stat[row];
            q = Running{st.origin, 1.0f / st.inv_sum, 0.0f};
            if (y >= L.vocab) c = NAN;
        }
        if constexpr (kGrad) {
            const RowGrad grad{origin(q.m), c, kStream ? out.stat[row].inv_sum : 1.0f / q.s, y < L.vocab ? (int)y : -16};
            if (g.edge >= 0) {
                const int j0 = g.edge * n - g.lead;
                float d[n];
                grad_values(L, load_edge(z, j0, L.vocab), grad, j0, d);
                store_some(dz, j0, L.vocab, d);
            }
            for (int k = g.lo; k < g.hi; k += kStageVectors, turn.next()) {
                const int s = turn.at, left = g.hi - k, j0 = (k + (int)threadIdx.x) * n - g.lead;
                if (!mbar_wait(&ring.full[s], turn.round)) return give_up();
                const unsigned char* stage = stages + s * kStageBytes;
                if (left >= kStageVectors) {
                    Vec<T> v[kPerThread];
#pragma unroll
                    for (int u = 0; u < kPerThread; ++u) v[u] = stage_vector<T>(stage, (int)threadIdx.x + u * kConsumers);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring.empty[s]);
#pragma unroll
                    for (int u = 0; u < kPerThread; ++u) grad_vector(L, v[u], grad, j0 + u * kConsumers * n, dz, same);
                } else {
                    for (int i = (int)threadIdx.x; i < left; i += kConsumers)
                        grad_vector(L, stage_vector<T>(stage, i), grad, (k + i) * n - g.lead, dz, same);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring.empty[s]);
                }
            }
        }
    }
}

// The gradient with the rows' statistics and coefficients given: a stream, a cluster of CTAs per row for few rows.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kRowResident / kThreads) row_grad_kernel(LogitRows L, const RowStat* stat,
                                                                             const float* coef, T* out, int64_t ld_d) {
    wait_prerequisite();
    allow_dependents();
    const int64_t row = L.rows - 1 - blockIdx.x / cluster_size();  // the rows that were read last are still in L2
    const T* z = reinterpret_cast<const T*>(L.z) + row * L.ld;
    T* dz = out + row * ld_d;
    const bool same = (reinterpret_cast<uintptr_t>(dz) - reinterpret_cast<uintptr_t>(z)) % 16 == 0;
    const int64_t y = target_of(L, row);
    const RowVectors g = row_vectors(z, L.vocab);
    const float given = y < 0 ? 0.0f : coef[row], c = y < L.vocab ? given : NAN;
    if (given == 0.0f) {  // (a row in no sequence, whatever its target)
        zero_row<T, kThreads>(g, L.vocab, dz, same);
        return;
    }
    const RowStat st = stat[row];
    grad_row<T, kThreads>(L, z, g, RowGrad{origin(st.origin), c, st.inv_sum, y < L.vocab ? (int)y : -16}, dz, same);
}

// ----------------------------------------------------------------------------------------------------------------------
// per-token and per-pair terms
// ----------------------------------------------------------------------------------------------------------------------

constexpr int kSumThreads = 1024, kSumWarps = kSumThreads / 32;

// A sum in two float32, hi + lo, to some 2^-45 of its terms: what each addition rounds away is added up too. (This chip has
// next to no float64: 96 tokens' sums in it took 37 us.) hi alone once it is infinite or a NaN.
struct Sum {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float t = hi + x, z = t - hi;
        lo += (hi - (t - z)) + (x - z);
        hi = t;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.hi);
        lo += o.lo;
    }
    // the sum over n, to as many bits: what hi / n rounds away is exactly a float32 times 1 / n
    __device__ __forceinline__ Sum over(float n) const {
        const float q = hi / n;
        return Sum{q, (fmaf(-q, n, hi) + lo) / n};
    }
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// The lanes' sums in order, in lane 0.
__device__ __forceinline__ Sum warp_total(Sum s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const Sum o{__shfl_down_sync(~0u, s.hi, d), __shfl_down_sync(~0u, s.lo, d)};
        s.add(o);
    }
    return s;
}

__global__ void __launch_bounds__(kSumThreads) policy_sums_kernel(LogitRows L, PolicyTerms P, const float* logps,
                                                                  float* stats) {
    __shared__ Sum part[3][kSumWarps];
    wait_prerequisite();
    allow_dependents();
    Sum sum[3] = {};  // surrogate, KL, clipped
    for (int64_t row = threadIdx.x; row < L.rows; row += kSumThreads) {
        const int64_t y = target_of(L, row);
        const float lp = logps[row], A = P.advantages[row], old = P.old_logps[row];
        const float w = P.weights ? P.weights[row] : 1.0f, ref = P.ref_logps ? P.ref_logps[row] : 0.0f;
        if (y < 0) continue;
        const float r = expf(lp - old), plain = r * A, held = fminf(fmaxf(r, P.lo), P.hi) * A;
        sum[0].add(-w * (held < plain ? held : plain));
        if (P.ref_logps) sum[1].add(w * (expm1f(ref - lp) - (ref - lp)));
        sum[2].add(held < plain ? w : 0.0f);
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const Sum s = warp_total(sum[i]);
        if (lane == 0) part[i][warp] = s;
    }
    __syncthreads();
    if (warp == 0) {
        float v[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i] = warp_total(part[i][lane]).value() * P.inv_denom;
        if (lane == 0) {
            stats[0] = P.ref_logps ? fmaf(P.kl_coef, v[1], v[0]) : v[0];
            stats[1] = v[0];
            stats[2] = v[1];
            stats[3] = v[2];
        }
    }
}

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

__device__ __forceinline__ int64_t clamp_row(int64_t x, int64_t rows) { return x < 0 ? 0 : x > rows ? rows : x; }

// One CTA. Teams of warps sum the sequences (as many teams as sequences, at most one a warp); then the threads take the
// pairs' losses and slopes; then the teams write their sequences' coefficients. sums[s] and sums[2 n + s], n sequences: a
// sequence's sum (a pair's difference may be far smaller than its sums, and is rounded once), and sums[n + s], 1 over what
// that was divided by; then sums[s]: its rows' coefficient.
__global__ void __launch_bounds__(kSumThreads) pairs_kernel(LogitRows L, PairTerms P, const float* logps,
                                                            const float* rest, float* sums, float* loss, float* rewards,
                                                            float* coef) {
    __shared__ Sum part[kSumWarps];
    __shared__ int count[kSumWarps];
    wait_prerequisite();
    allow_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = 2 * P.pairs;
    int team = kSumWarps;  // warps of a team
    while (team > 1 && kSumWarps / team < n) team /= 2;
    const int first = warp / team, step = kSumWarps / team, rank = (warp % team) * 32 + lane, stride = team * 32;
    if (coef)
        for (int64_t row = threadIdx.x; row < L.rows; row += kSumThreads) coef[row] = 0.0f;
    const int rounds = (n + step - 1) / step;
    for (int i = 0; i < rounds; ++i) {
        const int s = first + i * step;
        Sum d{};
        int scored = 0;
        if (s < n) {
            const int64_t a = clamp_row(P.cu_seqlens[s], L.rows), b = clamp_row(P.cu_seqlens[s + 1], L.rows);
#pragma unroll 4
            for (int64_t row = a + rank; row < b; row += stride) {
                const bool on = target_of(L, row) >= 0;
                const float hi = logps[row], lo = rest[row], ref = P.ref_logps ? P.ref_logps[row] : 0.0f;
                d.add(on ? hi : 0.0f);
                d.add(on ? -ref : 0.0f);
                d.lo += lo;
                scored += on;
            }
        }
        d = warp_total(d);
        scored = __reduce_add_sync(~0u, scored);
        __syncthreads();  // the last round's parts have been read
        if (lane == 0) {
            part[warp] = d;
            count[warp] = scored;
        }
        __syncthreads();
        if (rank == 0 && s < n) {
            for (int w = 1; w < team; ++w) {
                d.add(part[warp + w]);
                scored += count[warp + w];
            }
            const float by = P.length_norm && scored > 0 ? (float)scored : 1.0f;
            if (P.length_norm) d = d.over(by);
            sums[s] = d.hi;
            sums[n + s] = 1.0f / by;
            sums[2 * n + s] = d.lo;
            if (rewards) rewards[s] = P.beta * d.value();
        }
    }
    __syncthreads();
    Sum mine{};
    for (int p = threadIdx.x; p < P.pairs; p += kSumThreads) {
        Sum apart{sums[2 * p], sums[2 * n + 2 * p]};
        apart.add(Sum{-sums[2 * p + 1], -sums[2 * n + 2 * p + 1]});
        const float d = apart.value(), h = P.beta * d;
        float l, slope;  // the pair's loss and its derivative by d
        if (P.kind == MICA_PREF_SIGMOID) {
            l = (1.0f - P.smoothing) * softplus(-h) + (P.smoothing > 0.0f ? P.smoothing * softplus(h) : 0.0f);
            slope = P.beta * (P.smoothing / (1.0f + expf(-h)) - (1.0f - P.smoothing) / (1.0f + expf(h)));
        } else if (P.kind == MICA_PREF_HINGE) {
            l = h < 1.0f ? 1.0f - h : (h >= 1.0f ? 0.0f : h);  // (a NaN stays one)
            slope = h < 1.0f ? -P.beta : (h >= 1.0f ? 0.0f : h);
        } else {
            const float gap = d - 0.5f / P.beta;
            l = gap * gap;
            slope = 2.0f * gap;
        }
        mine.add(l);
        sums[2 * p] = slope * P.grad_factor;
        sums[2 * p + 1] = -slope * P.grad_factor;
    }
    mine = warp_total(mine);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const Sum total = warp_total(part[lane]);
        if (lane == 0) *loss = P.pairs ? total.value() / (float)P.pairs : 0.0f;
    }
    if (!coef) return;
    for (int s = first; s < n; s += step) {
        const int64_t a = clamp_row(P.cu_seqlens[s], L.rows), b = clamp_row(P.cu_seqlens[s + 1], L.rows);
        const float c = sums[s] * sums[n + s];
        for (int64_t row = a + rank; row < b; row += stride) coef[row] = c;
    }
}

// Many rows go through the ring, the shorter the more there have to be. Measured both ways, in us, the ring first, bfloat16:
// log-probabilities of 8,192 rows of 1,024 logits 21 and 19, 1,536: 23 and 27, 4,096: 27 and 40, 32,768: 80 and 90; of 1,200
// rows of 50,257 26 and 26, of 300 of 16,384 10 and 12; policy gradients of 6,144 rows of 16,384: 91 and 79, 32,768: 135 and
// 154, 50,257: 196 and 267; of 300 rows of 131,072: 33 and 43.
bool takes_ring(const LogitRows& L, bool grad) {
    const int64_t bytes = L.vocab * (L.dtype == MICA_F32 ? 4 : 2);
    if (grad) return L.rows >= kRingRows && bytes >= 64 << 10;
    return (L.rows >= kRingRows && bytes >= 16 << 10) || (L.rows >= kShortRingRows && bytes >= 3 << 10);
}

// How a row is cut otherwise: C CTAs of `threads` threads.
struct RowShape {
    int C, threads;
};

RowShape row_shape(const LogitRows& L) {
    const int64_t n = L.dtype == MICA_F32 ? 4 : 8, vectors = (L.vocab + n - 1) / n + 1;  // one more for a row's alignment
    if (vectors <= kBatch * kShortThreads) return RowShape{1, kShortThreads};
    int C = 1;
    while (C < kMostCluster && L.rows * C < kFewCtas && vectors > C * kRowThreads) C *= 2;
    return RowShape{C, kRowThreads};
}

template <typename K, typename... A>
cudaError_t launch_clusters(K kernel, int64_t ctas, int C, int threads, size_t shared, void* stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, RowKind kKind, bool kStream>
cudaError_t launch_ring(const LogitRows& L, const PolicyTerms& P, const RowOut& out, void* stream) {
    auto go = [&](auto shape) {
        using S = decltype(shape);
        const auto kernel = ring_kernel<T, kKind, kStream, S>;
        g_ring_launched = true;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
        return e != cudaSuccess ? e : launch_clusters(kernel, L.rows, 1, S::threads, S::bytes, stream, L, P, out);
    };
    if constexpr (kKind == kLogps || kKind == kEntropy)
        return L.vocab * (int64_t)sizeof(T) > kLongReadBytes ? go(ReadRing{}) : go(ShortReadRing{});
    else if constexpr (kStream) return go(StreamRing{});
    else return L.vocab * (int64_t)sizeof(T) > kLongRowBytes ? go(LongGradRing{}) : go(GradRing{});
}

template <RowKind kKind, typename T>
cudaError_t launch_rows_of(const LogitRows& L, const PolicyTerms& P, const RowOut& out, void* stream) {
    if (takes_ring(L, kKind == kGiven || kKind == kPolicy)) return launch_ring<T, kKind, false>(L, P, out, stream);
    const RowShape s = row_shape(L);
    const int64_t ctas = L.rows * s.C;
    return s.threads == kShortThreads
               ? launch_clusters(row_kernel<T, kShortThreads, kKind>, ctas, s.C, s.threads, 0, stream, L, P, out)
               : launch_clusters(row_kernel<T, kRowThreads, kKind>, ctas, s.C, s.threads, 0, stream, L, P, out);
}

template <RowKind kKind>
int launch_rows(const LogitRows& L, const PolicyTerms& P, const RowOut& out, void* stream) {
    return (int)(L.dtype == MICA_F32   ? launch_rows_of<kKind, float>(L, P, out, stream)
                 : L.dtype == MICA_F16 ? launch_rows_of<kKind, __half>(L, P, out, stream)
                                       : launch_rows_of<kKind, __nv_bfloat16>(L, P, out, stream));
}

template <typename T>
int launch_row_grad_of(const LogitRows& L, const RowStat* stat, const float* coef, void* dz, int64_t ld_d, void* stream) {
    if (takes_ring(L, true))
        return (int)launch_ring<T, kGiven, true>(
            L, PolicyTerms{}, RowOut{nullptr, nullptr, nullptr, const_cast<RowStat*>(stat), coef, 1.0f, dz, ld_d}, stream);
    const RowShape s = row_shape(L);
    T* out = static_cast<T*>(dz);
    const auto kernel = s.threads == kShortThreads ? row_grad_kernel<T, kShortThreads> : row_grad_kernel<T, kRowThreads>;
    return (int)launch_clusters(kernel, L.rows * s.C, s.C, s.threads, 0, stream, L, stat, coef, out, ld_d);
}

}  // namespace

int launch_row_logps(const LogitRows& L, float* logps, float* rest_logps, float* entropy, RowStat* stat, void* stream) {
    const RowOut out{logps, rest_logps, entropy, stat, nullptr, 0.0f, nullptr, 0};
    return entropy ? launch_rows<kEntropy>(L, PolicyTerms{}, out, stream)
                   : launch_rows<kLogps>(L, PolicyTerms{}, out, stream);
}

int launch_row_softmax_grad(const LogitRows& L, const float* coef, float factor, void* dz, int64_t ld_d, void* stream) {
    const RowOut out{nullptr, nullptr, nullptr, nullptr, coef, factor, dz, ld_d};
    return launch_rows<kGiven>(L, PolicyTerms{}, out, stream);
}

int launch_row_policy_grad(const LogitRows& L, const PolicyTerms& P, float* logps, void* dz, int64_t ld_d, void* stream) {
    return launch_rows<kPolicy>(L, P, RowOut{logps, nullptr, nullptr, nullptr, nullptr, 0.0f, dz, ld_d}, stream);
}

int launch_row_grad(const LogitRows& L, const RowStat* stat, const float* coef, void* dz, int64_t ld_d, void* stream) {
    return L.dtype == MICA_F32   ? launch_row_grad_of<float>(L, stat, coef, dz, ld_d, stream)
           : L.dtype == MICA_F16 ? launch_row_grad_of<__half>(L, stat, coef, dz, ld_d, stream)
                                 : launch_row_grad_of<__nv_bfloat16>(L, stat, coef, dz, ld_d, stream);
}

int launch_policy_sums(const LogitRows& L, const PolicyTerms& P, const float* logps, float* stats, void* stream) {
    return (int)launch_clusters(policy_sums_kernel, 1, 1, kSumThreads, 0, stream, L, P, logps, stats);
}

int launch_pairs(const LogitRows& L, const PairTerms& P, const float* logps, const float* rest, float* sums, float* loss,
                 float* rewards, float* coef, void* stream) {
    return (int)launch_clusters(pairs_kernel, 1, 1, kSumThreads, 0, stream, L, P, logps, rest, sums, loss, rewards, coef);
}

int read_logits_status(unsigned int* status) {
    *status = 0;
    if (!g_ring_launched) return (int)cudaSuccess;
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_logits_status, sizeof v);
    if (e != cudaSuccess) return (int)e;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_logits_status, &zero, sizeof zero);
    }
    *status = v;
    return (int)e;
}

}  // namespace mica
