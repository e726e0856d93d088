// The losses over logits: log-probabilities, preference and policy losses, and the gradient of the logits.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "mica_optim.h"
#include "plan.h"
#include "stream.cuh"
#include "train.h"

namespace mica {
namespace {

constexpr int kRowThreads = 256, kRowResident = 1280, kShortThreads = 64;  // threads of a CTA, and of those an SM holds; for short rows
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMostCluster = 8;  // CTAs of a portable cluster
constexpr int kBatch = 4;        // vectors of a thread in flight
constexpr int64_t kFewCtas = 304;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFarBelow = -1000.0f;  // an exponent of 2 whose power is 0, and finite (0 * it is 0)
// ex2.approx's relative error averages -4.9e-8 over every unit interval (measured on GB300; 2^0 is exact), and so does that
// of a sum of its values past the largest one's 1: a log-probability that is to be summed over a sequence takes it out.
constexpr double kExp2Bias = 4.9e-8;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

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
// Measured on GB300, 8,192 rows of 50,257 bfloat16 logits of which 6,144 count: log-probabilities and entropies 116 us
// (5.3 TB/s), 138 us with CTAs of 512 threads. Rows held in the registers of a cluster, read once from L2 too, took 295 us:
// the share of a thread was so small that the joins were most of its work.
//
// Vectors start at 16-byte addresses, whatever the row's alignment (an odd vocabulary puts each row elsewhere): the first
// and the last may reach outside the row, and are then read and written element by element, the rest as -inf.

// z[j] - max in units of log2, 2^that being the weight: a = log2(e) / temperature split in two floats, since the relative
// error of one alone (up to 2^-24) would shift every log-probability of a sequence the same way. a_lo > 0 (the host sees
// to it), so that a banned token's -inf stays -inf.
__device__ __forceinline__ float exponent(const LogitRows& L, float z, float origin) {
    const float d = z - origin;
    return fmaf(d, L.a_hi, d * L.a_lo);
}

// Two float32 in one register pair: additions and products of both in one instruction, each rounded as it would be alone.
// What bounds these kernels next to memory is the instructions that they issue.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 each(Two a) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
    return f;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// A part that has seen nothing but -inf counts from 0, so that no difference of two infinities makes its zero weight a NaN.
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

// The softmax of part of a row: the largest logit, s = sum 2^x and u = sum x 2^x, x the exponents.
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
    __device__ __forceinline__ float max() const {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
        } else {
            using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
            const T2* p = reinterpret_cast<const T2*>(&raw);
            const T2 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
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
    double* wide_logps;   // kLogps, or null: the log-probabilities before they are rounded
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

// One vector of the gradient c * ((j == y) - p), from the element j0 on.
template <typename T>
__device__ __forceinline__ void grad_values(const LogitRows& L, const Vec<T>& v, const RowGrad& q, int j0,
                                            float (&d)[Vec<T>::n]) {
    constexpr int n = Vec<T>::n;
    const float k = -q.c * q.inv;
    const Two o = two(-q.o, -q.o), a = two(L.a, L.a), kk = two(k, k);
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        const float2 x = each((v.pair(i) + o) * a);
        const float2 e = each(two(exp2_fast(x.x), exp2_fast(x.y)) * kk);
        d[2 * i] = e.x;
        d[2 * i + 1] = e.y;
    }
    if ((unsigned)(q.at - j0) < (unsigned)n) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (j0 + i == q.at) d[i] = q.c * (1.0f - q.inv * exp2_fast((v.get(i) - q.o) * L.a));
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

// Adds a vector's weights, counted from o, to s (and their moments to u).
template <typename T, bool kMoment>
__device__ __forceinline__ void add_vector(const LogitRows& L, const Vec<T>& v, float o, float& s, float& u) {
    const Two away = two(-o, -o), hi = two(L.a_hi, L.a_hi), lo = two(L.a_lo, L.a_lo);
    Two sv = two(0.0f, 0.0f), uv = two(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < Vec<T>::n / 2; ++i) {
        const Two d = v.pair(i) + away;
        const float2 x = each(fma2(d, hi, d * lo));
        const Two e = two(exp2_fast(x.x), exp2_fast(x.y));
        sv = sv + e;
        if (kMoment) uv = fma2(e, two(fmaxf(x.x, kFarBelow), fmaxf(x.y, kFarBelow)), uv);
    }
    const float2 t = each(sv);
    s += t.x + t.y;
    if (kMoment) {
        const float2 w = each(uv);
        u += w.x + w.y;
    }
}

// Counts a part from `m`, a larger maximum.
template <bool kMoment>
__device__ __forceinline__ void raise(const LogitRows& L, Running& r, float m) {
    const float x = fmaxf(exponent(L, r.m, m), kFarBelow), f = exp2_fast(x);
    if (kMoment) r.u = f * fmaf(r.s, x, r.u);
    r.s *= f;
    r.m = m;
}

struct Parts {
    Running warp[kRowWarps];
    Running cta;
    float c;
};

// The lanes' parts as one, in all lanes alike.
template <bool kMoment>
__device__ __forceinline__ Running join_warp(const LogitRows& L, const Running& p) {
    Running r;
    r.m = warp_max(p.m);
    const float x = fmaxf(exponent(L, p.m, origin(r.m)), kFarBelow), f = exp2_fast(x);
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

// Writes a row's results and returns the gradient's coefficient (c itself where it was given). zy: the target's logit, in
// thread 0.
template <RowKind kKind>
__device__ __forceinline__ float finish_row(const LogitRows& L, const PolicyTerms& P, const RowOut& out, int64_t row,
                                            int64_t y, float zy, const Running& r, float c, Parts& parts) {
    const float o = origin(r.m);
    const bool head = threadIdx.x == 0 && cluster_rank() == 0;
    if constexpr (kKind == kLogps || kKind == kEntropy) {
        if (head) {
            const double lp = y < L.vocab ? ((double)zy - o) * L.wide_inv_t - (log((double)r.s) + kExp2Bias * (1.0 - 1.0 / r.s)) : NAN;
            out.logps[row] = (float)lp;
            if (kKind == kLogps && out.wide_logps) out.wide_logps[row] = lp;
            if (kKind == kEntropy) out.entropy[row] = logf(r.s) - kLn2 * r.u / r.s;
            if (kKind == kLogps && out.stat) out.stat[row] = RowStat{r.m, 1.0f / r.s};
        }
    }
    if constexpr (kKind == kPolicy) {
        if (threadIdx.x == 0) {
            const float lp = y < L.vocab ? fmaf(zy - o, L.inv_t, -logf(r.s)) : NAN;
            parts.c = policy_coef(P, row, lp);
            if (head) out.logps[row] = lp;
        }
        __syncthreads();
        c = parts.c;
    }
    return y < L.vocab ? c : NAN;
}

template <typename T, int kThreads, RowKind kKind>
__global__ void __launch_bounds__(kThreads, kRowResident / kThreads) row_kernel(LogitRows L, PolicyTerms P, RowOut out) {
    constexpr int n = Vec<T>::n;
    constexpr bool kGrad = kKind == kGiven || kKind == kPolicy, kMoment = kKind == kEntropy;
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
        if (kKind != kGiven && threadIdx.x == 0 && cluster_rank() == 0) {
            out.logps[row] = 0.0f;
            if (kKind == kLogps && out.wide_logps) out.wide_logps[row] = 0.0;
            if (kKind == kEntropy) out.entropy[row] = 0.0f;
        }
        return;
    }
    const float zy = threadIdx.x == 0 && y < L.vocab ? widen(z[y]) : 0.0f;  // (dz may be written over z after the join)
    Running r{-INFINITY, 0.0f, 0.0f};
    int k = g.lo + (int)threadIdx.x;
    for (; k + (kBatch - 1) * kThreads < g.hi; k += kBatch * kThreads) {
        const T* at = z + (k * n - g.lead);
        Vec<T> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            v[u] = Vec<T>{kGrad ? ld16_again(at + u * kThreads * n) : ld16_stream(at + u * kThreads * n)};
        float m = v[0].max();
#pragma unroll
        for (int u = 1; u < kBatch; ++u) m = fmaxf(m, v[u].max());
        if (m > r.m) raise<kMoment>(L, r, m);
        const float o = origin(r.m);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) add_vector<T, kMoment>(L, v[u], o, r.s, r.u);
    }
    auto add_one = [&](const Vec<T>& v) {
        const float m = v.max();
        if (m > r.m) raise<kMoment>(L, r, m);
        add_vector<T, kMoment>(L, v, origin(r.m), r.s, r.u);
    };
    for (; k < g.hi; k += kThreads) add_one(Vec<T>{kGrad ? ld16_again(z + (k * n - g.lead)) : ld16_stream(z + (k * n - g.lead))});
    if (g.edge >= 0) add_one(load_edge(z, g.edge * n - g.lead, L.vocab));
    r = join_parts<kMoment>(L, parts, r);
    c = finish_row<kKind>(L, P, out, row, y, zy, r, c, parts);
    if constexpr (kGrad) {
        const RowGrad q{origin(r.m), c, 1.0f / r.s, y < L.vocab ? (int)y : -16};
        if (c == 0.0f) zero_row<T, kThreads>(g, L.vocab, dz, same);
        else grad_row<T, kThreads>(L, z, g, q, dz, same);
    }
    leave_cluster();
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
    const float c = y < 0 ? 0.0f : y < L.vocab ? coef[row] : NAN;
    if (c == 0.0f) {
        zero_row<T, kThreads>(g, L.vocab, dz, same);
        return;
    }
    const RowStat st = stat[row];
    grad_row<T, kThreads>(L, z, g, RowGrad{origin(st.zmax), c, st.inv_sum, y < L.vocab ? (int)y : -16}, dz, same);
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
    wait_prerequisite();
    allow_dependents();
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
__global__ void __launch_bounds__(kSumThreads) pairs_kernel(LogitRows L, PairTerms P, const double* logps, double* sums,
                                                            float* loss, float* rewards, float* coef) {
    __shared__ double shared[kSumThreads / 32];
    wait_prerequisite();
    allow_dependents();
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
            if (target_of(L, row) >= 0) d += logps[row] - (P.ref_logps ? (double)P.ref_logps[row] : 0.0);
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

// How a row is cut: C CTAs of `threads` threads.
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
cudaError_t launch_clusters(K kernel, int64_t ctas, int C, int threads, void* stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
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

template <RowKind kKind, typename T>
cudaError_t launch_rows_of(const LogitRows& L, const PolicyTerms& P, const RowOut& out, void* stream) {
    const RowShape s = row_shape(L);
    const int64_t ctas = L.rows * s.C;
    return s.threads == kShortThreads
               ? launch_clusters(row_kernel<T, kShortThreads, kKind>, ctas, s.C, s.threads, stream, L, P, out)
               : launch_clusters(row_kernel<T, kRowThreads, kKind>, ctas, s.C, s.threads, stream, L, P, out);
}

template <RowKind kKind>
int launch_rows(const LogitRows& L, const PolicyTerms& P, const RowOut& out, void* stream) {
    return (int)(L.dtype == MICA_F32   ? launch_rows_of<kKind, float>(L, P, out, stream)
                 : L.dtype == MICA_F16 ? launch_rows_of<kKind, __half>(L, P, out, stream)
                                       : launch_rows_of<kKind, __nv_bfloat16>(L, P, out, stream));
}

template <typename T>
int launch_row_grad_of(const LogitRows& L, const RowStat* stat, const float* coef, void* dz, int64_t ld_d, void* stream) {
    const RowShape s = row_shape(L);
    T* out = static_cast<T*>(dz);
    return (int)(s.threads == kShortThreads ? launch_clusters(row_grad_kernel<T, kShortThreads>, L.rows * s.C, s.C, s.threads,
                                                              stream, L, stat, coef, out, ld_d)
                                            : launch_clusters(row_grad_kernel<T, kRowThreads>, L.rows * s.C, s.C, s.threads,
                                                              stream, L, stat, coef, out, ld_d));
}

}  // namespace

int launch_row_logps(const LogitRows& L, float* logps, double* wide_logps, float* entropy, RowStat* stat, void* stream) {
    const RowOut out{logps, wide_logps, entropy, stat, nullptr, 0.0f, nullptr, 0};
    return entropy ? launch_rows<kEntropy>(L, PolicyTerms{}, out, stream) : launch_rows<kLogps>(L, PolicyTerms{}, out, stream);
}

int launch_row_softmax_grad(const LogitRows& L, const float* coef, float factor, void* dz, int64_t ld_d, void* stream) {
    return launch_rows<kGiven>(L, PolicyTerms{}, RowOut{nullptr, nullptr, nullptr, nullptr, coef, factor, dz, ld_d}, stream);
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
    return (int)launch_clusters(policy_sums_kernel, 1, 1, kSumThreads, stream, L, P, logps, stats);
}

int launch_pairs(const LogitRows& L, const PairTerms& P, const double* logps, double* sums, float* loss, float* rewards,
                 float* coef, void* stream) {
    return (int)launch_clusters(pairs_kernel, 1, 1, kSumThreads, stream, L, P, logps, sums, loss, rewards, coef);
}

}  // namespace mica
