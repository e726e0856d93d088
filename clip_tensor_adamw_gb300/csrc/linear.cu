// Losses from hidden states h (rows x features) and an output embedding W (vocabulary x features): log-probabilities of given
// tokens under the softmax of z = h W^T / T, and their gradients. The logits are not stored. The gradients do store a matrix of
// the logits' size: theirs, d, in 16 bits, of as many rows at a time as 1 GB holds (but no fewer than a tile's 256).
//
//   forward   lse_i = log sum_j exp z_ij, logp_i = z_i,target - lse_i
//   gradient  d_ij = c_i (1[j = target] - exp(z_ij - lse_i)), c_i = dlogps_i / T; dh = d W, dW = d^T h
//
// The rows that count are gathered first, so that unscored rows (prompts) cost nothing, and taken in pieces of at most
// kGradBytes of d. The forward pass is one product over all of the vocabulary whose epilogue keeps a running maximum and sum
// for each row. The gradient takes the product again, since float32 logits would take twice d's room.
// d is rounded to 16 bits once, in that product's epilogue, and multiplied with W and with h in one launch.
//
// Cross entropy, which has the forward pass and the gradient in one call, needs the product once in bfloat16: its epilogue
// leaves q_ij = exp(z_ij - z_i,target), which needs no maximum (the sum is at least 1) and has bfloat16's range, and sums it
// up. The rest is a factor 1 / sum_j q_ij for each row: in dh's epilogue, and on h's rows for dW. The few rows whose sum leaves
// the range, whose targets are less likely than some e^-44, are taken again, counted from lse. Against taking the product
// twice: 16 x 256 x 5,000 42 us and 44, 1,024 x 768 x 50,257 176 and 211, 8,192 x 768 x 50,257 1,254 and 1,564. The sum of a
// row may be 2^80 and its coefficient 2^-100: the coefficient is brought to 2^-1 by a power of two, which the gradients'
// epilogues take out again. Scaling h's rows rounds them once more. The target's element of q, most of a row, is rounded with the
// rest, which the factor makes up for: dh comes out with its own rounding and no more (1.7e-3 of its norm), a float32 dW off by
// 1.7e-3 (without: 2.4e-3 both; 2,048 x 768 x 20,011). The product taken twice (mica_linear_logps and its gradient) comes to
// 1.9e-3 and 0.9e-3 where the coefficients are a power of two, which leaves d's target elements exact, and to 2.4e-3 and 1.7e-3
// elsewhere.
//
// Logits, maxima, sums and gradients' sums are float32. d is rounded to the operands' type because the tensor cores multiply
// what they are given in 16 bits: relative 2^-9 (bfloat16) or 2^-12 of each of its elements on average. binary16 has not the
// range for d, so it is scaled by a power of two that brings the largest |c_i| to 2^15 (d is at most |c_i|), which the
// gradients' epilogues take out again.
#include <cuda_runtime.h>

#include <type_traits>

#include "gemm.cuh"
#include "linear.h"

namespace mica {
namespace {

constexpr int64_t kGradBytes = (int64_t)1 << 30;    // of d, that a piece of the rows takes (or 256 rows, if that is more)
constexpr int64_t kStatBytes = (int64_t)256 << 20;  // of the forward pass's maxima and sums
constexpr int kMostRows = 16384;                    // of a piece in the forward pass
// Rows up to which every CTA of the gather looks through all targets, which saves a launch: log-probabilities of 1,024 rows 22.0
// us so and 23.5 with a scan before, of 2,048 27.9 and 26.9, of 16,384 131 and 103.
constexpr int kLookRows = 1024;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMostSum = 0x1p64f;                 // of exp(z - z_target) over 32 columns
// Whether cross entropy takes the product once: binary16 has not the range.
template <typename T>
constexpr bool kTakenOnce = std::is_same<T, __nv_bfloat16>::value;

// What the scan of the targets leaves for the kernels after it.
struct Meta {
    int count;        // rows that count
    float coef;       // cross entropy: every row's coefficient, with the scale of d in it
    float scale;      // of d
    float inv_scale;
    unsigned int ticket;  // CTAs of the rows' joins that have ended
};

// Rows [from, from + rows) of those that count.
struct Span {
    int from, rows;
};

// The j-th piece: as few as hold `most` (a multiple of 256) rows each, all but the last of the same size.
__device__ __forceinline__ Span span_of(int count, int most, int j) {
    const int pieces = (count + most - 1) / most;
    if (j >= pieces) return Span{count, 0};
    const int each = ((count + pieces - 1) / pieces + 255) / 256 * 256;
    const int from = j * each;
    return from >= count ? Span{count, 0} : Span{from, count - from < each ? count - from : each};
}
// Whether the j-th piece is the last with rows in it.
__device__ __forceinline__ bool last_span(int count, int most, int j) { return span_of(count, most, j + 1).rows == 0; }

// How a piece of the rows is dealt, which the gather works out for the products: their divisions would take each of them
// some 2 us before its first load.
struct Dealt {
    Span span;
    int first, last;    // piece
    SplitDeal dh, dw;   // of pair 0
    int dh_left;        // dh's pieces in their last round
    float inv_scale;    // of d
    int no_grad;        // every row's coefficient is 0: d is zeros, whatever the logits are
};

__device__ __forceinline__ int64_t target_at(const void* targets, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
}

// ------------------------------------------------------------------------------------------------------------------------
// the rows that count, side by side
// ------------------------------------------------------------------------------------------------------------------------

struct Gather {
    const void* targets;
    const unsigned short* h;
    int64_t ld_h;
    int rows, features, vocab, wide, aligned;
    const float* dlogps;   // or null: a row whose dlogps is 0 does not count
    const float* lse;      // with dlogps
    float inv_t;
    float ce_factor;       // cross entropy: -grad_scale / T, divided by `denom` or, where that is 0, by the count
    float denom;
    int scaled;            // d is scaled (bfloat16, the logits taken once: what its rows are multiplied by)
    int scaled_to;         // and the largest |c| brought to [2^scaled_to, 2^(scaled_to + 1))
    int most, piece;
    Meta* meta;            // written by the first piece
    Dealt* dealt;          // by each
    int pairs, has_dh, has_dw;
    int* index;            // the rows that count
    unsigned short* out;   // [most][ld]
    int ld;
    int* target;           // [most] -1: past the vocabulary
    float* coef;           // [most] c * scale, or null
    float* origin;         // [most] lse * log2(e), or z_target a (below), or null
    const unsigned short* w;  // where z_target is wanted, or null
    int64_t ld_w;
    float a;               // log2(e) / T
    int* again;            // [1 + most / 256] or null: zeroed
    float* logps;          // or null; logps and lse_out of rows that do not count are 0
    float* lse_out;        // or null
    unsigned short* zero;  // rows that do not count get zeros here, or null
    int64_t ld_zero;
};

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ bool row_counts(const Gather& g, int i, float* c) {
    if (target_at(g.targets, g.wide, i) < 0) return false;
    *c = g.dlogps ? g.dlogps[i] : 1.0f;
    return *c != 0.0f;
}

// Of a row's coefficient, what the scale of d goes by: nothing where it is an infinity or a NaN, which shows in its row's d
// under any scale and must not take the other rows' bits.
__device__ __forceinline__ float size_of(const Gather& g, float c) {
    const float size = fabsf(c * g.inv_t);
    return size < INFINITY ? size : 0.0f;
}

// What the first look at the targets leaves: how many rows count, and the largest of their coefficients' sizes.
__device__ __forceinline__ Meta meta_of(const Gather& g, int count, float top) {
    Meta m{count, 0.0f, 1.0f, 1.0f, 0u};
    const float ce = g.ce_factor / (g.denom > 0.0f ? g.denom : (float)count);
    const float largest = g.dlogps ? top : fabsf(ce);
    if (g.scaled && largest > 0.0f && largest < INFINITY) {
        int e = (int)(__float_as_uint(largest) >> 23) - 127;  // largest < 2^(e + 1); a subnormal counts as 2^-127
        e = g.scaled_to - (e < -100 ? -100 : e);
        if (e < -126) e = -126;  // (bfloat16 only, whose range holds what is left)
        m.scale = power_of_two(e);
        m.inv_scale = power_of_two(-e);
    }
    m.coef = ce * m.scale;
    // Cross entropy in binary16: every row's coefficient is the same, so that what it has beside a power of two can wait for the
    // epilogues, and d's target elements, most of a row, are exact where p is small. (An infinite one stays as it is.)
    const float size = fabsf(m.coef);
    if (!g.dlogps && g.scaled && !g.w && size >= 0x1p14f && size < 0x1p15f) {
        m.inv_scale *= size * 0x1p-14f;
        m.coef = copysignf(0x1p14f, m.coef);
    }
    return m;
}

// A row that does not count, by a warp.
__device__ __forceinline__ void leave_row(const Gather& g, int64_t i, int lane) {
    if (g.zero) {
        unsigned short* z = g.zero + i * g.ld_zero;
        for (int x = lane; x < g.features; x += 32) z[x] = 0;
    }
    if (lane == 0 && g.logps) g.logps[i] = 0.0f;
    if (lane == 0 && g.lse_out) g.lse_out[i] = 0.0f;
}

// Row i to place r of the piece, by a warp.
template <typename T>
__device__ __forceinline__ void take_row(const Gather& g, const Meta& m, int64_t i, int r, int lane) {
    const unsigned short* in = g.h + i * g.ld_h;
    unsigned short* out = g.out + (int64_t)r * g.ld;
    const int64_t y = target_at(g.targets, g.wide, i);
    const unsigned short* own = kTakenOnce<T> && g.w && y < g.vocab ? g.w + y * g.ld_w : nullptr;  // (16-byte aligned)
    const int whole = g.aligned ? g.features / 8 : 0;
    float z = 0.0f;  // the target's logit
#pragma unroll 2
    for (int x = lane; x < whole; x += 32) {
        const uint4 u = reinterpret_cast<const uint4*>(in)[x];
        reinterpret_cast<uint4*>(out)[x] = u;
        if (!own) continue;
        const uint4 v = reinterpret_cast<const uint4*>(own)[x];
        const T *a = reinterpret_cast<const T*>(&u), *b = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int e = 0; e < 8; ++e) z = fmaf(widen(a[e]), widen(b[e]), z);
    }
    for (int x = whole * 8 + lane; x < g.features; x += 32) {
        const unsigned short u = in[x];
        out[x] = u;
        if (own) z = fmaf(widen(reinterpret_cast<const T&>(u)), widen(reinterpret_cast<const T*>(own)[x]), z);
    }
    if (own) {
#pragma unroll
        for (int d = 16; d; d /= 2) z += __shfl_xor_sync(~0u, z, d);
    }
    if (lane) return;
    g.target[r] = y < g.vocab ? (int)y : -1;
    if (g.coef) g.coef[r] = y >= g.vocab ? NAN : g.dlogps ? g.dlogps[i] * g.inv_t * m.scale : m.coef;
    if (g.dlogps) g.origin[r] = g.lse[i] * kLog2E;
    else if (g.w) g.origin[r] = y >= g.vocab ? NAN : z * g.a;
}

// What one CTA does for a piece beside its rows: how it is dealt, and the zeros behind its rows up to the next multiple of 64,
// which the weight gradient adds up.
__device__ __forceinline__ void begin_piece(const Gather& g, const Meta& m, const Span& span) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 32) {
        const int across = (g.features + kTile - 1) / kTile, stages = (span.rows + kDepth - 1) / kDepth;
        Dealt d;
        d.span = span;
        d.first = g.piece == 0;
        d.last = last_span(m.count, g.most, g.piece);
        d.dh = split_deal(g.has_dh ? (span.rows + kTile - 1) / kTile * across : 0, (g.vocab + kDepth - 1) / kDepth, 0, g.pairs);
        d.dw = split_deal(g.has_dw && (span.rows || d.first) ? (g.vocab + kTile - 1) / kTile * across : 0, stages ? stages : 1, 0,
                          g.pairs);
        d.dh_left = d.dh.pieces % g.pairs;
        d.inv_scale = m.inv_scale;
        d.no_grad = !g.dlogps && m.coef == 0.0f;
        *g.dealt = d;
    }
    if (g.again)
        for (int i = threadIdx.x; i < 1 + g.most / kTile; i += 256) g.again[i] = 0;
    for (int r = span.rows + warp; r < (span.rows + 63) / 64 * 64; r += 8)
        for (int c = lane; c < g.ld / 8; c += 32) reinterpret_cast<uint4*>(g.out + (int64_t)r * g.ld)[c] = uint4{};
}

// Many rows (over kLookRows): one CTA looks through the targets and writes down which count, in order, and behind them, backwards,
// the others; gather_kernel takes a piece of them. 8,192 rows: 12 us and 8; 1 M rows: 0.2 ms.
__global__ void __launch_bounds__(1024) scan_kernel(Gather g) {
    __shared__ int sums[32];
    __shared__ float tops[32];
    wait_prerequisite();
    allow_dependents();
    constexpr int kItems = 8;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int before = 0;
    float top = 0.0f;
    for (int base = 0; base < g.rows; base += 1024 * kItems) {
        const int first = base + threadIdx.x * kItems;
        uint32_t on = 0;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            float c;
            if (first + k >= g.rows || !row_counts(g, first + k, &c)) continue;
            on |= 1u << k;
            top = fmaxf(top, size_of(g, c));
        }
        const int mine = __popc(on);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int at = before + upto - mine, all = 0;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) at += sums[i];
            all += sums[i];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = first + k;
            if (i >= g.rows) break;
            if (on >> k & 1) g.index[at++] = i;
            else g.index[g.rows - 1 - (i - at)] = i;
        }
        before += all;
    }
#pragma unroll
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 0; i < 32; ++i) top = fmaxf(top, tops[i]);
    *g.meta = meta_of(g, before, top);
}

// A warp to a row, of those that scan_kernel wrote down.
template <typename T>
__global__ void __launch_bounds__(256) gather_kernel(Gather g) {
    wait_prerequisite();
    allow_dependents();
    const Meta m = *g.meta;
    const Span span = span_of(m.count, g.most, g.piece);
    const int lane = threadIdx.x % 32, others = g.piece ? 0 : g.rows - m.count;
    if (blockIdx.x == gridDim.x - 1) begin_piece(g, m, span);
    for (int64_t r = blockIdx.x * 8ll + threadIdx.x / 32; r < (int64_t)span.rows + others; r += gridDim.x * 8ll) {
        if (r < span.rows) take_row<T>(g, m, g.index[span.from + r], (int)r, lane);
        else leave_row(g, g.index[g.rows - 1 - (r - span.rows)], lane);
    }
}

// Few rows: a CTA takes neighbouring ones, and each looks through all of the targets, for the rows that count before its own and
// altogether: a launch less.
template <typename T>
__global__ void __launch_bounds__(256) look_kernel(Gather g) {
    __shared__ int sums[2][8];
    __shared__ float tops[8];
    __shared__ uint32_t flags[8];
    wait_prerequisite();
    allow_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int each = (g.rows + (int)gridDim.x - 1) / (int)gridDim.x;
    const int from = (int)blockIdx.x * each, to = from + each < g.rows ? from + each : g.rows;
    int before = 0, count = 0;
    float top = 0.0f;
    constexpr int kAtOnce = 8;  // loads of a thread in flight
    for (int i0 = threadIdx.x; i0 < g.rows; i0 += 256 * kAtOnce) {
        bool scored[kAtOnce];
        float c[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int i = i0 + 256 * k;
            scored[k] = i < g.rows && target_at(g.targets, g.wide, i) >= 0;
            c[k] = g.dlogps && i < g.rows ? g.dlogps[i] : 1.0f;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (!scored[k] || c[k] == 0.0f) continue;
            ++count;
            before += i0 + 256 * k < from;
            top = fmaxf(top, size_of(g, c[k]));
        }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        before += __shfl_xor_sync(~0u, before, d);
        count += __shfl_xor_sync(~0u, count, d);
        top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = count;
        tops[warp] = top;
    }
    __syncthreads();
    before = count = 0;
    for (int i = 0; i < 8; ++i) {
        before += sums[0][i];
        count += sums[1][i];
        top = fmaxf(top, tops[i]);
    }
    const Meta m = meta_of(g, count, top);
    const Span span = span_of(count, g.most, g.piece);
    if (blockIdx.x == 0) {
        if (g.piece == 0 && threadIdx.x == 0) *g.meta = m;
        begin_piece(g, m, span);
    }
    // 256 rows at a time: their flags, and then a warp to a row
    for (int base = from; base < to; base += 256) {
        const int own = base + threadIdx.x;
        float c;
        const uint32_t word = __ballot_sync(~0u, own < to && row_counts(g, own, &c));
        if (lane == 0) flags[warp] = word;
        __syncthreads();
        int rank = before;
        for (int k = 0; k < 8; ++k) {
            const uint32_t f = flags[k];
            for (int j = warp; j < 32 && base + 32 * k + j < to; j += 8) {  // rows 32 k + warp, + 8, ...
                const int i = base + 32 * k + j, at = rank + __popc(f & ((1u << j) - 1)), r = at - span.from;
                if (!(f >> j & 1)) {
                    if (g.piece == 0) leave_row(g, i, lane);
                } else if (r >= 0 && r < span.rows) {
                    if (lane == 0) g.index[at] = i;
                    take_row<T>(g, m, i, r, lane);
                }
            }
            rank += __popc(f);
        }
        before = rank;
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------------------------------------
// the logits' product, forward
// ------------------------------------------------------------------------------------------------------------------------

// A row's part of the vocabulary: sum 2^(z a - origin), with z a in units of log 2.
struct RowSum {
    float origin, sum;
};
// The origin of a part without a logit so far: finite, so that minus infinity counts from it as 0.
constexpr float kLeastOrigin = -1e38f;

struct Logits {
    static constexpr unsigned int kStatus = 0x100u;
    static constexpr bool kAhead = false, kJoins = false;
    CUtensorMap h, w;
    const Dealt* dealt;
    const int* target;
    int vocab, stages, across;  // across: tiles
    float a;  // log2(e) / T

    __device__ __forceinline__ void prefetch() const {
        prefetch_map(&h);
        prefetch_map(&w);
    }

    struct Deal {
        int rows, row_tiles, pieces, next, pairs;
        bool no_grad;
    };
    __device__ __forceinline__ Deal deal(int pair, int pairs) const {
        const int rows = dealt->span.rows, row_tiles = (rows + kTile - 1) / kTile;
        return Deal{rows, row_tiles, row_tiles * across, pair, pairs, dealt->no_grad != 0};
    }
    // rows first: h stays in L2 while W passes once
    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        const int i = d.next;
        if (i >= d.pieces) return false;
        d.next += d.pairs;
        *q = Piece{{&h, 0, true}, {&w, 0, true}, i % d.row_tiles * kTile, i / d.row_tiles * kTile, kTile,
                   0, stages, i, -1, 1, 0, 0, 0, 0};
        return true;
    }
};

struct LogitSums : Logits {
    RowSum* sums;  // [most][vocabulary / 128]
    int parts;
    float* at;     // [most] the targets' logits

    struct Epilogue {
        const LogitSums& p;
        int row, column, target;
        bool live;
        RowSum s;
        __device__ __forceinline__ Epilogue(const LogitSums& p, const Deal& d, const Piece& q, const Place& at)
            : p(p), row(q.m0 + at.row), column(q.n0 + at.first_column), s{kLeastOrigin, 0.0f} {
            live = row < d.rows;
            target = live ? p.target[row] : -1;
        }
        __device__ __forceinline__ void chunk(int c, float (&v)[32]) {
            const int first = column + 32 * c;
            if (first >= p.vocab) return;
            if (first + 32 > p.vocab) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (first + i >= p.vocab) v[i] = -INFINITY;
            }
            if ((unsigned)(target - first) < 32u) {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (target == first + i) z = v[i];
                p.at[row] = z;
            }
            float top = v[0];
#pragma unroll
            for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
            top *= p.a;
            if (top > s.origin) {
                s.sum *= exp2_fast(s.origin - top);
                s.origin = top;
            }
            float part[4] = {};
#pragma unroll
            for (int i = 0; i < 32; ++i) part[i % 4] += exp2_fast(fmaf(v[i], p.a, -s.origin));
            s.sum += (part[0] + part[1]) + (part[2] + part[3]);
        }
        __device__ __forceinline__ void done() {
            if (live && column < p.vocab) p.sums[(int64_t)row * p.parts + column / kHalf] = s;
        }
    };
};

// The product that cross entropy takes once (and, so that its loss is the same, without gradients too): q = 2^(z a - origin), 0
// at the target, and its sum. A sum counts from the target's logit; where 32 columns leave the range (kMostSum), from the
// largest so far, and the row is taken again.
struct LogitOnce : Logits {
    using T = __nv_bfloat16;
    RowSum* sums;         // [most][vocabulary / 128]; null the second time
    int parts;
    const float* origin;  // the target's logit times a; lse, in rows taken again
    const float* at;      // the second time: the targets' elements
    const int* again;     // the second time: whether there are any such rows, and in which tiles; or null
    T* d;                 // [most][ld], or null for the sums alone
    int ld;

    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        if (!again) return Logits::piece(d, q);
        if (!again[0]) return false;
        while (Logits::piece(d, q))
            if (again[1 + q->m0 / kTile]) return true;
        return false;
    }

    struct Epilogue {
        const LogitOnce& p;
        int row, column, target, lane, stored;
        bool live, kept;
        float c, at_target;
        RowSum s;
        unsigned char* staging;
        unsigned short* to;
        __device__ __forceinline__ Epilogue(const LogitOnce& p, const Deal& d, const Piece& q, const Place& at)
            : p(p), row(q.m0 + at.row), column(q.n0 + at.first_column), lane(at.lane), staging(at.staging) {
            live = row < d.rows;
            kept = live && !d.no_grad;
            target = live ? p.target[row] : -1;
            c = live ? p.origin[row] : INFINITY;
            if (c < kLeastOrigin) c = kLeastOrigin;  // a banned target, whose origin no banned token may be counted from
            at_target = live && p.again ? p.at[row] : 0.0f;
            s = RowSum{c, 0.0f};
            stored = (d.rows + 63) / 64 * 64 - (row - lane);  // rows of the warp's 32 that the weight gradient reads
            to = reinterpret_cast<unsigned short*>(p.d) + (int64_t)(row - lane) * p.ld;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int first = column + 32 * k;
            if (first >= p.ld || stored <= 0) return;  // (ld: the vocabulary, rounded up)
            if (first + 32 > p.vocab) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (first + i >= p.vocab) v[i] = -INFINITY;
            }
            const bool here = (unsigned)(target - first) < 32u;
            if (here) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (target == first + i) v[i] = -INFINITY;
            }
            float part[4] = {};
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float q0 = exp2_fast(fmaf(v[i], p.a, -c)), q1 = exp2_fast(fmaf(v[i + 1], p.a, -c));
                part[i % 4] += q0;
                part[i % 4 + 1] += q1;
                if (here) {
                    if (target == first + i) q0 = at_target;
                    if (target == first + i + 1) q1 = at_target;
                }
                w[i / 2] = kept ? pack2<T>(q0, q1) : 0u;  // (whatever z was)
            }
            const float sum = (part[0] + part[1]) + (part[2] + part[3]);
            if (!live) {
            } else if (s.origin == c && sum < kMostSum) {
                s.sum += sum;
            } else {
                float top = v[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) top = fmaxf(top, v[i]);
                top *= p.a;
                if (top > s.origin) {
                    s.sum *= exp2_fast(s.origin - top);
                    s.origin = top;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) s.sum += exp2_fast(fmaf(v[i], p.a, -s.origin));
            }
            if (p.d) store_block(to, p.ld, stored, p.ld, 0, first, lane, true, staging, w);
        }
        __device__ __forceinline__ void done() {
            if (p.sums && live && column < p.vocab) p.sums[(int64_t)row * p.parts + column / kHalf] = s;
        }
    };
};

// A float32 sum with what its rounding left out.
struct Exact {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ void add(Exact x) {
        add(x.hi);
        lo += x.lo;
    }
    __device__ __forceinline__ float value() const { return fabsf(hi) < INFINITY ? hi + lo : hi; }
};

struct Join {
    Meta* meta;
    const int* index;
    const int* target;
    const RowSum* sums;
    int most, piece, parts;
    float a;
    float* logps;
    float* lse;            // or null
    // the logits' sums
    const float* at;       // the targets' logits
    float* origin;         // or null: lse * log2(e)
    // the sums of the product taken once
    int once;
    float* at_target;      // what d holds at the target
    float* factor;         // of a row of d
    int* again;
    unsigned short* d;     // null: no gradients
    int ld_d;
    const unsigned short* h;
    unsigned short* scaled_h;
    int ld_h, features;
    // cross entropy's loss, or null
    float* loss;
    float denom;
    Exact* partial;        // [CTAs of all pieces]
    int all;               // of those
};

__device__ __forceinline__ RowSum operator+(RowSum x, RowSum y) {
    const float o = fmaxf(x.origin, y.origin);
    return RowSum{o, x.sum * exp2_fast(x.origin - o) + y.sum * exp2_fast(y.origin - o)};
}

// A row's sum, by a warp, in a fixed order.
__device__ __forceinline__ RowSum row_sum(const Join& j, int row, int lane) {
    RowSum s{kLeastOrigin, 0.0f};
    const RowSum* own = j.sums + (int64_t)row * j.parts;
#pragma unroll 4
    for (int k = lane; k < j.parts; k += 32) s = s + own[k];
#pragma unroll
    for (int d = 16; d; d /= 2) s = s + RowSum{__shfl_xor_sync(~0u, s.origin, d), __shfl_xor_sync(~0u, s.sum, d)};
    return s;
}

// A row of the product taken once: the target's logit is the origin c that its sum (over the others) counts from, unless
// it left the range. d's element at the target is that of p - 1: minus the others' sum. Returns the log-probability.
__device__ __forceinline__ float join_once(const Join& j, const Meta& m, RowSum s, int row, int lane) {
    using T = __nv_bfloat16;
    const float c = j.origin[row], k = -m.coef;
    __syncwarp();
    float logp, factor, at;
    if (!(c < INFINITY)) {  // inf - inf, or no target
        logp = factor = at = NAN;
    } else if (!(s.origin > c)) {
        logp = -log1pf(s.sum);
        factor = k / (1.0f + s.sum);
        at = -s.sum;
        // The target's element, most of the row, is rounded to T: the factor makes up for that, and shifts the others, whose own
        // roundings are as large, by as much. (Below 2^-100 it counts for nothing, and near 2^-126 T has fewer bits.)
        if (s.sum > 0x1p-100f) factor *= s.sum / widen(narrow<T>(s.sum));
    } else {  // counted from lse the second time
        const float lse = s.origin + log2f(s.sum + exp2_fast(c - s.origin));
        logp = (c - lse) * kLn2;
        factor = k;
        at = expm1f(logp);
        if (lane == 0 && j.d) {
            j.origin[row] = lse;
            j.again[0] = 1;
            j.again[1 + row / kTile] = 1;
        }
    }
    if (!j.d) return logp;
    if (k == 0.0f) factor = at = 0.0f;
    const int y = j.target[row];
    if (lane == 0) {
        j.factor[row] = factor;
        j.at_target[row] = at;
        if (y >= 0) reinterpret_cast<T*>(j.d)[(int64_t)row * j.ld_d + y] = narrow<T>(at);
    }
    const T* in = reinterpret_cast<const T*>(j.h) + (int64_t)row * j.ld_h;
    T* out = reinterpret_cast<T*>(j.scaled_h) + (int64_t)row * j.ld_h;
    for (int x = lane * 4; x < j.features; x += 128) {  // (ld_h is a multiple of 8)
        const float4 v = load4(in + x, 4, true);
        store4(out + x, make_float4(v.x * factor, v.y * factor, v.z * factor, v.w * factor), 4, true);
    }
    return logp;
}

// A warp to a row; and cross entropy's loss, whose parts the CTA that ends last adds up in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) join_rows_kernel(Join j) {
    __shared__ Exact part[256];
    __shared__ bool last;
    wait_prerequisite();
    allow_dependents();
    const Meta m = *j.meta;
    const Span span = span_of(m.count, j.most, j.piece);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row = blockIdx.x * 8 + warp;
    float logp = 0.0f;
    if (row < span.rows) {
        const RowSum s = row_sum(j, row, lane);
        const int64_t i = j.index[span.from + row];
        if constexpr (kTakenOnce<T>) {
            if (j.once) logp = join_once(j, m, s, row, lane);
        }
        if (!kTakenOnce<T> || !j.once) {
            const float l = log2f(s.sum);
            logp = j.target[row] < 0 ? NAN : (fmaf(j.at[row], j.a, -s.origin) - l) * kLn2;
            if (lane == 0 && j.lse) j.lse[i] = (s.origin + l) * kLn2;
            if (lane == 0 && j.origin) j.origin[row] = s.origin + l;
        }
        if (lane == 0) j.logps[i] = logp;
    } else if (j.scaled_h && row < (span.rows + 63) / 64 * 64) {
        unsigned short* out = j.scaled_h + (int64_t)row * j.ld_h;
        for (int x = lane; x < j.ld_h / 8; x += 32) reinterpret_cast<uint4*>(out)[x] = uint4{};
    }
    if (!j.loss) return;
    if (lane == 0) part[warp] = Exact{logp, 0.0f};
    __syncthreads();
    if (threadIdx.x == 0) {
        Exact e;
        for (int i = 0; i < 8; ++i) e.add(part[i]);
        j.partial[j.piece * (int)gridDim.x + blockIdx.x] = e;
        __threadfence();
        last = atomicAdd(&j.meta->ticket, 1u) == (unsigned)j.all - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    Exact e;
    for (int i = threadIdx.x; i < j.all; i += 256) {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(j.partial + i));
        e.add(Exact{f.x, f.y});
    }
    part[threadIdx.x] = e;
    for (int n = 128; n; n /= 2) {
        __syncthreads();
        if (threadIdx.x < n) {
            Exact x = part[threadIdx.x];
            x.add(part[threadIdx.x + n]);
            part[threadIdx.x] = x;
        }
    }
    if (threadIdx.x == 0) *j.loss = m.count ? -part[0].value() / (j.denom > 0.0f ? j.denom : (float)m.count) : 0.0f;
}

// ------------------------------------------------------------------------------------------------------------------------
// the gradient of the logits
// ------------------------------------------------------------------------------------------------------------------------

template <typename T>
struct LogitGrad : Logits {
    const float* coef;
    const float* origin;
    T* d;  // [most][ld]
    int ld;

    struct Epilogue {
        const LogitGrad& p;
        int row, column, target, lane, stored;
        bool live;
        float c, origin;
        unsigned char* staging;
        unsigned short* to;
        __device__ __forceinline__ Epilogue(const LogitGrad& p, const Deal& d, const Piece& q, const Place& at)
            : p(p), row(q.m0 + at.row), column(q.n0 + at.first_column), lane(at.lane), staging(at.staging) {
            live = row < d.rows && !d.no_grad;
            target = live ? p.target[row] : -1;
            c = live ? p.coef[row] : 0.0f;
            origin = live ? p.origin[row] : 0.0f;
            stored = (d.rows + 63) / 64 * 64 - (row - lane);  // rows of the warp's 32 that the weight gradient reads
            to = reinterpret_cast<unsigned short*>(p.d) + (int64_t)(row - lane) * p.ld;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int first = column + 32 * k;
            if (first >= p.ld || stored <= 0) return;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = -c * exp2_fast(fmaf(v[i], p.a, -origin));
            if ((unsigned)(target - first) < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (target == first + i) v[i] += c;
            }
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = live ? pack2<T>(v[2 * i], v[2 * i + 1]) : 0u;  // (whatever z was)
            store_block(to, p.ld, stored, p.ld, 0, first, lane, true, staging, w);
        }
        __device__ __forceinline__ void done() {}
    };
};

// ------------------------------------------------------------------------------------------------------------------------
// the gradients of the hidden states and of the embedding
// ------------------------------------------------------------------------------------------------------------------------

// dh = scale * factor * d W, to the rows' places
template <typename T>
struct HiddenGrad {
    CUtensorMap d, w;
    const Dealt* dealt;
    const int* index;
    int features;
    const float* factor;  // of a row, or null
    T* dh;                // or null
    int64_t ld;
    int wide, wide16;  // rows aligned for stores of four elements, of eight
    float* parts;

    struct Deal : SplitDeal {
        Span span;
        int column_tiles;
        float scale;
    };
    __device__ __forceinline__ Deal deal(const Dealt& t, int pair) const {
        Deal r;
        static_cast<SplitDeal&>(r) = t.dh;
        r.next = pair;
        r.span = t.span;
        r.column_tiles = (features + kTile - 1) / kTile;
        r.scale = t.inv_scale;
        return r;
    }
    __device__ __forceinline__ bool piece(Deal& r, Piece* q) const {
        if (!split_piece(r, q)) return false;
        q->m0 = q->tile / r.column_tiles * kTile;
        q->n0 = q->tile % r.column_tiles * kTile;
        q->columns = columns_of(features - q->n0, kTile);
        q->a = Operand{&d, 0, true};
        q->b = Operand{&w, 0, false};
        return true;
    }
    __device__ __forceinline__ int rows_of(const Deal& r) const { return r.span.rows; }
    __device__ __forceinline__ float factor_of(int row) const { return factor ? factor[row] : 1.0f; }
    // four sums of a row
    __device__ __forceinline__ void put(const Deal& r, int row, int col, float4 v) const {
        if (row >= r.span.rows || col >= features) return;
        const float f = factor_of(row), s = r.scale;  // (one after the other: their product may leave float32's range)
        store4<T>(dh + index[r.span.from + row] * ld + col,
                  make_float4(v.x * f * s, v.y * f * s, v.z * f * s, v.w * f * s), features - col, wide);
    }
    // a warp's 32 x 32 of them
    __device__ __forceinline__ void block(const Deal& r, int row0, int col0, const Place& at, float (&v)[32]) const {
        if (row0 >= r.span.rows || col0 >= features) return;
        const float f = row0 + at.lane < r.span.rows ? factor_of(row0 + at.lane) : 0.0f, s = r.scale;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<T>(v[2 * i] * f * s, v[2 * i + 1] * f * s);
        uint4 x[4];
        by_columns16(at.staging, at.lane, w, x);
        const int row = row0 + at.lane / 4, col = col0 + at.lane % 4 * 8;
        if (col >= features) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + 8 * i < r.span.rows)
                store8(reinterpret_cast<unsigned short*>(dh + index[r.span.from + row + 8 * i] * ld + col), x[i], features - col,
                       wide16);
    }
    __device__ __forceinline__ void tile_at(const Deal& r, int tile, int* m0, int* n0) const {
        *m0 = tile / r.column_tiles * kTile;
        *n0 = tile % r.column_tiles * kTile;
    }
};

// dW = add + scale * d^T h, piece after piece of the rows: sums of earlier ones wait in `sums` (dW itself where that is
// float32).
template <typename O>
struct WeightGrad {
    CUtensorMap d, h;
    int most, vocab, features;
    O* dw;         // or null
    int64_t ld;
    const O* add;  // or null
    int64_t ld_add;
    float* sums;   // null where there is one piece only
    int64_t ld_sums;
    int wide, wide16, wide_add, wide_sums;
    float* parts;

    struct Deal : SplitDeal {
        int column_tiles, first_stage;
        bool first, last;
        float scale;
    };
    __device__ __forceinline__ Deal deal(const Dealt& t, int pair) const {
        Deal r;
        static_cast<SplitDeal&>(r) = t.dw;
        // dh's last round goes on with dw's first pieces
        r.next = pair >= t.dh_left ? pair - t.dh_left : pair - t.dh_left + r.pairs;
        r.column_tiles = (features + kTile - 1) / kTile;
        r.first_stage = t.span.rows ? 0 : most / kDepth;  // without rows: past the matrices, where zeros are read
        r.first = t.first;
        r.last = t.last;
        r.scale = t.inv_scale;
        return r;
    }
    __device__ __forceinline__ bool piece(Deal& r, Piece* q) const {
        if (!split_piece(r, q)) return false;
        tile_at(r, q->tile, &q->m0, &q->n0);
        q->columns = columns_of(features - q->n0, kTile);
        q->from += r.first_stage;
        q->to += r.first_stage;
        q->a = Operand{&d, 0, false};
        q->b = Operand{&h, 0, false};
        return true;
    }
    __device__ __forceinline__ void put(const Deal& r, int row, int col, float4 v) const {
        if (row >= vocab || col >= features) return;
        const int there = features - col;
        const float s = r.scale;
        float4 a{};
        if (!r.first) a = load4(sums + row * ld_sums + col, there, wide_sums);
        else if (add) a = load4(add + row * ld_add + col, there, wide_add);
        v = make_float4(fmaf(v.x, s, a.x), fmaf(v.y, s, a.y), fmaf(v.z, s, a.z), fmaf(v.w, s, a.w));
        if (r.last) store4<O>(dw + row * ld + col, v, there, wide);
        else store4<float>(sums + row * ld_sums + col, v, there, wide_sums);
    }
    __device__ __forceinline__ int rows_of(const Deal&) const { return vocab; }
    __device__ __forceinline__ void block(const Deal& r, int row0, int col0, const Place& at, float (&v)[32]) const {
        if (row0 >= vocab || col0 >= features) return;
        if constexpr (sizeof(O) == 2) {
            if (r.first && r.last && !add) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack2<O>(v[2 * i] * r.scale, v[2 * i + 1] * r.scale);
                store_block(reinterpret_cast<unsigned short*>(dw), ld, vocab, features, row0, col0, at.lane, wide16, at.staging, w);
                return;
            }
        }
        float4 x[8];
        by_columns(at.staging, at.lane, v, x);
        const int row = row0 + at.lane / 8, col = col0 + at.lane % 8 * 4;
        if (!(wide && wide_sums && wide_add && row0 + 32 <= vocab && col0 + 32 <= features)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) put(r, row + 4 * i, col, x[i]);
            return;
        }
        float4 a[8] = {};
        if (!r.first) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = load4(sums + (row + 4 * i) * ld_sums + col, 4, true);
        } else if (add) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = load4(add + (row + 4 * i) * ld_add + col, 4, true);
        }
        const float s = r.scale;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = make_float4(fmaf(x[i].x, s, a[i].x), fmaf(x[i].y, s, a[i].y), fmaf(x[i].z, s, a[i].z), fmaf(x[i].w, s, a[i].w));
        if (r.last) {
#pragma unroll
            for (int i = 0; i < 8; ++i) store4<O>(dw + (row + 4 * i) * ld + col, x[i], 4, true);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) store4<float>(sums + (row + 4 * i) * ld_sums + col, x[i], 4, true);
        }
    }
    __device__ __forceinline__ void tile_at(const Deal& r, int tile, int* m0, int* n0) const {
        *m0 = tile / r.column_tiles * kTile;  // columns first: h stays in L2 while d passes once
        *n0 = tile % r.column_tiles * kTile;
    }
};

// Both in one launch, dh's pieces first: dW's, which are more and shorter, fill what these leave of the pairs' time.
template <typename T, typename O>
struct Gradients {
    static constexpr unsigned int kStatus = 0x200u;
    static constexpr bool kAhead = false, kJoins = false;
    HiddenGrad<T> dh;
    WeightGrad<O> dw;

    struct Deal {
        typename HiddenGrad<T>::Deal dh;
        typename WeightGrad<O>::Deal dw;
    };
    __device__ __forceinline__ void prefetch() const {
        prefetch_map(&dh.d);
        prefetch_map(&dh.w);
        prefetch_map(&dw.d);
        prefetch_map(&dw.h);
    }
    __device__ __forceinline__ Deal deal(int pair, int) const {
        const Dealt t = *dh.dealt;
        return Deal{dh.deal(t, pair), dw.deal(t, pair)};
    }
    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        if (dh.piece(d.dh, q)) return true;
        if (!dw.piece(d.dw, q)) return false;
        q->tile = -1 - q->tile;
        return true;
    }
    // whole tiles to where they belong, parts of split ones to the workspace
    struct Epilogue {
        const Gradients& p;
        const Deal& deal;
        const Piece& q;
        Place at;
        __device__ __forceinline__ Epilogue(const Gradients& p, const Deal& deal, const Piece& q, const Place& at)
            : p(p), deal(deal), q(q), at(at) {}
        __device__ __forceinline__ void chunk(int c, float (&v)[32]) {
            const bool hidden = q.tile >= 0;
            const int row0 = at.row - at.lane, col0 = at.first_column + 32 * c;
            if (q.part < 0) {
                if (hidden) p.dh.block(deal.dh, q.m0 + row0, q.n0 + col0, at, v);
                else p.dw.block(deal.dw, q.m0 + row0, q.n0 + col0, at, v);
                return;
            }
            if (q.m0 + row0 >= (hidden ? p.dh.rows_of(deal.dh) : p.dw.vocab) || q.n0 + col0 >= p.dw.features) return;
            float4 x[8];
            by_columns(at.staging, at.lane, v, x);
            float* to = (hidden ? p.dh.parts : p.dw.parts) + q.part * kPartFloats + (row0 + at.lane / 8) * kTile + col0 +
                        at.lane % 8 * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(to + i * 4 * kTile) = x[i];
        }
        __device__ __forceinline__ void done() {}
    };
};

// Joins the parts of split tiles, 4 rows to a CTA at a time.
constexpr int kJoinRows = 4;
template <typename G>
__device__ __forceinline__ void join_split(const G& g, const typename G::Deal& deal, int rows, int features) {
    if (deal.parts == 1) return;
    const int64_t all = (int64_t)(deal.tiles - deal.whole) * (kTile / kJoinRows);
    const int col = threadIdx.x % 64 * 4;
    for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const int k = (int)(u / (kTile / kJoinRows)), row = (int)(u % (kTile / kJoinRows)) * kJoinRows + threadIdx.x / 64;
        int m0, n0;
        g.tile_at(deal, deal.whole + k, &m0, &n0);
        if (m0 + row >= rows || n0 + col >= features) continue;
        const float* from = g.parts + (int64_t)k * deal.parts * kPartFloats + row * kTile + col;
        float4 s{};
#pragma unroll 8
        for (int part = 0; part < deal.parts; ++part) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from + part * kPartFloats));
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        g.put(deal, m0 + row, n0 + col, s);
    }
}
template <typename T, typename O>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ Gradients<T, O> p) {
    wait_prerequisite();
    allow_dependents();
    const typename Gradients<T, O>::Deal deal = p.deal(0, 0);
    join_split(p.dh, deal.dh, deal.dh.span.rows, p.dh.features);
    join_split(p.dw, deal.dw, p.dw.vocab, p.dw.features);
}

// ------------------------------------------------------------------------------------------------------------------------
// the host side
// ------------------------------------------------------------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// Places in a workspace, one after another, each at a multiple of 256 bytes; without a base only their extent.
class Places {
  public:
    explicit Places(void* base) : base_(static_cast<char*>(base)) {}
    template <typename T>
    T* take(int64_t count) {
        T* p = base_ ? reinterpret_cast<T*>(base_ + at_) : nullptr;
        at_ += round_up(count * (int64_t)sizeof(T), 256);
        return p;
    }
    int64_t bytes() const { return at_; }

  private:
    char* base_;
    int64_t at_ = 0;
};

// Rows of a piece: a multiple of 256, no more than there are or than `bytes` take.
int rows_of_piece(int64_t rows, int64_t bytes_a_row, int64_t bytes, int64_t most) {
    int64_t n = bytes / bytes_a_row / 256 * 256;
    n = n < 256 ? 256 : n > most ? most : n;
    const int64_t need = round_up(rows > 0 ? rows : 1, 256);
    return (int)(n < need ? n : need);
}

struct Room {
    int most;       // rows of a piece
    int pieces;
    Meta* meta;
    Dealt* dealt;
    int* index;
    unsigned short* w;  // a copy with aligned rows, or null
    int64_t ld_w;       // of what is used
    int* target;
    unsigned short* h;
    int ld_h;
    // the logits' sums
    int parts;
    RowSum* sums;
    float* at;
    // gradients
    int ld_d;
    float* coef;
    float* origin;
    unsigned short* d;
    float *dh_parts, *dw_parts;
    float* dw_sums;
    int64_t ld_sums;
    // cross entropy
    bool once;
    Exact* partial;
    float* factor;
    unsigned short* scaled_h;
    int* again;
};

// TMA reads rows that begin at multiples of 16 bytes and whose stride fits 40 bits.
bool readable(const Linear& L) { return rows_aligned(L.w, L.ld_w) && L.ld_w >= L.features && L.ld_w < (int64_t)1 << 39; }

// What a call needs: the forward pass's sums, or gradients, or (cross entropy) both.
Room places_of(const Linear& L, bool sums, const LinearGrad* G, bool ce, int sms, Places* p) {
    Room c{};
    const int grad_rows = rows_of_piece(L.rows, round_up(L.vocab, 64) * 2, kGradBytes, (int64_t)1 << 30);
    const int sum_rows = rows_of_piece(L.rows, tiles_of(L.vocab) * 16, kStatBytes, kMostRows);
    c.most = G && (!sums || grad_rows < sum_rows) ? grad_rows : sum_rows;
    c.pieces = (int)((L.rows + c.most - 1) / c.most);
    if (c.pieces < 1) c.pieces = 1;  // (without rows too: dw is add, the loss 0)
    c.meta = p->take<Meta>(1);
    c.dealt = p->take<Dealt>(1);
    c.index = p->take<int>(L.rows);
    c.target = p->take<int>(c.most);
    c.ld_h = (int)round_up(L.features, 8);
    c.h = p->take<unsigned short>((int64_t)c.most * c.ld_h);
    c.ld_w = L.ld_w;
    if (!readable(L)) {
        c.ld_w = round_up(L.features, 8);
        c.w = p->take<unsigned short>(L.vocab * c.ld_w);
    }
    c.origin = p->take<float>(c.most);
    if (sums) {
        c.parts = (int)((L.vocab + kHalf - 1) / kHalf);
        c.sums = p->take<RowSum>((int64_t)c.parts * c.most);
        c.at = p->take<float>(c.most);
    }
    if (ce) c.partial = p->take<Exact>((int64_t)c.pieces * (c.most / 8));
    c.once = ce && L.dtype == MICA_BF16;  // (kTakenOnce)
    c.ld_d = (int)round_up(L.vocab, 64);
    if (!G) return c;
    const int pairs = sms / 2 < 1 ? 1 : sms / 2;
    c.coef = p->take<float>(c.most);
    c.d = p->take<unsigned short>((int64_t)c.most * c.ld_d);
    if (G->dh) c.dh_parts = p->take<float>(kMostRounds * pairs * kPartFloats);
    if (G->dw) c.dw_parts = p->take<float>(kMostRounds * pairs * kPartFloats);
    if (G->dw && c.pieces > 1 && G->dw_dtype != MICA_F32) {
        c.ld_sums = round_up(L.features, 4);
        c.dw_sums = p->take<float>(L.vocab * c.ld_sums);
    }
    if (c.once) {
        c.factor = p->take<float>(c.most);
        c.scaled_h = p->take<unsigned short>((int64_t)c.most * c.ld_h);
        c.again = p->take<int>(1 + c.most / kTile);
    }
    return c;
}

CUtensorMapDataType map_type(int32_t dtype) {
    return dtype == MICA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

#define MICA_STEP(x)                              \
    do {                                          \
        const cudaError_t step_e = (x);           \
        if (step_e != cudaSuccess) return step_e; \
    } while (0)

cudaError_t copy_w(const Linear& L, const Room& c, void* stream) {
    if (!c.w) return cudaSuccess;
    const int64_t ctas = (L.vocab * (c.ld_w / 8) + 255) / 256;
    return launch_after(align_rows_kernel, ctas < (1 << 16) ? ctas : (1 << 16), 256, 0, stream,
                        static_cast<const unsigned short*>(L.w), L.ld_w, (int64_t)L.vocab, (int64_t)L.features, c.w, c.ld_w);
}

// One call: logps and lse where given (with sums), gradients where G is, from dlogps and lse_in or as cross entropy's.
struct Call {
    const Linear& L;
    const LinearGrad* G;
    const float* lse_in;
    const float* dlogps;
    float* logps;
    float* lse;
    float* loss;  // null: not cross entropy
    double denom, grad_scale;
    int sms;
    void* stream;
};

template <typename T>
cudaError_t gather(const Call& call, const Room& c, int piece) {
    const Linear& L = call.L;
    Gather g{};
    g.targets = L.targets;
    g.h = static_cast<const unsigned short*>(L.h);
    g.ld_h = L.ld_h;
    g.rows = (int)L.rows;
    g.features = L.features;
    g.vocab = L.vocab;
    g.wide = L.wide_targets;
    g.aligned = reinterpret_cast<uintptr_t>(L.h) % 16 == 0 && L.ld_h % 8 == 0;
    g.dlogps = call.dlogps;
    g.lse = call.lse_in;
    g.inv_t = (float)(1.0 / L.temperature);
    g.ce_factor = (float)(-call.grad_scale / L.temperature);
    g.denom = (float)call.denom;
    g.scaled = L.dtype == MICA_F16 || c.once;
    g.scaled_to = c.once ? -1 : 14;
    g.most = c.most;
    g.piece = piece;
    g.meta = c.meta;
    g.dealt = c.dealt;
    g.pairs = call.sms / 2 < 1 ? 1 : call.sms / 2;
    g.has_dh = call.G && call.G->dh;
    g.has_dw = call.G && call.G->dw;
    g.index = c.index;
    g.out = c.h;
    g.ld = c.ld_h;
    g.target = c.target;
    g.coef = c.coef;
    g.origin = c.origin;
    g.a = (float)(1.4426950408889634074 / L.temperature);
    if (c.once) {
        g.w = c.w ? c.w : static_cast<const unsigned short*>(L.w);
        g.ld_w = c.ld_w;
        g.again = c.again;
    }
    g.logps = call.logps;
    g.lse_out = call.lse;
    if (call.G) {
        g.zero = static_cast<unsigned short*>(call.G->dh);
        g.ld_zero = call.G->ld_dh;
    }
    const int64_t ctas = (L.rows + 7) / 8, most = 4 * (int64_t)call.sms;
    if (L.rows <= kLookRows) return launch_after(look_kernel<T>, ctas < 1 ? 1 : ctas, 256, 0, call.stream, g);
    if (piece == 0) MICA_STEP(launch_after(scan_kernel, 1, 1024, 0, call.stream, g));
    return launch_after(gather_kernel<T>, ctas < most ? ctas : most, 256, 0, call.stream, g);
}

// What the products over the vocabulary share.
bool fill(Logits* p, const Linear& L, const Room& c) {
    p->dealt = c.dealt;
    p->target = c.target;
    p->vocab = L.vocab;
    p->across = (int)tiles_of(L.vocab);
    p->stages = (L.features + kDepth - 1) / kDepth;
    p->a = (float)(1.4426950408889634074 / L.temperature);
    return matrix_map(&p->h, map_type(L.dtype), c.h, L.features, c.most, c.ld_h, 1) &&
           matrix_map(&p->w, map_type(L.dtype), c.w ? c.w : L.w, L.features, L.vocab, c.ld_w, 1);
}

template <typename T>
cudaError_t join_rows(const Call& call, const Room& c, int piece) {
    Join j{};
    j.meta = c.meta;
    j.index = c.index;
    j.target = c.target;
    j.sums = c.sums;
    j.most = c.most;
    j.piece = piece;
    j.parts = c.parts;
    j.a = (float)(1.4426950408889634074 / call.L.temperature);
    j.logps = call.logps;
    j.lse = call.lse;
    j.at = c.at;
    j.origin = call.G || c.once ? c.origin : nullptr;
    j.once = c.once;
    j.at_target = c.at;
    j.factor = c.factor;
    j.again = c.again;
    j.d = c.d;
    j.ld_d = c.ld_d;
    j.h = c.h;
    j.scaled_h = c.scaled_h;
    j.ld_h = c.ld_h;
    j.features = call.L.features;
    j.loss = call.loss;
    j.denom = (float)call.denom;
    j.partial = c.partial;
    j.all = c.pieces * (c.most / 8);
    return launch_after(join_rows_kernel<T>, c.most / 8, 256, 0, call.stream, j);
}

template <typename T, typename O>
cudaError_t gradients(const Call& call, const Room& c) {
    const Linear& L = call.L;
    const LinearGrad& G = *call.G;
    Gradients<T, O> p{};
    const auto type = map_type(L.dtype);
    CUtensorMap d;
    if (!matrix_map(&d, type, c.d, L.vocab, c.most, c.ld_d, 1)) return cudaErrorInvalidValue;
    HiddenGrad<T>& x = p.dh;
    x.d = d;
    x.dealt = c.dealt;
    x.index = c.index;
    x.features = L.features;
    x.factor = c.factor;
    x.dh = static_cast<T*>(G.dh);
    x.ld = G.ld_dh;
    x.wide = reinterpret_cast<uintptr_t>(G.dh) % 8 == 0 && G.ld_dh % 4 == 0;
    x.wide16 = reinterpret_cast<uintptr_t>(G.dh) % 16 == 0 && G.ld_dh % 8 == 0;
    x.parts = c.dh_parts;
    if (!matrix_map(&x.w, type, c.w ? c.w : L.w, L.features, L.vocab, c.ld_w, 1)) return cudaErrorInvalidValue;
    WeightGrad<O>& y = p.dw;
    y.d = d;
    y.most = c.most;
    y.vocab = L.vocab;
    y.features = L.features;
    y.dw = static_cast<O*>(G.dw);
    y.ld = G.ld_dw;
    y.add = static_cast<const O*>(G.add);
    y.ld_add = G.ld_add;
    y.sums = sizeof(O) == 4 ? static_cast<float*>(G.dw) : c.dw_sums;
    y.ld_sums = sizeof(O) == 4 ? G.ld_dw : c.ld_sums;
    const size_t four = 4 * sizeof(O);
    y.wide = reinterpret_cast<uintptr_t>(G.dw) % four == 0 && G.ld_dw % 4 == 0;
    y.wide16 = reinterpret_cast<uintptr_t>(G.dw) % 16 == 0 && G.ld_dw % 8 == 0;
    y.wide_add = reinterpret_cast<uintptr_t>(G.add) % four == 0 && G.ld_add % 4 == 0;
    y.wide_sums = sizeof(O) == 4 ? y.wide : 1;
    y.parts = c.dw_parts;
    if (!matrix_map(&y.h, type, c.once ? c.scaled_h : c.h, L.features, c.most, c.ld_h, 1)) return cudaErrorInvalidValue;
    const int pairs = call.sms / 2 < 1 ? 1 : call.sms / 2;
    MICA_STEP((launch_gemm<T>(p, pairs, call.sms, call.stream)));
    // no tile of a sum this short is split
    const bool short_dh = !G.dh || (L.vocab + kDepth - 1) / kDepth < 2 * kLeastStages;
    const bool short_dw = !G.dw || (L.rows + kDepth - 1) / kDepth < 2 * kLeastStages;
    if (short_dh && short_dw) return cudaSuccess;
    return launch_after(join_parts_kernel<T, O>, 8 * (int64_t)call.sms, 256, 0, call.stream, p);
}

// Tiles of the product over the vocabulary, of a whole piece.
int64_t logit_tiles(const Linear& L, const Room& c) { return c.most / kTile * tiles_of(L.vocab); }

// Cross entropy's product taken once, and again for rows whose sum has left its range.
cudaError_t logits_once(const Call& call, const Room& c, int piece) {
    LogitOnce p{};
    if (!fill(&p, call.L, c)) return cudaErrorInvalidValue;
    p.sums = c.sums;
    p.parts = c.parts;
    p.origin = c.origin;
    p.d = reinterpret_cast<LogitOnce::T*>(c.d);
    p.ld = c.ld_d;
    MICA_STEP((launch_gemm<LogitOnce::T>(p, logit_tiles(call.L, c), call.sms, call.stream)));
    MICA_STEP(join_rows<LogitOnce::T>(call, c, piece));
    if (!call.G) return cudaSuccess;
    p.sums = nullptr;
    p.at = c.at;
    p.again = c.again;
    return launch_gemm<LogitOnce::T>(p, logit_tiles(call.L, c), call.sms, call.stream);
}

template <typename T>
cudaError_t run(const Call& call, const Room& c) {
    const Linear& L = call.L;
    const bool forward = call.logps || call.loss;
    const int64_t tiles = logit_tiles(L, c);
    MICA_STEP(copy_w(L, c, call.stream));
    for (int piece = 0; piece < c.pieces; ++piece) {
        MICA_STEP(gather<T>(call, c, piece));
        if constexpr (kTakenOnce<T>) {
            if (c.once) MICA_STEP(logits_once(call, c, piece));
        }
        if (forward && !c.once) {
            LogitSums p{};
            if (!fill(&p, L, c)) return cudaErrorInvalidValue;
            p.sums = c.sums;
            p.parts = c.parts;
            p.at = c.at;
            MICA_STEP((launch_gemm<T>(p, tiles, call.sms, call.stream)));
            MICA_STEP(join_rows<T>(call, c, piece));
        }
        if (!call.G) continue;
        if (!c.once) {
            LogitGrad<T> p{};
            if (!fill(&p, L, c)) return cudaErrorInvalidValue;
            p.coef = c.coef;
            p.origin = c.origin;
            p.d = reinterpret_cast<T*>(c.d);
            p.ld = c.ld_d;
            MICA_STEP((launch_gemm<T>(p, tiles, call.sms, call.stream)));
        }
        const int32_t type = call.G->dw ? call.G->dw_dtype : L.dtype;
        MICA_STEP((type == MICA_F32   ? gradients<T, float>(call, c)
                   : type == MICA_F16 ? gradients<T, __half>(call, c)
                                      : gradients<T, __nv_bfloat16>(call, c)));
    }
    return cudaSuccess;
}

int run_typed(const Call& call, const Room& c) {
    return (int)(call.L.dtype == MICA_BF16 ? run<__nv_bfloat16>(call, c) : run<__half>(call, c));
}

}  // namespace

int64_t linear_logps_workspace(const Linear& L) {
    if (L.rows == 0) return 0;
    Places p(nullptr);
    places_of(L, true, nullptr, false, 1, &p);
    return p.bytes();
}

int launch_linear_logps(const Linear& L, float* logps, float* lse, void* workspace, int sms, void* stream) {
    Places p(workspace);
    const Room c = places_of(L, true, nullptr, false, sms, &p);
    return run_typed(Call{L, nullptr, nullptr, nullptr, logps, lse, nullptr, 0.0, 0.0, sms, stream}, c);
}

int64_t linear_grad_workspace(const Linear& L, const LinearGrad& G, int sms) {
    Places p(nullptr);
    places_of(L, false, &G, false, sms, &p);
    return p.bytes();
}

int launch_linear_grad(const Linear& L, const float* lse, const float* dlogps, const LinearGrad& G, void* workspace, int sms,
                       void* stream) {
    Places p(workspace);
    const Room c = places_of(L, false, &G, false, sms, &p);
    return run_typed(Call{L, &G, lse, dlogps, nullptr, nullptr, nullptr, 0.0, 0.0, sms, stream}, c);
}

int64_t linear_ce_workspace(const Linear& L, const LinearGrad& G, int sms) {
    Places p(nullptr);
    places_of(L, true, G.dh || G.dw ? &G : nullptr, true, sms, &p);
    return p.bytes();
}

int launch_linear_ce(const Linear& L, double denom, double grad_scale, float* loss, float* logps, const LinearGrad& G,
                     void* workspace, int sms, void* stream) {
    Places p(workspace);
    const LinearGrad* g = G.dh || G.dw ? &G : nullptr;
    const Room c = places_of(L, true, g, true, sms, &p);
    return run_typed(Call{L, g, nullptr, nullptr, logps, nullptr, loss, denom, grad_scale, sms, stream}, c);
}

int read_linear_status(unsigned int* status) { return (int)read_gemm_status(status); }

}  // namespace mica
