// Losses from hidden states h (rows x features) and an output embedding W (vocabulary x features): log-probabilities of given
// tokens under the softmax of z = h W^T / T, and their gradients, without a matrix of logits.
//
//   forward   lse_i = log sum_j exp z_ij, logp_i = z_i,target - lse_i
//   gradient  d_ij = c_i (1[j = target] - exp(z_ij - lse_i)), c_i = dlogps_i / T; dh = d W, dW = d^T h
//
// The rows that count are gathered first, so that unscored rows (prompts) cost nothing, and taken in pieces of at most
// kGradBytes of d. The forward pass is one product over all of the vocabulary whose epilogue keeps a running maximum and sum
// for each row; the gradient takes the product again (a third more of the operations; keeping the logits would take memory
// that grows with rows x vocabulary), rounds d to 16 bits once, in its epilogue, and multiplies it with W and with h.
//
// Logits, maxima, sums and gradients' sums are float32. d is rounded to the operands' type because the tensor cores multiply
// what they are given in 16 bits: relative 2^-9 (bfloat16) or 2^-12 of each of its elements on average. binary16 has not the
// range for d, so it is scaled by a power of two that brings the largest |c_i| to 2^15 (d is at most |c_i|), which the
// gradients' epilogues take out again.
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "linear.h"

namespace mica {
namespace {

constexpr int kScanThreads = 1024, kScanItems = 8;
constexpr int64_t kGradBytes = (int64_t)1 << 30;   // of d, that a piece of the rows takes
constexpr int64_t kStatBytes = (int64_t)256 << 20;  // of the forward pass's maxima and sums
constexpr int kMostRows = 16384;                    // of a piece in the forward pass
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What the scan of the targets leaves for the kernels after it.
struct Meta {
    int count;        // rows that count
    float coef;       // cross entropy: every row's coefficient, with the scale of d in it
    float scale;      // of d
    float inv_scale;
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

__device__ __forceinline__ int64_t target_at(const void* targets, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(targets)[i] : static_cast<const int32_t*>(targets)[i];
}

// ------------------------------------------------------------------------------------------------------------------------
// which rows count
// ------------------------------------------------------------------------------------------------------------------------

struct Scan {
    const void* targets;
    int wide, rows;
    const float* dlogps;  // or null: a row whose dlogps is 0 does not count
    float* logps;         // or null; logps and lse of rows that do not count are 0
    float* lse;           // or null
    int* index;           // the rows that count, in order, and after them, backwards, the others
    Meta* meta;
    float inv_t;
    float ce_factor;      // cross entropy: -grad_scale / T, divided by `denom` or, where that is 0, by the count
    float denom;
    int scaled;           // d is scaled
};

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// One CTA: a few microseconds for 8,192 rows.
__global__ void __launch_bounds__(kScanThreads) scan_kernel(Scan s) {
    __shared__ int sums[32];
    __shared__ float tops[32];
    wait_prerequisite();
    allow_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int before = 0;
    float top = 0.0f;
    for (int base = 0; base < s.rows; base += kScanThreads * kScanItems) {
        const int first = base + threadIdx.x * kScanItems;
        uint32_t on = 0;
#pragma unroll
        for (int k = 0; k < kScanItems; ++k) {
            const int i = first + k;
            if (i >= s.rows || target_at(s.targets, s.wide, i) < 0) continue;
            const float c = s.dlogps ? s.dlogps[i] : 1.0f;
            if (c == 0.0f) continue;
            on |= 1u << k;
            if (fabsf(c) > top || c != c) top = fabsf(c);  // (a NaN stays: nothing is larger)
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
        for (int k = 0; k < kScanItems; ++k) {
            const int i = first + k;
            if (i >= s.rows) break;
            if (on >> k & 1) {
                s.index[at++] = i;
            } else {
                s.index[s.rows - 1 - (i - at)] = i;
                if (s.logps) s.logps[i] = 0.0f;
                if (s.lse) s.lse[i] = 0.0f;
            }
        }
        before += all;
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        const float v = __shfl_xor_sync(~0u, top, d);
        if (v > top || v != v) top = v;
    }
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 0; i < 32; ++i)
        if (tops[i] > top || tops[i] != tops[i]) top = tops[i];
    Meta m{before, 0.0f, 1.0f, 1.0f};
    const float ce = s.ce_factor / (s.denom > 0.0f ? s.denom : (float)before);
    const float most = s.dlogps ? top * s.inv_t : fabsf(ce);
    if (s.scaled && most > 0.0f && most < INFINITY) {
        int e = (int)(__float_as_uint(most) >> 23) - 127;  // most < 2^(e + 1); a subnormal counts as 2^-127
        e = 14 - (e < -100 ? -100 : e);
        m.scale = power_of_two(e);
        m.inv_scale = power_of_two(-e);
    }
    m.coef = ce * m.scale;
    *s.meta = m;
}

// ------------------------------------------------------------------------------------------------------------------------
// the rows that count, side by side
// ------------------------------------------------------------------------------------------------------------------------

struct Gather {
    const unsigned short* h;
    const void* targets;
    int64_t ld_h;
    int rows, features, vocab, wide, aligned;
    const int* index;
    const Meta* meta;
    int most, piece;
    const float* lse;      // or null
    const float* dlogps;   // or null
    float inv_t;
    unsigned short* out;   // [most][ld]
    int ld;
    int* target;           // [most] -1: past the vocabulary
    float* coef;           // [most] c * scale, or null
    float* origin;         // [most] lse * log2(e)
    unsigned short* zero;  // rows that do not count get zeros here, or null
    int64_t ld_zero;
};

// A warp to a row. Rows up to the next multiple of 64 are zeros: the weight gradient adds them up.
__global__ void __launch_bounds__(256) gather_kernel(Gather g) {
    wait_prerequisite();
    allow_dependents();
    const Meta m = *g.meta;
    const Span span = span_of(m.count, g.most, g.piece);
    const int lane = threadIdx.x % 32, padded = (span.rows + 63) / 64 * 64;
    const int others = g.zero && g.piece == 0 ? g.rows - m.count : 0;
    for (int64_t r = blockIdx.x * 8ll + threadIdx.x / 32; r < padded + others; r += gridDim.x * 8ll) {
        if (r >= padded) {
            unsigned short* to = g.zero + (int64_t)g.index[g.rows - 1 - (r - padded)] * g.ld_zero;
            for (int c = lane; c < g.features; c += 32) to[c] = 0;
            continue;
        }
        unsigned short* to = g.out + r * g.ld;
        if (r >= span.rows) {
            for (int c = lane; c < g.ld / 8; c += 32) reinterpret_cast<uint4*>(to)[c] = uint4{};
            continue;
        }
        const int64_t i = g.index[span.from + r];
        const unsigned short* from = g.h + i * g.ld_h;
        const int whole = g.aligned ? g.features / 8 : 0;
        for (int c = lane; c < whole; c += 32) reinterpret_cast<uint4*>(to)[c] = reinterpret_cast<const uint4*>(from)[c];
        for (int c = whole * 8 + lane; c < g.features; c += 32) to[c] = from[c];
        if (lane == 0) {
            const int64_t y = target_at(g.targets, g.wide, i);
            g.target[r] = y < g.vocab ? (int)y : -1;
            if (g.coef) {
                g.coef[r] = y >= g.vocab ? NAN : g.dlogps ? g.dlogps[i] * g.inv_t * m.scale : m.coef;
                g.origin[r] = g.lse[i] * kLog2E;
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------------------------------
// the logits' product, forward
// ------------------------------------------------------------------------------------------------------------------------

// A row's part of the vocabulary: sum 2^(z a - origin), with z a in units of log 2.
struct RowSum {
    float origin, sum;
};

struct Logits {
    static constexpr unsigned int kStatus = 0x100u;
    static constexpr bool kAhead = false;
    CUtensorMap h, w;
    const Meta* meta;
    const int* target;
    int most, piece_index, vocab, stages;
    float a;  // log2(e) / T

    struct Deal {
        int rows, row_tiles, pieces, next, pairs;
    };
    __device__ __forceinline__ Deal deal(int pair, int pairs) const {
        const int rows = span_of(meta->count, most, piece_index).rows, row_tiles = (rows + kTile - 1) / kTile;
        return Deal{rows, row_tiles, row_tiles * ((vocab + kTile - 1) / kTile), pair, pairs};
    }
    // rows first: h stays in L2 while W passes once
    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        const int i = d.next;
        if (i >= d.pieces) return false;
        d.next += d.pairs;
        *q = Piece{{&h, 0, true}, {&w, 0, true}, i % d.row_tiles * kTile, i / d.row_tiles * kTile, kTile, 0, stages, i, -1, 0, 0};
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
            : p(p), row(q.m0 + at.row), column(q.n0 + at.first_column), s{-1e38f, 0.0f} {
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

struct Join {
    const Meta* meta;
    const int* index;
    const int* target;
    const RowSum* sums;
    const float* at;
    int most, piece, parts;
    float a;
    float* logps;
    float* lse;  // or null
};

__device__ __forceinline__ RowSum operator+(RowSum x, RowSum y) {
    const float o = fmaxf(x.origin, y.origin);
    return RowSum{o, x.sum * exp2_fast(x.origin - o) + y.sum * exp2_fast(y.origin - o)};
}

// A warp to a row; joined in a fixed order.
__global__ void __launch_bounds__(256) join_rows_kernel(Join j) {
    wait_prerequisite();
    allow_dependents();
    const Span span = span_of(j.meta->count, j.most, j.piece);
    const int lane = threadIdx.x % 32, row = blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= span.rows) return;
    RowSum s{-1e38f, 0.0f};
    const RowSum* own = j.sums + (int64_t)row * j.parts;
#pragma unroll 4
    for (int k = lane; k < j.parts; k += 32) s = s + own[k];
#pragma unroll
    for (int d = 16; d; d /= 2)
        s = s + RowSum{__shfl_xor_sync(~0u, s.origin, d), __shfl_xor_sync(~0u, s.sum, d)};
    if (lane) return;
    const int64_t i = j.index[span.from + row];
    const float l = log2f(s.sum);
    j.logps[i] = j.target[row] < 0 ? NAN : (fmaf(j.at[row], j.a, -s.origin) - l) * kLn2;
    if (j.lse) j.lse[i] = (s.origin + l) * kLn2;
}

// A float32 sum with what its rounding left out.
struct Exact {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
};

// loss = -sum logps / denom, or / the scored rows' number; rows that do not count hold zeros
__global__ void __launch_bounds__(1024) loss_kernel(const float* logps, int rows, const Meta* meta, float denom, float* loss) {
    __shared__ Exact part[1024];
    wait_prerequisite();
    allow_dependents();
    Exact e;
    for (int i = threadIdx.x; i < rows; i += 1024) e.add(logps[i]);
    part[threadIdx.x] = e;
    for (int n = 512; n; n /= 2) {
        __syncthreads();
        if (threadIdx.x < n) {
            Exact x = part[threadIdx.x];
            x.add(part[threadIdx.x + n].hi);
            x.lo += part[threadIdx.x + n].lo;
            part[threadIdx.x] = x;
        }
    }
    if (threadIdx.x) return;
    const int count = meta->count;
    const float sum = part[0].hi == part[0].hi && fabsf(part[0].hi) < INFINITY ? part[0].hi + part[0].lo : part[0].hi;
    *loss = count ? -sum / (denom > 0.0f ? denom : (float)count) : 0.0f;
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
            live = row < d.rows;
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

template <typename T>
struct HiddenGrad {
    static constexpr unsigned int kStatus = 0x200u;
    static constexpr bool kAhead = false;
    CUtensorMap d, w;
    const Meta* meta;
    const int* index;
    int most, piece_index, vocab, features;
    T* dh;
    int64_t ld;
    int wide, wide16;  // rows aligned for stores of four elements, of eight
    float* parts;

    struct Deal : SplitDeal {
        Span span;
        int column_tiles;
        float scale;
    };
    __device__ __forceinline__ Deal deal(int pair, int pairs) const {
        const Meta m = *meta;
        const Span span = span_of(m.count, most, piece_index);
        const int column_tiles = (features + kTile - 1) / kTile;
        Deal r;
        static_cast<SplitDeal&>(r) = split_deal((span.rows + kTile - 1) / kTile * column_tiles, (vocab + kDepth - 1) / kDepth,
                                                pair, pairs);
        r.span = span;
        r.column_tiles = column_tiles;
        r.scale = m.inv_scale;
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
    // four sums of a row
    __device__ __forceinline__ void put(const Deal& r, int row, int col, float4 v) const {
        if (row >= r.span.rows || col >= features) return;
        const float s = r.scale;
        store4<T>(dh + index[r.span.from + row] * ld + col, make_float4(v.x * s, v.y * s, v.z * s, v.w * s), features - col,
                  wide);
    }
    // a warp's 32 x 32 of them
    __device__ __forceinline__ void block(const Deal& r, int row0, int col0, const Place& at, float (&v)[32]) const {
        if (row0 >= r.span.rows || col0 >= features) return;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<T>(v[2 * i] * r.scale, v[2 * i + 1] * r.scale);
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
    static constexpr unsigned int kStatus = 0x400u;
    static constexpr bool kAhead = false;
    CUtensorMap d, h;
    const Meta* meta;
    int most, piece_index, vocab, features;
    O* dw;
    int64_t ld;
    const O* add;  // or null
    int64_t ld_add;
    float* sums;   // null where there is one piece only
    int64_t ld_sums;
    int wide, wide16, wide_add, wide_sums;
    float* parts;

    struct Deal : SplitDeal {
        int column_tiles, first_stage;
        bool first, last, none;
        float scale;
    };
    __device__ __forceinline__ Deal deal(int pair, int pairs) const {
        const Meta m = *meta;
        const Span span = span_of(m.count, most, piece_index);
        const int column_tiles = (features + kTile - 1) / kTile;
        Deal r;
        const int stages = (span.rows + kDepth - 1) / kDepth;
        r.none = span.rows == 0 && piece_index > 0;
        static_cast<SplitDeal&>(r) = split_deal(r.none ? 0 : (vocab + kTile - 1) / kTile * column_tiles, stages ? stages : 1, pair, pairs);
        r.first_stage = stages ? 0 : most / kDepth;  // without rows: past the matrices, where zeros are read
        r.column_tiles = column_tiles;
        r.first = piece_index == 0;
        r.last = last_span(m.count, most, piece_index);
        r.scale = m.inv_scale;
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
        v = make_float4(fmaf(v.x, s, a.x), fmaf(v.y, s, a.y), fmaf(v.z, s, a.z), fmaf(v.w, s, a.w));  // (s: a power of two)
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

// The epilogue of both: whole tiles to where they belong, parts of split ones to the workspace.
template <typename G>
struct Split : G {
    struct Epilogue {
        const Split& p;
        const typename G::Deal& deal;
        const Piece& q;
        Place at;
        __device__ __forceinline__ Epilogue(const Split& p, const typename G::Deal& deal, const Piece& q, const Place& at)
            : p(p), deal(deal), q(q), at(at) {}
        __device__ __forceinline__ void chunk(int c, float (&v)[32]) {
            const int row0 = at.row - at.lane, col0 = at.first_column + 32 * c;
            if (q.part < 0) {
                p.block(deal, q.m0 + row0, q.n0 + col0, at, v);
                return;
            }
            if (q.m0 + row0 >= p.rows_of(deal) || q.n0 + col0 >= p.features) return;
            float4 x[8];
            by_columns(at.staging, at.lane, v, x);
            float* to = p.parts + q.part * kPartFloats + (row0 + at.lane / 8) * kTile + col0 + at.lane % 8 * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(to + i * 4 * kTile) = x[i];
        }
        __device__ __forceinline__ void done() {}
    };
};

// Joins the parts of split tiles, 4 rows to a CTA at a time.
constexpr int kJoinRows = 4;
template <typename G>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ Split<G> p, int pairs) {
    wait_prerequisite();
    allow_dependents();
    const typename G::Deal deal = p.deal(0, pairs);
    if (deal.parts == 1) return;
    const int64_t all = (int64_t)(deal.tiles - deal.whole) * (kTile / kJoinRows);
    const int col = threadIdx.x % 64 * 4;
    for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const int k = (int)(u / (kTile / kJoinRows)), row = (int)(u % (kTile / kJoinRows)) * kJoinRows + threadIdx.x / 64;
        int m0, n0;
        p.tile_at(deal, deal.whole + k, &m0, &n0);
        if (m0 + row >= p.rows_of(deal) || n0 + col >= p.features) continue;
        const float* from = p.parts + (int64_t)k * deal.parts * kPartFloats + row * kTile + col;
        float4 s{};
#pragma unroll 8
        for (int part = 0; part < deal.parts; ++part) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from + part * kPartFloats));
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        p.put(deal, m0 + row, n0 + col, s);
    }
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

struct Common {
    Meta* meta;
    int* index;
    unsigned short* w;  // a copy with aligned rows, or null
    int64_t ld_w;       // of what is used
    int* target;
    unsigned short* h;
    int ld_h;
};
struct ForwardPlaces {
    int most, parts;
    RowSum* sums;
    float* at;
};
struct GradPlaces {
    int most, ld;
    float* coef;
    float* origin;
    unsigned short* d;
    float* parts;
    float* sums;
    int64_t ld_sums;
};

// TMA reads rows that begin at multiples of 16 bytes and whose stride fits 40 bits.
bool readable(const Linear& L) { return rows_aligned(L.w, L.ld_w) && L.ld_w >= L.features && L.ld_w < (int64_t)1 << 39; }

int forward_rows(const Linear& L) { return rows_of_piece(L.rows, tiles_of(L.vocab) * 16, kStatBytes, kMostRows); }
int grad_rows(const Linear& L) { return rows_of_piece(L.rows, round_up(L.vocab, 64) * 2, kGradBytes, (int64_t)1 << 30); }

Common place_common(const Linear& L, int most, Places* p) {
    Common c{};
    c.meta = p->take<Meta>(1);
    c.index = p->take<int>(L.rows);
    c.target = p->take<int>(most);
    c.ld_h = (int)round_up(L.features, 8);
    c.h = p->take<unsigned short>((int64_t)most * c.ld_h);
    c.ld_w = L.ld_w;
    if (!readable(L)) {
        c.ld_w = round_up(L.features, 8);
        c.w = p->take<unsigned short>(L.vocab * c.ld_w);
    }
    return c;
}
ForwardPlaces place_forward(const Linear& L, Places* p) {
    ForwardPlaces f{};
    f.most = forward_rows(L);
    f.parts = (int)((L.vocab + kHalf - 1) / kHalf);
    f.sums = p->take<RowSum>((int64_t)f.parts * f.most);
    f.at = p->take<float>(f.most);
    return f;
}
GradPlaces place_grad(const Linear& L, const LinearGrad& G, int sms, Places* p) {
    GradPlaces g{};
    g.most = grad_rows(L);
    g.ld = (int)round_up(L.vocab, 64);
    g.coef = p->take<float>(g.most);
    g.origin = p->take<float>(g.most);
    g.d = p->take<unsigned short>((int64_t)g.most * g.ld);
    const int pairs = sms / 2 < 1 ? 1 : sms / 2;
    g.parts = p->take<float>(kMostRounds * pairs * kPartFloats);
    if (G.dw && L.rows > g.most && G.dw_dtype != MICA_F32) {
        g.ld_sums = round_up(L.features, 4);
        g.sums = p->take<float>(L.vocab * g.ld_sums);
    }
    return g;
}

CUtensorMapDataType map_type(int32_t dtype) {
    return dtype == MICA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

#define MICA_STEP(x)                             \
    do {                                         \
        const cudaError_t step_e = (x);          \
        if (step_e != cudaSuccess) return step_e; \
    } while (0)

cudaError_t copy_w(const Linear& L, const Common& c, void* stream) {
    if (!c.w) return cudaSuccess;
    const int64_t ctas = (L.vocab * (c.ld_w / 8) + 255) / 256;
    return launch_after(align_rows_kernel, ctas < (1 << 16) ? ctas : (1 << 16), 256, 0, stream,
                        static_cast<const unsigned short*>(L.w), L.ld_w, (int64_t)L.vocab, (int64_t)L.features, c.w, c.ld_w);
}

cudaError_t gather(const Linear& L, const Common& c, int most, int piece, const float* lse, const float* dlogps,
                   const GradPlaces* g, const LinearGrad* G, void* stream) {
    Gather a{};
    a.h = static_cast<const unsigned short*>(L.h);
    a.targets = L.targets;
    a.ld_h = L.ld_h;
    a.rows = (int)L.rows;
    a.features = L.features;
    a.vocab = L.vocab;
    a.wide = L.wide_targets;
    a.aligned = reinterpret_cast<uintptr_t>(L.h) % 16 == 0 && L.ld_h % 8 == 0;
    a.index = c.index;
    a.meta = c.meta;
    a.most = most;
    a.piece = piece;
    a.lse = lse;
    a.dlogps = dlogps;
    a.inv_t = (float)(1.0 / L.temperature);
    a.out = c.h;
    a.ld = c.ld_h;
    a.target = c.target;
    if (g) {
        a.coef = g->coef;
        a.origin = g->origin;
    }
    if (G && G->dh && piece == 0) {
        a.zero = static_cast<unsigned short*>(G->dh);
        a.ld_zero = G->ld_dh;
    }
    const int64_t ctas = ((a.zero ? L.rows + 64 : most) + 7) / 8;
    return launch_after(gather_kernel, ctas < 4096 ? ctas : 4096, 256, 0, stream, a);
}

// What both products over the vocabulary share.
bool fill(Logits* p, const Linear& L, const Common& c, int most, int piece) {
    p->meta = c.meta;
    p->target = c.target;
    p->most = most;
    p->piece_index = piece;
    p->vocab = L.vocab;
    p->stages = (L.features + kDepth - 1) / kDepth;
    p->a = (float)(1.4426950408889634074 / L.temperature);
    return matrix_map(&p->h, map_type(L.dtype), c.h, L.features, most, c.ld_h, 1) &&
           matrix_map(&p->w, map_type(L.dtype), c.w ? c.w : L.w, L.features, L.vocab, c.ld_w, 1);
}

template <typename T>
cudaError_t forward(const Linear& L, const Common& c, const ForwardPlaces& f, float* logps, float* lse, int sms, void* stream) {
    for (int64_t at = 0, piece = 0; at < L.rows; at += f.most, ++piece) {
        MICA_STEP(gather(L, c, f.most, (int)piece, nullptr, nullptr, nullptr, nullptr, stream));
        LogitSums p{};
        if (!fill(&p, L, c, f.most, (int)piece)) return cudaErrorInvalidValue;
        p.sums = f.sums;
        p.parts = f.parts;
        p.at = f.at;
        MICA_STEP((launch_gemm<T>(p, f.most / kTile * tiles_of(L.vocab), sms, stream)));
        const Join j{c.meta, c.index, c.target, f.sums, f.at, f.most, (int)piece, f.parts, p.a, logps, lse};
        MICA_STEP(launch_after(join_rows_kernel, f.most / 8, 256, 0, stream, j));
    }
    return cudaSuccess;
}

// stages: how many there can be at most
template <typename T, typename G>
cudaError_t split_product(const Split<G>& p, int64_t tiles, int64_t stages, int sms, void* stream) {
    const int pairs = sms / 2 < 1 ? 1 : sms / 2;
    MICA_STEP((launch_gemm<T>(p, pairs, sms, stream)));
    if (stages < 2 * kLeastStages) return cudaSuccess;  // no tile is split
    const int64_t ctas = (tiles < pairs ? tiles : pairs) * (kTile / kJoinRows);
    return launch_after(join_parts_kernel<G>, ctas, 256, 0, stream, p, pairs);
}

template <typename T, typename O>
cudaError_t weight_grad(const Linear& L, const Common& c, const GradPlaces& g, const LinearGrad& G, int piece, int sms,
                        void* stream) {
    Split<WeightGrad<O>> p{};
    p.meta = c.meta;
    p.most = g.most;
    p.piece_index = piece;
    p.vocab = L.vocab;
    p.features = L.features;
    p.dw = static_cast<O*>(G.dw);
    p.ld = G.ld_dw;
    p.add = static_cast<const O*>(G.add);
    p.ld_add = G.ld_add;
    p.sums = sizeof(O) == 4 ? static_cast<float*>(G.dw) : g.sums;
    p.ld_sums = sizeof(O) == 4 ? G.ld_dw : g.ld_sums;
    const size_t four = 4 * sizeof(O);
    p.wide = reinterpret_cast<uintptr_t>(G.dw) % four == 0 && G.ld_dw % 4 == 0;
    p.wide16 = reinterpret_cast<uintptr_t>(G.dw) % 16 == 0 && G.ld_dw % 8 == 0;
    p.wide_add = reinterpret_cast<uintptr_t>(G.add) % four == 0 && G.ld_add % 4 == 0;
    p.wide_sums = sizeof(O) == 4 ? p.wide : 1;
    p.parts = g.parts;
    if (!matrix_map(&p.d, map_type(L.dtype), g.d, L.vocab, g.most, g.ld, 1) ||
        !matrix_map(&p.h, map_type(L.dtype), c.h, L.features, g.most, c.ld_h, 1))
        return cudaErrorInvalidValue;
    return split_product<T>(p, tiles_of(L.vocab) * tiles_of(L.features), (L.rows + kDepth - 1) / kDepth, sms, stream);
}

// lse: as the forward pass leaves it; dlogps null: cross entropy
template <typename T>
cudaError_t backward(const Linear& L, const Common& c, const GradPlaces& g, const LinearGrad& G, const float* lse,
                     const float* dlogps, int sms, void* stream) {
    // (without rows too: dw is add)
    for (int64_t at = 0, piece = 0; piece == 0 || at < L.rows; at += g.most, ++piece) {
        MICA_STEP(gather(L, c, g.most, (int)piece, lse, dlogps, &g, &G, stream));
        LogitGrad<T> p{};
        if (!fill(&p, L, c, g.most, (int)piece)) return cudaErrorInvalidValue;
        p.coef = g.coef;
        p.origin = g.origin;
        p.d = reinterpret_cast<T*>(g.d);
        p.ld = g.ld;
        MICA_STEP((launch_gemm<T>(p, g.most / kTile * tiles_of(L.vocab), sms, stream)));
        if (G.dh) {
            Split<HiddenGrad<T>> q{};
            q.meta = c.meta;
            q.index = c.index;
            q.most = g.most;
            q.piece_index = (int)piece;
            q.vocab = L.vocab;
            q.features = L.features;
            q.dh = static_cast<T*>(G.dh);
            q.ld = G.ld_dh;
            q.wide = reinterpret_cast<uintptr_t>(G.dh) % 8 == 0 && G.ld_dh % 4 == 0;
            q.wide16 = reinterpret_cast<uintptr_t>(G.dh) % 16 == 0 && G.ld_dh % 8 == 0;
            q.parts = g.parts;
            q.w = p.w;
            if (!matrix_map(&q.d, map_type(L.dtype), g.d, L.vocab, g.most, g.ld, 1)) return cudaErrorInvalidValue;
            MICA_STEP((split_product<T>(q, g.most / kTile * tiles_of(L.features), (L.vocab + kDepth - 1) / kDepth, sms, stream)));
        }
        if (G.dw)
            MICA_STEP((G.dw_dtype == MICA_F32   ? weight_grad<T, float>(L, c, g, G, (int)piece, sms, stream)
                       : G.dw_dtype == MICA_F16 ? weight_grad<T, __half>(L, c, g, G, (int)piece, sms, stream)
                                                : weight_grad<T, __nv_bfloat16>(L, c, g, G, (int)piece, sms, stream)));
    }
    return cudaSuccess;
}

cudaError_t scan(const Linear& L, const Common& c, const float* dlogps, float* logps, float* lse, double denom,
                 double grad_scale, void* stream) {
    const Scan s{L.targets, L.wide_targets, (int)L.rows, dlogps, logps, lse, c.index, c.meta, (float)(1.0 / L.temperature),
                 (float)(-grad_scale / L.temperature), (float)denom, L.dtype == MICA_F16};
    return launch_after(scan_kernel, 1, kScanThreads, 0, stream, s);
}

}  // namespace

int64_t linear_logps_workspace(const Linear& L) {
    if (L.rows == 0) return 0;
    Places p(nullptr);
    place_common(L, forward_rows(L), &p);
    place_forward(L, &p);
    return p.bytes();
}

int launch_linear_logps(const Linear& L, float* logps, float* lse, void* workspace, int sms, void* stream) {
    Places p(workspace);
    const Common c = place_common(L, forward_rows(L), &p);
    const ForwardPlaces f = place_forward(L, &p);
    MICA_STEP(scan(L, c, nullptr, logps, lse, 0.0, 0.0, stream));
    MICA_STEP(copy_w(L, c, stream));
    return L.dtype == MICA_BF16 ? forward<__nv_bfloat16>(L, c, f, logps, lse, sms, stream)
                                : forward<__half>(L, c, f, logps, lse, sms, stream);
}

int64_t linear_grad_workspace(const Linear& L, const LinearGrad& G, int sms) {
    Places p(nullptr);
    place_common(L, grad_rows(L), &p);
    place_grad(L, G, sms, &p);
    return p.bytes();
}

int launch_linear_grad(const Linear& L, const float* lse, const float* dlogps, const LinearGrad& G, void* workspace, int sms,
                       void* stream) {
    Places p(workspace);
    const Common c = place_common(L, grad_rows(L), &p);
    const GradPlaces g = place_grad(L, G, sms, &p);
    MICA_STEP(scan(L, c, dlogps, nullptr, nullptr, 0.0, 0.0, stream));
    MICA_STEP(copy_w(L, c, stream));
    return L.dtype == MICA_BF16 ? backward<__nv_bfloat16>(L, c, g, G, lse, dlogps, sms, stream)
                                : backward<__half>(L, c, g, G, lse, dlogps, sms, stream);
}

static int ce_rows(const Linear& L) { return forward_rows(L) > grad_rows(L) ? forward_rows(L) : grad_rows(L); }

int64_t linear_ce_workspace(const Linear& L, const LinearGrad& G, int sms) {
    Places p(nullptr);
    place_common(L, ce_rows(L), &p);
    p.take<float>(L.rows);
    place_forward(L, &p);
    if (G.dh || G.dw) place_grad(L, G, sms, &p);
    return p.bytes();
}

int launch_linear_ce(const Linear& L, double denom, double grad_scale, float* loss, float* logps, const LinearGrad& G,
                     void* workspace, int sms, void* stream) {
    Places p(workspace);
    const Common c = place_common(L, ce_rows(L), &p);
    float* lse = p.take<float>(L.rows);
    const ForwardPlaces f = place_forward(L, &p);
    MICA_STEP(scan(L, c, nullptr, logps, lse, denom, grad_scale, stream));
    MICA_STEP(copy_w(L, c, stream));
    MICA_STEP(L.dtype == MICA_BF16 ? forward<__nv_bfloat16>(L, c, f, logps, lse, sms, stream)
                                   : forward<__half>(L, c, f, logps, lse, sms, stream));
    MICA_STEP(launch_after(loss_kernel, 1, 1024, 0, stream, (const float*)logps, (int)L.rows, (const Meta*)c.meta, (float)denom,
                           loss));
    if (!G.dh && !G.dw) return cudaSuccess;
    const GradPlaces g = place_grad(L, G, sms, &p);
    return L.dtype == MICA_BF16 ? backward<__nv_bfloat16>(L, c, g, G, lse, nullptr, sms, stream)
                                : backward<__half>(L, c, g, G, lse, nullptr, sms, stream);
}

int read_linear_status(unsigned int* status) { return (int)read_gemm_status(status); }

}  // namespace mica
