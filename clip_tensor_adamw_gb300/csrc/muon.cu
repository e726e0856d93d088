// Matrices orthogonalised by Newton-Schulz products, and the optimizer step that takes its update from them.
//
//   x = u / (|u| + eps);  A = x x^T (wide) or x^T x (tall);  B = a I + b A + c A^2;  x = B x (wide) or x B (tall);  and again
//
// A list goes through every product together: matrices of the same shape are a class, which lies in the workspace as one
// array with one tensor map, and a launch takes the tiles of all classes. So a step of the iteration is three launches
// whatever the list holds, and small matrices fill the GPU between them. Nothing is transposed: a tall matrix's A takes x as
// MN-major operands, and A and B are symmetric. Of A and B only the tiles on and above the diagonal are computed; the
// others are written as their mirror image, which is a thread's column and so coalesced too.
//
// x, A and B are stored in binary16: 11 bits where bfloat16 has 8, at the same rate, and the range is known, since the
// singular values stay of order 1. They are scaled by 2^10, so that elements down to 2^-24 are normal. With a x folded into
// B's diagonal the last product needs no other input. A result is off by 1.0e-3 to 1.6e-3 of its norm for gradients with
// most of their energy in a few directions (bfloat16: 0.8e-2 to 1.5e-2).
//
// Where that is not enough (kPreciseSide, and on request) x, A and B are pairs of binary16, the second what the first's
// rounding left out, and each product is three: high x high, high x low, low x high. A result is then off by some 1e-6.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "gemm.cuh"
#include "muon.h"

namespace mica {
namespace {

constexpr int kMostClasses = 8;      // of a batch
constexpr int kMostMatrices = 256;
constexpr int64_t kBatchElements = (int64_t)128 << 20;
// Elements whose momentum and first x are taken one after the other, so that the second kernel finds g and m in L2.
constexpr int64_t kGroupElements = (int64_t)8 << 20;
constexpr int kItem = 8192;          // elements that a CTA of the streaming kernels has in registers
constexpr int kMostItems = 2048;     // parts of a matrix's square sum
constexpr float kScale = 1024.0f;
// Matrices whose smaller side is at most this are held in pairs: a small matrix's elements are large beside a weight's, so the
// error would show in a float32 weight (a step of rate r changes the weights' norm by r / 0.02 sqrt(side) of it or so), and
// its products, a tile or a few for each matrix, are short.
constexpr int kPreciseSide = 256;

struct Class {
    CUtensorMap x[2], a, b;
    __half* px[2];
    __half* pa;
    __half* pb;
    int rows, cols, count, first;    // first: of its matrices, in the batch
    int low;                         // 0, or `count`: the low halves' first place in z
    int side, ld_x, ld_a;            // side: A's
    int gram_tiles, out_tiles;       // of a matrix
    int gram_before, out_before;     // tiles of the classes before
    int items, items_before;         // of a matrix; of the classes before
    int64_t item;                    // elements
    float rate;                      // lr, adjusted

    __host__ __device__ bool wide() const { return rows <= cols; }
};

struct Batch {
    Class c[kMostClasses];
    int classes, matrices, gram_pieces, out_pieces, items;
    int width;  // a tile's columns
};

// The class that tile (or item) i belongs to.
template <int Class::*before>
__device__ __forceinline__ int class_of(const Batch& b, int i) {
    int k = 0;
    while (k + 1 < b.classes && i >= b.c[k + 1].*before) ++k;
    return k;
}

// ------------------------------------------------------------------------------------------------------------------------
// momentum, norm, and the first x
// ------------------------------------------------------------------------------------------------------------------------

struct Streams {
    const void* in[kMostMatrices];  // x, or g
    float* m[kMostMatrices];
};

struct Update {
    float keep, mu;  // 1 - momentum, momentum
    int nesterov, zero_grad, skip;
    const float* factor;
};

// A matrix's part: elements [from, to) of matrix `z` of class `c`.
struct Item {
    int c, z, part;
    int64_t from, to;
};
__device__ __forceinline__ Item item_at(const Batch& b, int i) {
    const int c = class_of<&Class::items_before>(b, i), k = i - b.c[c].items_before;
    const int z = k / b.c[c].items, part = k % b.c[c].items;
    const int64_t n = (int64_t)b.c[c].rows * b.c[c].cols, from = part * b.c[c].item;
    return Item{c, z, part, from, from + b.c[c].item < n ? from + b.c[c].item : n};
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ __forceinline__ float momentum_of(float g, float m, const Update& u) { return m + u.keep * (g - m); }
__device__ __forceinline__ float update_of(float g, float m, const Update& u) { return u.nesterov ? g + u.mu * (m - g) : m; }

// m, and each item's square sum of u. A sum of squares counts from its item's largest element, so that none overflows or
// vanishes, and is widened to float64 at its end.
template <typename T, bool kMuon>
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ Batch b, const __grid_constant__ Streams s,
                                                       Update u, int from, double* squares) {
    __shared__ float part[8];
    wait_prerequisite();
    allow_dependents();
    const Item it = item_at(b, from + blockIdx.x);
    const int k = b.c[it.c].first + it.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T* in = static_cast<const T*>(s.in[k]);
    float* m = kMuon ? s.m[k] : nullptr;
    const float f = kMuon && u.factor ? *u.factor : 1.0f;
    if (kMuon && u.skip && !(f > 0.0f)) return;
    const bool wide = aligned16(in) && aligned16(m);
    double sum = 0.0;
    for (int64_t base = it.from; base < it.to; base += kItem) {
        float v[32];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = base + j * 1024 + threadIdx.x * 4;
            const int there = at >= it.to ? 0 : it.to - at < 4 ? (int)(it.to - at) : 4;
            const float4 x = load4(in + at, there, wide);
            float e[4] = {x.x, x.y, x.z, x.w};
            if (kMuon) {
                const float4 old = load4(m + at, there, wide);
                const float o[4] = {old.x, old.y, old.z, old.w};
                float n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gh = e[i] * f;
                    n[i] = momentum_of(gh, o[i], u);
                    e[i] = update_of(gh, n[i], u);
                }
                store4(m + at, make_float4(n[0], n[1], n[2], n[3]), there, wide);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[j * 4 + i] = e[i];
                top = fmaxf(top, fabsf(e[i]));
            }
        }
#pragma unroll
        for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        __syncthreads();
        if (lane == 0) part[warp] = top;
        __syncthreads();
        for (int i = 0; i < 8; ++i) top = fmaxf(top, part[i]);
        int e = (int)(__float_as_uint(top) >> 23) - 127;  // top < 2^(e + 1)
        e = e < -100 ? -100 : e > 100 ? 100 : e;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) q = fmaf(v[i] * down, v[i] * down, q);
#pragma unroll
        for (int d = 16; d; d /= 2) q += __shfl_xor_sync(~0u, q, d);
        __syncthreads();
        if (lane == 0) part[warp] = q;
        __syncthreads();
        if (threadIdx.x == 0) {
            q = 0.0f;
            for (int i = 0; i < 8; ++i) q += part[i];
            sum += ldexp((double)q, 2 * e);
        }
    }
    if (threadIdx.x == 0) squares[from + blockIdx.x] = sum;
}

// What rounding to binary16 leaves out.
__device__ __forceinline__ float rest_of(float x) { return x - __half2float(__float2half_rn(x)); }

// x = 2^10 u / (|u| + eps) in binary16, rows ld_x apart.
template <typename T, bool kMuon>
__global__ void __launch_bounds__(256) first_kernel(const __grid_constant__ Batch b, const __grid_constant__ Streams s,
                                                    Update u, int from, const double* squares, double eps) {
    __shared__ double part[8];
    __shared__ float scale;
    wait_prerequisite();
    allow_dependents();
    const Item it = item_at(b, from + blockIdx.x);
    const Class& c = b.c[it.c];
    const int k = c.first + it.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T* in = static_cast<const T*>(s.in[k]);
    const float* m = kMuon ? s.m[k] : nullptr;
    const float f = kMuon && u.factor ? *u.factor : 1.0f;
    const bool skip = kMuon && u.skip && !(f > 0.0f);
    const bool wide = aligned16(in) && aligned16(m);
    const bool even = c.cols % 4 == 0;
    if (!skip) {
        const double* mine = squares + c.items_before + it.z * c.items;
        double sum = 0.0;
        for (int i = threadIdx.x; i < c.items; i += 256) sum += mine[i];
#pragma unroll
        for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            sum = 0.0;
            for (int i = 0; i < 8; ++i) sum += part[i];
            scale = (float)((double)kScale / (sqrt(sum) + eps));
        }
        __syncthreads();
    }
    __half* x = c.px[0] + (int64_t)it.z * c.rows * c.ld_x;
    const int64_t low = (int64_t)c.low * c.rows * c.ld_x;
    // the row and column of the thread's elements, which go on by 1,024
    int64_t at = it.from + threadIdx.x * 4;
    int64_t row = at / c.cols;
    int col = (int)(at - row * c.cols);
    const int rows_on = 1024 / c.cols, cols_on = 1024 - rows_on * c.cols;
    for (; at < it.to; at += 4 * 1024) {
        float4 g[4], now[4];
        int there[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t a = at + j * 1024;
            there[j] = a >= it.to ? 0 : it.to - a < 4 ? (int)(it.to - a) : 4;
            g[j] = load4(in + a, there[j], wide);
            if (kMuon) now[j] = load4(m + a, there[j], wide);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!skip) {
                float e[4] = {g[j].x, g[j].y, g[j].z, g[j].w};
                if (kMuon) {
                    const float n[4] = {now[j].x, now[j].y, now[j].z, now[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) e[i] = update_of(e[i] * f, n[i], u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] *= scale;
                __half* to = x + row * c.ld_x;
                if (even) {
                    store4(to + col, make_float4(e[0], e[1], e[2], e[3]), there[j], true);
                    if (low)
                        store4(to + col + low, make_float4(rest_of(e[0]), rest_of(e[1]), rest_of(e[2]), rest_of(e[3])), there[j],
                               true);
                } else {
                    int k = col;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (k == c.cols) k = 0, to += c.ld_x;
                        if (i < there[j]) {
                            to[k] = __float2half_rn(e[i]);
                            if (low) to[k + low] = __float2half_rn(rest_of(e[i]));
                        }
                        ++k;
                    }
                }
            }
            if (kMuon && u.zero_grad) store4(const_cast<T*>(in) + at + j * 1024, float4{}, there[j], wide);
            row += rows_on;
            col += cols_on;
            if (col >= c.cols) col -= c.cols, ++row;
        }
    }
}

// ------------------------------------------------------------------------------------------------------------------------
// the products
// ------------------------------------------------------------------------------------------------------------------------

// Which tile of which matrix a piece is.
struct Where {
    int c, z;
};
__device__ __forceinline__ Where unpack(int tile) { return Where{tile & 7, tile >> 3}; }
static_assert(kMostClasses <= 8, "a piece's class has three bits");

// Tile (m, n) of a product over `depth` with `cols` columns.
__device__ __forceinline__ Piece piece_of(const Class& c, int width, const Operand& a, const Operand& b, int m, int n, int cols,
                                          int depth, int tile) {
    const int stages = (depth + kDepth - 1) / kDepth;
    return Piece{a, b, m * kTile, n * width, columns_of(cols - n * width, width), 0, c.low ? 3 * stages : stages, tile, -1, c.low, stages};
}

// Tiles on and above the diagonal of a symmetric matrix (of a row of tiles, those from the one on the diagonal on).
__host__ __device__ inline int triangle_tiles(int side, int width) {
    const int down = (side + kTile - 1) / kTile, across = (side + width - 1) / width;
    return down * across - kTile / width * (down * (down - 1) / 2);
}
__device__ __forceinline__ void triangle(int t, int side, int width, int* i, int* j) {
    const int across = (side + width - 1) / width, step = kTile / width;
    int row = 0;
    while (t >= across - step * row) {
        t -= across - step * row;
        ++row;
    }
    *i = row;
    *j = step * row + t;
}

// v, and `low` elements further on what its rounding leaves out, to the warp's 32 x 32 at (row0, col0) of rows x cols. (ld is
// a multiple of 8: what is stored past cols is the row's.)
__device__ __forceinline__ void store_half(__half* to, int ld, int rows, int cols, int row0, int col0, int lane,
                                           unsigned char* staging, const float (&v)[32], int64_t low) {
    uint32_t w[16];
    unsigned short* at = reinterpret_cast<unsigned short*>(to);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<__half>(v[2 * i], v[2 * i + 1]);
    store_block(at, ld, rows, (cols + 7) & ~7, row0, col0, lane, true, staging, w);
    if (!low) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<__half>(rest_of(v[2 * i]), rest_of(v[2 * i + 1]));
    store_block(at + low, ld, rows, (cols + 7) & ~7, row0, col0, lane, true, staging, w);
}

// A symmetric matrix's tile, and its mirror image.
__device__ __forceinline__ void store_symmetric(__half* to, int ld, int side, int row0, int col0, int lane,
                                                unsigned char* staging, const float (&v)[32], bool mirror, int64_t low) {
    store_half(to, ld, side, side, row0, col0, lane, staging, v, low);
    if (!mirror || row0 + lane >= side) return;
    __half* at = to + (int64_t)col0 * ld + row0 + lane;
    const int there = side - col0;
#pragma unroll
    for (int i = 0; i < 32; ++i, at += ld)
        if (i < there) *at = __float2half_rn(v[i]);
    if (!low) return;
    at = to + low + (int64_t)col0 * ld + row0 + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i, at += ld)
        if (i < there) *at = __float2half_rn(rest_of(v[i]));
}

// A = x x^T or x^T x
struct Gram {
    static constexpr unsigned int kStatus = 0x800u;
    Batch b;
    int from;  // the buffer that x is in

    struct Deal {};
    __device__ __forceinline__ Deal deal(int) const { return Deal{}; }
    __device__ __forceinline__ bool piece(const Deal&, int i, Piece* q) const {
        if (i >= b.gram_pieces) return false;
        const int k = class_of<&Class::gram_before>(b, i);
        const Class& c = b.c[k];
        const int z = (i - c.gram_before) / c.gram_tiles;
        int m, n;
        triangle((i - c.gram_before) % c.gram_tiles, c.side, b.width, &m, &n);
        const Operand x{&c.x[from], z, c.wide()};
        const int depth = c.wide() ? c.cols : c.rows;
        *q = piece_of(c, b.width, x, x, m, n, c.side, depth, z << 3 | k);
        return true;
    }
    struct Epilogue {
        const Class& c;
        __half* to;
        int row0, col0, lane;
        unsigned char* staging;
        bool mirror;
        __device__ __forceinline__ Epilogue(const Gram& p, const Deal&, const Piece& q, const Place& at)
            : c(p.b.c[unpack(q.tile).c]), lane(at.lane), staging(at.staging) {
            to = c.pa + (int64_t)unpack(q.tile).z * c.side * c.ld_a;
            row0 = q.m0 + at.row - at.lane;
            col0 = q.n0 + at.first_column;
            mirror = q.n0 >= q.m0 + kTile;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col = col0 + 32 * k;
            if (row0 >= c.side || col >= c.side) return;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kScale;
            store_symmetric(to, c.ld_a, c.side, row0, col, lane, staging, v, mirror, (int64_t)c.low * c.side * c.ld_a);
        }
        __device__ __forceinline__ void done() {}
    };
};

// B = a I + b A + c A^2
struct Poly {
    static constexpr unsigned int kStatus = 0x1000u;
    Batch b;
    float ca, cb, cc;

    struct Deal {};
    __device__ __forceinline__ Deal deal(int) const { return Deal{}; }
    __device__ __forceinline__ bool piece(const Deal&, int i, Piece* q) const {
        if (i >= b.gram_pieces) return false;
        const int k = class_of<&Class::gram_before>(b, i);
        const Class& c = b.c[k];
        const int z = (i - c.gram_before) / c.gram_tiles;
        int m, n;
        triangle((i - c.gram_before) % c.gram_tiles, c.side, b.width, &m, &n);
        const Operand a{&c.a, z, true};
        *q = piece_of(c, b.width, a, a, m, n, c.side, c.side, z << 3 | k);
        return true;
    }
    struct Epilogue {
        const Poly& p;
        const Class& c;
        const __half* a;
        __half* to;
        int row0, col0, lane;
        unsigned char* staging;
        bool mirror;
        __device__ __forceinline__ Epilogue(const Poly& p, const Deal&, const Piece& q, const Place& at)
            : p(p), c(p.b.c[unpack(q.tile).c]), lane(at.lane), staging(at.staging) {
            const int64_t first = (int64_t)unpack(q.tile).z * c.side * c.ld_a;
            a = c.pa + first;
            to = c.pb + first;
            row0 = q.m0 + at.row - at.lane;
            col0 = q.n0 + at.first_column;
            mirror = q.n0 >= q.m0 + kTile;
        }
        // v += b times 32 columns of A
        __device__ __forceinline__ void add_row(const __half* own, int row, int col, float (&v)[32]) const {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 u{};
                if (row < c.side && col + 8 * i < c.side) u = *reinterpret_cast<const uint4*>(own + 8 * i);
                const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = __half22float2(h[e]);
                    const int j = 8 * i + 2 * e;
                    v[j] = fmaf(p.cb, x.x, v[j]);
                    v[j + 1] = fmaf(p.cb, x.y, v[j + 1]);
                }
            }
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col = col0 + 32 * k, row = row0 + lane;
            if (row0 >= c.side || col >= c.side) return;
            const __half* own = a + (int64_t)row * c.ld_a + col;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= p.cc;
            add_row(own, row, col, v);
            if (c.low) add_row(own + (int64_t)c.low * c.side * c.ld_a, row, col, v);
            if ((unsigned)(row - col) < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (row == col + i) v[i] += p.ca;
            }
            store_symmetric(to, c.ld_a, c.side, row0, col, lane, staging, v, mirror, (int64_t)c.low * c.side * c.ld_a);
        }
        __device__ __forceinline__ void done() {}
    };
};

// x = B x or x B: what the middle steps and the last one share
struct Apply {
    static constexpr unsigned int kStatus = 0x2000u;
    Batch b;
    int from;

    struct Deal {};
    __device__ __forceinline__ Deal deal(int) const { return Deal{}; }
    __device__ __forceinline__ bool piece(const Deal&, int i, Piece* q) const {
        if (i >= b.out_pieces) return false;
        const int k = class_of<&Class::out_before>(b, i);
        const Class& c = b.c[k];
        const int z = (i - c.out_before) / c.out_tiles, t = (i - c.out_before) % c.out_tiles;
        const int row_tiles = (c.rows + kTile - 1) / kTile;
        const Operand x{&c.x[from], z, !c.wide()}, poly{&c.b, z, true};
        *q = piece_of(c, b.width, c.wide() ? poly : x, c.wide() ? x : poly, t % row_tiles, t / row_tiles, c.cols, c.side, z << 3 | k);
        return true;
    }
};

struct ApplyMiddle : Apply {
    struct Epilogue {
        const Class& c;
        __half* to;
        int row0, col0, lane;
        unsigned char* staging;
        __device__ __forceinline__ Epilogue(const ApplyMiddle& p, const Deal&, const Piece& q, const Place& at)
            : c(p.b.c[unpack(q.tile).c]), lane(at.lane), staging(at.staging) {
            to = c.px[p.from ^ 1] + (int64_t)unpack(q.tile).z * c.rows * c.ld_x;
            row0 = q.m0 + at.row - at.lane;
            col0 = q.n0 + at.first_column;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col0 = this->col0 + 32 * k;
            if (row0 >= c.rows || col0 >= c.cols) return;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kScale;
            store_half(to, c.ld_x, c.rows, c.cols, row0, col0, lane, staging, v, (int64_t)c.low * c.rows * c.ld_x);
        }
        __device__ __forceinline__ void done() {}
    };
};

// The last step: O to where it belongs (out of type O), or w = w * decay - rate * O (kMuon; O is float).
template <typename O, bool kMuon>
struct ApplyLast : Apply {
    O* out[kMostMatrices];
    float decay;
    int skip;
    const float* factor;

    struct Epilogue {
        const ApplyLast& p;
        const Class& c;
        O* to;
        int row0, col0, lane;
        unsigned char* staging;
        bool wide;
        __device__ __forceinline__ Epilogue(const ApplyLast& p, const Deal&, const Piece& q, const Place& at)
            : p(p), c(p.b.c[unpack(q.tile).c]), lane(at.lane), staging(at.staging) {
            to = p.out[c.first + unpack(q.tile).z];
            row0 = q.m0 + at.row - at.lane;
            col0 = q.n0 + at.first_column;
            wide = aligned16(to) && c.cols % 4 == 0;
            if (kMuon && p.skip && p.factor && !(*p.factor > 0.0f)) row0 = c.rows;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col0 = this->col0 + 32 * k;
            if (row0 >= c.rows || col0 >= c.cols) return;
            float4 x[8];
            by_columns(staging, lane, v, x);
            const int row = row0 + lane / 8, col = col0 + lane % 8 * 4, there = c.cols - col;
            if (col >= c.cols) return;
            O* at = to + (int64_t)row * c.cols + col;
            const int64_t step = 4 * (int64_t)c.cols;
            constexpr float kOne = 1.0f / (kScale * kScale);
            if constexpr (kMuon) {
                float4 w[8];
                const float rate = c.rate * kOne;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row + 4 * i < c.rows) w[i] = load4(at + i * step, there, wide);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = make_float4(w[i].x * p.decay - x[i].x * rate, w[i].y * p.decay - x[i].y * rate,
                                       w[i].z * p.decay - x[i].z * rate, w[i].w * p.decay - x[i].w * rate);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = make_float4(x[i].x * kOne, x[i].y * kOne, x[i].z * kOne, x[i].w * kOne);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row + 4 * i < c.rows) store4(at + i * step, x[i], there, wide);
        }
        __device__ __forceinline__ void done() {}
    };
};

// ------------------------------------------------------------------------------------------------------------------------
// the host side
// ------------------------------------------------------------------------------------------------------------------------

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Matrices of one shape, by their places in the list.
struct Group {
    int64_t rows, cols;
    std::vector<int32_t> which;
};

// The list cut into batches of classes. Classes with the longest sums come first, so that the last tiles are short ones.
std::vector<std::vector<Group>> batches_of(const int64_t* rows, const int64_t* cols, int32_t T) {
    std::vector<int32_t> order;
    for (int32_t k = 0; k < T; ++k)
        if (rows[k] > 0 && cols[k] > 0) order.push_back(k);
    std::stable_sort(order.begin(), order.end(), [&](int32_t i, int32_t j) {
        const int64_t a = std::max(rows[i], cols[i]), b = std::max(rows[j], cols[j]);
        return a != b ? a > b : rows[i] != rows[j] ? rows[i] > rows[j] : cols[i] > cols[j];
    });
    std::vector<std::vector<Group>> out;
    int64_t elements = 0;
    int matrices = 0;
    for (int32_t k : order) {
        const int64_t n = rows[k] * cols[k];
        bool same = !out.empty() && out.back().back().rows == rows[k] && out.back().back().cols == cols[k];
        if (out.empty() || elements + n > kBatchElements || matrices == kMostMatrices ||
            (!same && (int)out.back().size() == kMostClasses)) {
            out.emplace_back();
            elements = 0;
            matrices = 0;
            same = false;
        }
        if (!same) out.back().push_back(Group{rows[k], cols[k], {}});
        out.back().back().which.push_back(k);
        elements += n;
        ++matrices;
    }
    return out;
}

// A tile's columns: 256, or 128 where tiles of 256 would leave pairs without one. Products of 256 x 128 run at two thirds of
// the rate of 256 x 256 (four layers of GPT-2 XL: 3.93 ms with 128 columns, 3.24 with 256), but a list too small for the GPU
// is done sooner in twice as many (384 x 1536: 124 us with 128, 148 with 256).
int width_of(const std::vector<Group>& shapes, int sms) {
    int64_t gram = 0;
    for (const Group& s : shapes) gram += triangle_tiles((int)std::min(s.rows, s.cols), kTile) * (int64_t)s.which.size();
    return gram * 4 <= sms ? 128 : kTile;
}

// Fills a batch, with places in the workspace (null: sizes only); the bytes it takes.
int64_t place(const std::vector<Group>& shapes, bool precise, int sms, char* base, Batch* b, double** squares) {
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        char* p = base ? base + at : nullptr;
        at += round_up(bytes, 256);
        return p;
    };
    *b = Batch{};
    b->width = width_of(shapes, sms);
    for (const Group& s : shapes) {
        Class& c = b->c[b->classes++];
        c.rows = (int)s.rows;
        c.cols = (int)s.cols;
        c.count = (int)s.which.size();
        c.first = b->matrices;
        c.side = (int)std::min(s.rows, s.cols);
        c.low = precise || c.side <= kPreciseSide ? c.count : 0;
        c.ld_x = (int)round_up(s.cols, 8);
        c.ld_a = (int)round_up(c.side, 8);
        for (int i = 0; i < 2; ++i) c.px[i] = reinterpret_cast<__half*>(take((int64_t)(c.count + c.low) * c.rows * c.ld_x * 2));
        c.pa = reinterpret_cast<__half*>(take((int64_t)(c.count + c.low) * c.side * c.ld_a * 2));
        c.pb = reinterpret_cast<__half*>(take((int64_t)(c.count + c.low) * c.side * c.ld_a * 2));
        c.gram_tiles = triangle_tiles(c.side, b->width);
        c.out_tiles = ((c.rows + kTile - 1) / kTile) * ((c.cols + b->width - 1) / b->width);
        c.gram_before = b->gram_pieces;
        c.out_before = b->out_pieces;
        const int64_t n = s.rows * s.cols;
        c.item = round_up(std::max<int64_t>(kItem, (n + kMostItems - 1) / kMostItems), kItem);
        c.items = (int)((n + c.item - 1) / c.item);
        c.items_before = b->items;
        b->matrices += c.count;
        b->gram_pieces += c.count * c.gram_tiles;
        b->out_pieces += c.count * c.out_tiles;
        b->items += c.count * c.items;
    }
    *squares = reinterpret_cast<double*>(take((int64_t)b->items * sizeof(double)));
    return at;
}

bool maps(Batch* b) {
    constexpr auto type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    for (int k = 0; k < b->classes; ++k) {
        Class& c = b->c[k];
        for (int i = 0; i < 2; ++i)
            if (!matrix_map(&c.x[i], type, c.px[i], c.cols, c.rows, c.ld_x, c.count + c.low)) return false;
        if (!matrix_map(&c.a, type, c.pa, c.side, c.side, c.ld_a, c.count + c.low) ||
            !matrix_map(&c.b, type, c.pb, c.side, c.side, c.ld_a, c.count + c.low))
            return false;
    }
    return true;
}

#define MICA_STEP(x)                              \
    do {                                          \
        const cudaError_t step_e = (x);           \
        if (step_e != cudaSuccess) return step_e; \
    } while (0)

template <typename T, bool kMuon>
cudaError_t first(const Batch& b, const Streams& s, const Update& u, double* squares, double eps, void* stream) {
    int from = 0, to = 0;
    int64_t elements = 0;
    for (int k = 0; k < b.classes; ++k)
        for (int z = 0; z < b.c[k].count; ++z) {
            to += b.c[k].items;
            elements += (int64_t)b.c[k].rows * b.c[k].cols;
            if (elements < kGroupElements && to < b.items) continue;
            MICA_STEP(launch_after(momentum_kernel<T, kMuon>, to - from, 256, 0, stream, b, s, u, from, squares));
            MICA_STEP(launch_after(first_kernel<T, kMuon>, to - from, 256, 0, stream, b, s, u, from, (const double*)squares, eps));
            from = to;
            elements = 0;
        }
    return cudaSuccess;
}

template <typename O, bool kMuon>
cudaError_t last(const Muon& call, const Batch& b, const std::vector<Group>& shapes, int from, int sms, void* stream) {
    ApplyLast<O, kMuon> p{};
    p.b = b;
    p.from = from;
    int k = 0;
    for (const Group& s : shapes)
        for (int32_t i : s.which) p.out[k++] = static_cast<O*>(call.out[i]);
    p.decay = (float)(1.0 - call.hp.lr * call.hp.weight_decay);
    p.skip = (call.hp.flags & MICA_STEP_SKIP_NONFINITE) != 0;
    p.factor = call.d_factor;
    return launch_gemm<__half>(p, b.out_pieces, sms, stream);
}

cudaError_t run(const Muon& call, const std::vector<Group>& shapes, char* workspace, int sms, void* stream) {
    Batch b;
    double* squares;
    place(shapes, (call.ns->flags & MICA_NS_PRECISE) != 0, sms, workspace, &b, &squares);
    if (!maps(&b)) return cudaErrorInvalidValue;
    Streams s{};
    int k = 0;
    for (const Group& shape : shapes)
        for (int32_t i : shape.which) {
            s.in[k] = call.in[i];
            s.m[k++] = call.m ? call.m[i] : nullptr;
        }
    for (int i = 0; i < b.classes; ++i) {
        const double r = b.c[i].rows, c = b.c[i].cols;
        b.c[i].rate = (float)(call.hp.lr * (call.hp.adjust == MICA_MUON_ORIGINAL    ? std::sqrt(std::max(1.0, r / c))
                                            : call.hp.adjust == MICA_MUON_MATCH_RMS ? 0.2 * std::sqrt(std::max(r, c))
                                                                                    : 1.0));
    }
    const Update u{(float)(1.0 - call.hp.momentum), (float)call.hp.momentum, call.hp.nesterov, call.hp.zero_grad,
                   (call.hp.flags & MICA_STEP_SKIP_NONFINITE) != 0, call.d_factor};
    const double eps = call.ns->eps;
    if (call.m)
        MICA_STEP((call.in_dtype == MICA_F16 ? first<__half, true>(b, s, u, squares, eps, stream)
                                             : first<float, true>(b, s, u, squares, eps, stream)));
    else
        MICA_STEP((call.in_dtype == MICA_F16   ? first<__half, false>(b, s, u, squares, eps, stream)
                   : call.in_dtype == MICA_BF16 ? first<__nv_bfloat16, false>(b, s, u, squares, eps, stream)
                                                : first<float, false>(b, s, u, squares, eps, stream)));
    for (int step = 0; step < call.ns->steps; ++step) {
        const double* c = call.ns->coefficients + 3 * step;
        const int from = step & 1;
        Gram g{};
        g.b = b;
        g.from = from;
        MICA_STEP(launch_gemm<__half>(g, b.gram_pieces, sms, stream));
        Poly p{};
        p.b = b;
        p.ca = (float)(c[0] * kScale);
        p.cb = (float)c[1];
        p.cc = (float)(c[2] / kScale);
        MICA_STEP(launch_gemm<__half>(p, b.gram_pieces, sms, stream));
        if (step + 1 < call.ns->steps) {
            ApplyMiddle a{};
            a.b = b;
            a.from = from;
            MICA_STEP(launch_gemm<__half>(a, b.out_pieces, sms, stream));
        } else {
            MICA_STEP((call.m                         ? last<float, true>(call, b, shapes, from, sms, stream)
                       : call.out_dtype == MICA_F16 ? last<__half, false>(call, b, shapes, from, sms, stream)
                                                      : last<__nv_bfloat16, false>(call, b, shapes, from, sms, stream)));
        }
    }
    return cudaSuccess;
}

}  // namespace

int64_t muon_workspace(const int64_t* rows, const int64_t* cols, int32_t T, uint32_t flags) {
    int64_t most = 0;
    for (const auto& shapes : batches_of(rows, cols, T)) {
        Batch b;
        double* squares;
        most = std::max(most, place(shapes, (flags & MICA_NS_PRECISE) != 0, 1, nullptr, &b, &squares));
    }
    return most;
}

int launch_muon(const Muon& c, void* workspace, int sms, void* stream) {
    for (const auto& shapes : batches_of(c.rows, c.cols, c.count))
        MICA_STEP(run(c, shapes, static_cast<char*>(workspace), sms, stream));
    return cudaSuccess;
}

int read_muon_status(unsigned int* status) { return (int)read_gemm_status(status); }

}  // namespace mica
