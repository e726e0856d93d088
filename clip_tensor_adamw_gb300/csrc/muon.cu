// Matrices orthogonalised by Newton-Schulz products, and the optimizer step that takes its update from them.
//
//   x = u / (|u| + eps);  A = x x^T (wide) or x^T x (tall);  B = a I + b A + c A^2;  x = B x (wide) or x B (tall);  and again
//
// A list goes through every product together: matrices of the same shape are a class, which lies in the workspace as one
// array with one tensor map, and a launch takes the tiles of all classes. So a step of the iteration is three launches for up
// to 8 shapes, 256 matrices and 128 M elements (a batch; longer lists go through the whole iteration batch by batch), and
// small matrices fill the GPU between them. Nothing is transposed: a tall matrix's A takes x as MN-major operands, and A and B
// are symmetric. Of A and B only the tiles on and above the diagonal are computed; the others are written as their mirror
// image, which is a thread's column and so coalesced too.
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
constexpr int kItem = 8192;          // elements that a CTA of the streaming kernels has in registers
constexpr int kMostItems = 512;      // parts of a matrix's square sum
constexpr float kScale = 1024.0f;
// Matrices whose smaller side is at most this are held in pairs: a small matrix's elements are large beside a weight's, so the
// error would show in a float32 weight (a step of rate r changes the weights' norm by r / 0.02 sqrt(side) of it or so; 256 x
// 300 is off by 5e-8 so, 257 x 300 by 4e-6), and its products, a tile or a few for each matrix, are short. mica_orthogonalize,
// which rounds its result to 16 bits, gets binary16's own rounding and no more (2.0e-4 of the norm, where single binary16 comes
// to 1.1e-3 to 1.7e-3) and the bits that a step takes; it costs next to nothing there: six small and odd matrices take 188 us,
// and 184 with all of them single.
constexpr int kPreciseSide = 256;

struct Class {
    CUtensorMap x[2], a, b;
    __half* px[2];
    __half* pa;
    __half* pb;
    int rows, cols, count, first;    // first: of its matrices, in the batch
    int low;                         // 0, or `count`: the low halves' first place in z
    int side, ld_x, ld_a;            // side: A's
    int items, items_before;         // of a matrix; of the classes before
    int64_t item;                    // elements
    float rate;                      // lr, adjusted

    __host__ __device__ bool wide() const { return rows <= cols; }
};

struct Batch {
    Class c[kMostClasses];
    int classes, matrices, items;
};

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
    int c = 0;
    while (c + 1 < b.classes && i >= b.c[c + 1].items_before) ++c;
    const int k = i - b.c[c].items_before;
    const int z = k / b.c[c].items, part = k % b.c[c].items;
    const int64_t n = (int64_t)b.c[c].rows * b.c[c].cols, from = part * b.c[c].item;
    return Item{c, z, part, from, from + b.c[c].item < n ? from + b.c[c].item : n};
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ __forceinline__ float momentum_of(float g, float m, const Update& u) { return m + u.keep * (g - m); }
__device__ __forceinline__ float update_of(float g, float m, const Update& u) { return u.nesterov ? g + u.mu * (m - g) : m; }

// m, and each item's square sum of u. A thread's squares count from its largest element, so that none overflows or vanishes,
// and are widened to float64, of which this chip does next to nothing, once for every 16.
template <typename T, bool kMuon>
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ Batch b, const __grid_constant__ Streams s,
                                                       Update u, double* squares) {
    __shared__ double part[8];
    wait_prerequisite();
    allow_dependents();
    const Item it = item_at(b, blockIdx.x);
    const int k = b.c[it.c].first + it.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T* in = static_cast<const T*>(s.in[k]);
    float* m = kMuon ? s.m[k] : nullptr;
    const float f = kMuon && u.factor ? *u.factor : 1.0f;
    if (kMuon && u.skip && !(f > 0.0f)) return;
    const bool wide = aligned16(in) && aligned16(m);
    double sum = 0.0;
    constexpr int kLoads = 4;
    for (int64_t base = it.from + threadIdx.x * 4; base < it.to; base += kLoads * 1024) {
        float4 x[kLoads], old[kLoads];
        int there[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t at = base + j * 1024;
            there[j] = at >= it.to ? 0 : it.to - at < 4 ? (int)(it.to - at) : 4;
            x[j] = load4(in + at, there[j], wide);
            if (kMuon) old[j] = load4(m + at, there[j], wide);
        }
        float v[4 * kLoads];
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            float e[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            if (kMuon) {
                const float o[4] = {old[j].x, old[j].y, old[j].z, old[j].w};
                float n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gh = e[i] * f;
                    n[i] = momentum_of(gh, o[i], u);
                    e[i] = update_of(gh, n[i], u);
                }
                store4(m + base + j * 1024, make_float4(n[0], n[1], n[2], n[3]), there[j], wide);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[j * 4 + i] = e[i];
                top = fmaxf(top, fabsf(e[i]));
            }
        }
        int e = (int)(__float_as_uint(top) >> 23) - 127;  // top < 2^(e + 1)
        e = e < -100 ? -100 : e > 100 ? 100 : e;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * kLoads; ++i) q = fmaf(v[i] * down, v[i] * down, q);
        sum += (double)q * __hiloint2double((1023 + 2 * e) << 20, 0);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x) return;
    sum = 0.0;
    for (int i = 0; i < 8; ++i) sum += part[i];
    squares[blockIdx.x] = sum;
}

// What rounding to binary16 leaves out.
__device__ __forceinline__ float rest_of(float x) { return x - __half2float(__float2half_rn(x)); }

// x = 2^10 u / (|u| + eps) in binary16, rows ld_x apart.
template <typename T, bool kMuon>
__global__ void __launch_bounds__(256) first_kernel(const __grid_constant__ Batch b, const __grid_constant__ Streams s,
                                                    Update u, const double* squares, double eps, unsigned int* tickets,
                                                    int count) {
    __shared__ double part[8];
    __shared__ float scale;
    wait_prerequisite();
    allow_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < count; i += 256) tickets[i] = 0u;
    const Item it = item_at(b, blockIdx.x);
    const Class& c = b.c[it.c];
    const int k = c.first + it.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const T* in = static_cast<const T*>(s.in[k]);
    const float* m = kMuon ? s.m[k] : nullptr;
    const float f = kMuon && u.factor ? *u.factor : 1.0f;
    const bool skip = kMuon && u.skip && !(f > 0.0f);
    const bool wide = aligned16(in) && aligned16(m);
    const bool even = c.cols % 4 == 0;
    __half* x = c.px[0] + (int64_t)it.z * c.rows * c.ld_x;
    const int64_t low = (int64_t)c.low * c.rows * c.ld_x;
    // the row and column of the thread's elements, which go on by 1,024
    int64_t at = it.from + threadIdx.x * 4;
    int64_t row = at / c.cols;
    int col = (int)(at - row * c.cols);
    const int rows_on = 1024 / c.cols, cols_on = 1024 - rows_on * c.cols;
    float4 g[4], now[4];
    int there[4];
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t a = at + j * 1024;
            there[j] = a >= it.to ? 0 : it.to - a < 4 ? (int)(it.to - a) : 4;
            g[j] = load4(in + a, there[j], wide);
            if (kMuon) now[j] = load4(m + a, there[j], wide);
        }
    };
    load();  // (before the norm is known: its sum takes a while)
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
            const float q = (float)sum;
            scale = q > 1e-30f && q < 1e30f ? kScale / (sqrtf(q) + (float)eps) : (float)((double)kScale / (sqrt(sum) + eps));
        }
        __syncthreads();
    }
    for (; at < it.to; at += 4 * 1024, load()) {
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

// Which matrix a piece belongs to, in its `tile`.
struct Where {
    int c, z;
};
__device__ __forceinline__ Where unpack(int tile) { return Where{tile & 7, tile >> 3}; }
static_assert(kMostClasses <= 8, "a piece's class has three bits");

// The pieces of a launch come in groups that take the same time: a class's whole tiles, and its narrow ones at the matrices'
// right edge. The host deals them to the pairs, the long ones first and each to the pair that has least (so that a layer of
// GPT-2 XL's tiles of 100, 75 and 25 stages end together), and writes that down as rounds: each of a round's pairs takes one
// piece of its group, in the order of the pairs, so that neighbours share operands in L2.
constexpr int kMostPairs = 96, kMostGroups = 2 * kMostClasses, kRounds = 64;
struct Round {
    uint32_t pairs[kMostPairs / 32];
    int first;   // piece of the group
    int repeat;  // rounds like this one, one after the other
    int group;
};
struct Schedule {
    Round rows[kRounds];
    int rounds;
    int pieces;
    int width;               // a tile's columns
    int tiles[kMostGroups];  // of a matrix; group 2 k: class k's whole tiles, 2 k + 1: its narrow ones
    int slot[kMostGroups];   // tiles of the groups before,
    int first[kMostGroups];  // and their parts
    int parts[kMostClasses]; // of a tile
};
struct Turns {
    int pair, at, repeat;
};
// The pair's next piece: its group and place there; false when there are no more.
__device__ __forceinline__ bool next_piece(const Schedule& s, Turns& t, int* group, int* place) {
    for (; t.at < s.rounds; ++t.at, t.repeat = 0) {
        const Round& r = s.rows[t.at];
        if (t.repeat == r.repeat || !(r.pairs[t.pair / 32] >> t.pair % 32 & 1)) continue;
        int before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kMostPairs / 32; ++i) {
            all += __popc(r.pairs[i]);
            before += i < t.pair / 32 ? __popc(r.pairs[i]) : i == t.pair / 32 ? __popc(r.pairs[i] & ((1u << t.pair % 32) - 1)) : 0;
        }
        *group = r.group;
        *place = r.first + t.repeat++ * all + before;
        return true;
    }
    return false;
}

// Tile (m, n) of a product over `depth` with `cols` columns.
__device__ __forceinline__ Piece piece_of(const Class& c, int width, const Operand& a, const Operand& b, int m, int n, int cols,
                                          int depth, int tile) {
    const int stages = (depth + kDepth - 1) / kDepth;
    return Piece{a, b, m * kTile, n * width, columns_of(cols - n * width, width), 0, c.low ? 3 * stages : stages,
                 tile, -1, 1, 0, 0, c.low, stages};
}

// Whole columns of tiles, and whether there is a narrow one.
__host__ __device__ inline int whole_columns(int cols, int width) { return cols / width; }
__host__ __device__ inline bool has_narrow(int cols, int width) { return cols % width != 0; }
__host__ __device__ inline int row_tiles_of(int rows) { return (rows + kTile - 1) / kTile; }

// Tiles on and above the diagonal of a symmetric matrix (of a row of tiles, those from the diagonal's on).
__host__ __device__ inline int triangle_tiles(int side, int width) {
    int tiles = 0;
    for (int i = 0; i < row_tiles_of(side); ++i) {
        const int n = whole_columns(side, width) - kTile / width * i;
        tiles += n > 0 ? n : 0;
    }
    return tiles;
}
__device__ __forceinline__ void triangle(int t, int side, int width, int* i, int* j) {
    const int across = whole_columns(side, width), step = kTile / width;
    int row = 0;
    while (t >= across - step * row) {
        t -= across - step * row;
        ++row;
    }
    *i = row;
    *j = step * row + t;
}

// What the two symmetric products share: the pieces of the tiles on and above the diagonal.
struct Symmetric {
    Batch b;
    Schedule s;

    using Deal = Turns;
    __device__ __forceinline__ Deal deal(int pair, int) const { return Turns{pair, 0, 0}; }
    // the next piece's class, matrix, tile, and with its parts the tile's place among all
    __device__ __forceinline__ bool tile(Deal& d, int* k, int* z, int* m, int* n, int* part, int* slot, int* first) const {
        int group, place;
        if (!next_piece(s, d, &group, &place)) return false;
        *k = group / 2;
        *part = 0;
        if (s.parts[*k] > 1) {
            *part = place % s.parts[*k];
            place /= s.parts[*k];
        }
        *slot = s.slot[group] + place;
        *first = s.first[group] + place * s.parts[*k];
        const int tiles = s.tiles[group], side = b.c[*k].side, t = place % tiles;
        *z = place / tiles;
        if (group & 1) *m = t, *n = whole_columns(side, s.width);
        else triangle(t, side, s.width, m, n);
        return true;
    }
};

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

// The mirror image of the warp's 32 x 32: a lane's elements become a column, which the staging buffer turns to rows.
__device__ __forceinline__ void store_mirrored(__half* to, int ld, int side, int row0, int col0, int lane,
                                               unsigned char* staging, const uint32_t (&w)[16]) {
    unsigned short* t = reinterpret_cast<unsigned short*>(staging);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        t[(2 * i) * 32 + lane] = (unsigned short)w[i];
        t[(2 * i + 1) * 32 + lane] = (unsigned short)(w[i] >> 16);
    }
    __syncwarp();
    const int row = lane / 4, col = lane % 4 * 8, padded = (side + 7) & ~7;
    unsigned short* at = reinterpret_cast<unsigned short*>(to) + (int64_t)(col0 + row) * ld + row0 + col;
    if (row0 + col >= padded) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (col0 + row + 8 * i < side)
            *reinterpret_cast<uint4*>(at + (int64_t)(8 * i) * ld) = reinterpret_cast<const uint4*>(staging)[(row + 8 * i) * 4 + lane % 4];
}

// A symmetric matrix's tile, and its mirror image.
__device__ __forceinline__ void store_symmetric(__half* to, int ld, int side, int row0, int col0, int lane,
                                                unsigned char* staging, const float (&v)[32], bool mirror, int64_t low) {
    store_half(to, ld, side, side, row0, col0, lane, staging, v, low);
    if (!mirror) return;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<__half>(v[2 * i], v[2 * i + 1]);
    store_mirrored(to, ld, side, row0, col0, lane, staging, w);
    if (!low) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack2<__half>(rest_of(v[2 * i]), rest_of(v[2 * i + 1]));
    store_mirrored(to + low, ld, side, row0, col0, lane, staging, w);
}

// A = x x^T or x^T x
struct Gram : Symmetric {
    float* part_sums;
    unsigned int* tickets;
    static constexpr unsigned int kStatus = 0x800u;
    static constexpr bool kAhead = true, kJoins = true;
    int from;  // the buffer that x is in

    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        int k, z, m, n, part, slot, first;
        if (!tile(d, &k, &z, &m, &n, &part, &slot, &first)) return false;
        const Class& c = b.c[k];
        const Operand x{&c.x[from], z, c.wide()};
        *q = piece_of(c, s.width, x, x, m, n, c.side, c.wide() ? c.cols : c.rows, z << 3 | k);
        if (s.parts[k] > 1) {
            const int stages = q->to;
            q->part = part;
            q->parts = s.parts[k];
            q->slot = slot;
            q->first = first;
            q->from = stages * part / q->parts;
            q->to = stages * (part + 1) / q->parts;
        }
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
        __device__ __forceinline__ bool wants(int k) const { return row0 < c.side && col0 + 32 * k < c.side; }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col = col0 + 32 * k;
            if (!wants(k)) return;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kScale;
            store_symmetric(to, c.ld_a, c.side, row0, col, lane, staging, v, mirror, (int64_t)c.low * c.side * c.ld_a);
        }
        __device__ __forceinline__ void done() {}
    };
};

// B = a I + b A + c A^2
struct Poly : Symmetric {
    static constexpr unsigned int kStatus = 0x1000u;
    static constexpr bool kAhead = true, kJoins = false;
    float ca, cb, cc;

    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        int k, z, m, n, part, slot, first;
        if (!tile(d, &k, &z, &m, &n, &part, &slot, &first)) return false;
        const Class& c = b.c[k];
        const Operand a{&c.a, z, true};
        *q = piece_of(c, s.width, a, a, m, n, c.side, c.side, z << 3 | k);
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
        uint4 next[4];  // of A, for the next chunk
        __device__ __forceinline__ Epilogue(const Poly& p, const Deal&, const Piece& q, const Place& at)
            : p(p), c(p.b.c[unpack(q.tile).c]), lane(at.lane), staging(at.staging) {
            const int64_t first = (int64_t)unpack(q.tile).z * c.side * c.ld_a;
            a = c.pa + first;
            to = c.pb + first;
            row0 = q.m0 + at.row - at.lane;
            col0 = q.n0 + at.first_column;
            mirror = q.n0 >= q.m0 + kTile;
            load_block(0, col0, next);
        }
        // The warp's 32 x 32 of A (or of its low half, `low` elements further on), four lanes to a row
        __device__ __forceinline__ void load_block(int64_t low, int col, uint4 (&u)[4]) const {
            const __half* from = a + low + (int64_t)(row0 + lane / 4) * c.ld_a + col + lane % 4 * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = uint4{};
                if (row0 + lane / 4 + 8 * i < c.side && col + lane % 4 * 8 < c.side)
                    u[i] = __ldcg(reinterpret_cast<const uint4*>(from + (int64_t)(8 * i) * c.ld_a));
            }
        }
        // v += b times that, through the staging buffer to a row to a lane
        __device__ __forceinline__ void add_block(const uint4 (&u)[4], float (&v)[32]) const {
            uint4* s = reinterpret_cast<uint4*>(staging);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = i * 8 + lane / 4;
                s[row * 4 + (lane % 4 ^ ((row >> 1) & 3))] = u[i];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = s[lane * 4 + (i ^ ((lane >> 1) & 3))];
                const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(h[e]);
                    const int j = 8 * i + 2 * e;
                    v[j] = fmaf(p.cb, f.x, v[j]);
                    v[j + 1] = fmaf(p.cb, f.y, v[j + 1]);
                }
            }
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col = col0 + 32 * k, row = row0 + lane;
            if (row0 >= c.side || col >= c.side) return;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= p.cc;
            const uint4 now[4] = {next[0], next[1], next[2], next[3]};
            load_block(0, col + 32, next);  // (a tile's end reads a little on: the loads' latency is most of a chunk's time)
            add_block(now, v);
            if (c.low) {
                uint4 rest[4];
                load_block((int64_t)c.low * c.side * c.ld_a, col, rest);
                add_block(rest, v);
            }
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
    static constexpr bool kAhead = true, kJoins = false;
    Batch b;
    Schedule s;
    int from;

    using Deal = Turns;
    __device__ __forceinline__ Deal deal(int pair, int) const { return Turns{pair, 0, 0}; }
    __device__ __forceinline__ bool piece(Deal& d, Piece* q) const {
        int group, place;
        if (!next_piece(s, d, &group, &place)) return false;
        const int k = group / 2, tiles = s.tiles[group], z = place / tiles, t = place % tiles;
        const Class& c = b.c[k];
        const int rows = row_tiles_of(c.rows);
        const Operand x{&c.x[from], z, !c.wide()}, poly{&c.b, z, true};
        *q = piece_of(c, s.width, c.wide() ? poly : x, c.wide() ? x : poly, t % rows,
                      group & 1 ? whole_columns(c.cols, s.width) : t / rows, c.cols, c.side, z << 3 | k);
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
            wide = aligned16(to) && c.cols % (16 / (int)sizeof(O)) == 0;
            if (kMuon && p.skip && p.factor && !(*p.factor > 0.0f)) row0 = c.rows;
        }
        __device__ __forceinline__ void chunk(int k, float (&v)[32]) {
            const int col0 = this->col0 + 32 * k;
            if (row0 >= c.rows || col0 >= c.cols) return;
            constexpr float kOne = 1.0f / (kScale * kScale);
            if constexpr (!kMuon) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack2<O>(v[2 * i] * kOne, v[2 * i + 1] * kOne);
                store_block(reinterpret_cast<unsigned short*>(to), c.cols, c.rows, c.cols, row0, col0, lane, wide, staging, w);
            } else {
                float4 x[8], w[8];
                by_columns(staging, lane, v, x);
                const int row = row0 + lane / 8, col = col0 + lane % 8 * 4, there = c.cols - col;
                if (col >= c.cols) return;
                O* at = to + (int64_t)row * c.cols + col;
                const int64_t step = 4 * (int64_t)c.cols;
                const float rate = c.rate * kOne;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row + 4 * i < c.rows) w[i] = load4(at + i * step, there, wide);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = make_float4(w[i].x * p.decay - x[i].x * rate, w[i].y * p.decay - x[i].y * rate,
                                       w[i].z * p.decay - x[i].z * rate, w[i].w * p.decay - x[i].w * rate);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row + 4 * i < c.rows) store4(at + i * step, x[i], there, wide);
            }
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

// A group's pieces and how long each takes, in nanoseconds.
struct Work {
    int group, pieces, cost;
};

// Deals the groups, longest pieces first, each piece to the pair that has least so far; what the busiest pair has.
int64_t deal_out(std::vector<Work> work, int pairs, Schedule* s) {
    std::stable_sort(work.begin(), work.end(), [](const Work& a, const Work& b) { return a.cost > b.cost; });
    std::vector<int64_t> load(pairs, 0);
    std::vector<int> order(pairs);
    s->rounds = 0;
    for (size_t w = 0; w < work.size(); ++w) {
        int left = work[w].pieces, done = 0;
        while (left > 0) {
            Round& r = s->rows[s->rounds++];
            r = Round{};
            r.first = done;
            r.group = work[w].group;
            r.repeat = 1;
            // those that the next pieces go to before anyone gets two of them, least first; all, where rounds run short
            const bool plain = s->rounds + 2 * (int)(work.size() - w) >= kRounds;
            const int64_t least = *std::min_element(load.begin(), load.end());
            order.clear();
            for (int p = 0; p < pairs; ++p)
                if (plain || load[p] < least + work[w].cost) order.push_back(p);
            if ((int)order.size() > left) {
                std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return load[a] < load[b]; });
                order.resize(left);
            }
            const int each = (int)order.size();
            if (each == pairs) {
                r.repeat = left / pairs;
            } else if (each < left) {  // as often as it takes them to come near the others
                int64_t next = INT64_MAX;
                int64_t most = least;
                for (int p = 0; p < pairs; ++p)
                    if (load[p] >= least + work[w].cost) next = std::min(next, load[p]);
                    else most = std::max(most, load[p]);
                r.repeat = (int)std::max<int64_t>(1, std::min<int64_t>(left / each, (next - most) / work[w].cost));
            }
            for (int p : order) {
                r.pairs[p / 32] |= 1u << p % 32;
                load[p] += (int64_t)r.repeat * work[w].cost;
            }
            left -= r.repeat * each;
            done += r.repeat * each;
        }
    }
    return *std::max_element(load.begin(), load.end());
}

// A piece of `columns` columns: its stages, as measured (285 ns for a whole tile's; 250 to 270 for up to 128 columns, which have
// half the products and three quarters of the loads: what holds those up is not known), and a part of its epilogue, which the
// next piece's products do not hide.
int cost_of(const Class& c, int depth, int columns) {
    const int stages = (depth + kDepth - 1) / kDepth * (c.low ? 3 : 1);
    return columns > 128 ? stages * 285 + 1000 : stages * 255 + 600;
}

int most_pairs(int sms) { return std::max(1, std::min(sms / 2, kMostPairs)); }

// The parts that a tile's sum is split in, where pairs are idle. A part saves its share of the stages, a quarter of a
// microsecond each; joining costs two, and half of one for each part and 32 columns, which the last to come adds up alone. So
// 16 x 1,600 in pairs of binary16, a sum of 75 stages, is split in 6 (19 us without, 8 with), and 384 x 1,536, of 24, is not
// (12.7 us without, 14.5 in 4).
int parts_of(int stages, int columns) {
    const int chunks = (columns + 63) / 64, parts = (int)std::sqrt(stages / (2.0 * chunks));
    return parts > 1 && 0.25 * stages > 0.25 * stages / parts + 0.5 * parts * chunks + 2.0 ? parts : 1;
}
// The parts of each class's Gram sums, in tiles of 128 columns. Returns the pieces of all classes together where any is split,
// and 0 where none is.
int split_gram(const Batch& b, int pairs, int* parts) {
    int64_t tiles[kMostClasses], all = 0;
    std::fill(parts, parts + kMostClasses, 1);
    for (int k = 0; k < b.classes; ++k) {
        const Class& c = b.c[k];
        tiles[k] = (triangle_tiles(c.side, 128) + (has_narrow(c.side, 128) ? row_tiles_of(c.side) : 0)) * (int64_t)c.count;
        all += tiles[k];
    }
    if (all > pairs / 2) return 0;
    all = 0;
    bool any = false;
    for (int k = 0; k < b.classes; ++k) {
        const Class& c = b.c[k];
        parts[k] = parts_of((std::max(c.rows, c.cols) + kDepth - 1) / kDepth * (c.low ? 3 : 1), std::min(c.side, 128));
        all += parts[k] * tiles[k];
        any = any || parts[k] > 1;
    }
    if (any && all <= pairs) return (int)all;
    std::fill(parts, parts + kMostClasses, 1);
    return 0;
}
// tiles(class, narrow, width, &columns): a matrix's whole or narrow tiles; split: the product is Gram's, whose sums may be split.
// Returns how long the product takes.
template <typename Tiles, typename Depth>
int64_t schedule(const Batch& b, int sms, int width, bool split, Tiles tiles, Depth depth, Schedule* s) {
    std::vector<Work> work;
    const int pairs = most_pairs(sms);
    int n[kMostGroups], columns[kMostGroups], slots = 0;
    s->width = width;
    for (int g = 0; g < 2 * b.classes; ++g) {
        const Class& c = b.c[g / 2];
        n[g] = s->tiles[g] = tiles(c, (g & 1) != 0, width, &columns[g]);
        n[g] *= c.count;
        s->slot[g] = slots;
        s->parts[g / 2] = 1;
        slots += n[g];
    }
    if (split && width == 128) split_gram(b, pairs, s->parts);
    s->pieces = 0;
    for (int g = 0; g < 2 * b.classes; ++g) {
        const Class& c = b.c[g / 2];
        const int parts = s->parts[g / 2], count = n[g] * parts;
        s->first[g] = s->pieces;
        if (count) work.push_back(Work{g, count, cost_of(c, depth(c), columns[g]) / parts + (parts > 1 ? 1000 : 0)});
        s->pieces += count;
    }
    return deal_out(std::move(work), std::min(pairs, s->pieces), s) + (width > 128 ? 2500 : 1200);  // and the last epilogue
}

// Tiles of 256 columns, or of 128 where the product is done sooner so: their rate is two thirds (four layers of GPT-2 XL:
// 3.93 ms with 128 columns, 3.16 with 256), but a list too small for the GPU takes twice as many (384 x 1,536: 124 us with
// 128, 148 with 256).
template <typename Tiles, typename Depth>
void best_schedule(const Batch& b, int sms, bool split, Tiles tiles, Depth depth, Schedule* s) {
    Schedule narrow{};
    const int64_t wide = schedule(b, sms, kTile, split, tiles, depth, s);
    if (s->pieces < 2 * most_pairs(sms) && schedule(b, sms, 128, split, tiles, depth, &narrow) < wide) *s = narrow;
}

// The pieces of the three products.
struct Schedules {
    Schedule gram, poly, apply;
};
void schedules(const Batch& b, int sms, Schedules* s) {
    const auto triangle = [](const Class& c, bool narrow, int width, int* columns) {
        *columns = narrow ? columns_of(c.side % width, width) : width;
        return narrow ? (has_narrow(c.side, width) ? row_tiles_of(c.side) : 0) : triangle_tiles(c.side, width);
    };
    const auto all = [](const Class& c, bool narrow, int width, int* columns) {
        *columns = narrow ? columns_of(c.cols % width, width) : width;
        return row_tiles_of(c.rows) * (narrow ? has_narrow(c.cols, width) : whole_columns(c.cols, width));
    };
    best_schedule(b, sms, true, triangle, [](const Class& c) { return std::max(c.rows, c.cols); }, &s->gram);
    best_schedule(b, sms, false, triangle, [](const Class& c) { return c.side; }, &s->poly);
    best_schedule(b, sms, false, all, [](const Class& c) { return c.side; }, &s->apply);
}

// The rest of a batch's workspace.
constexpr int kTickets = kMostPairs / 2 * 2 * kTakers;  // of all tiles of a list that has split ones
struct Extra {
    double* squares;
    unsigned int* tickets;
    float* part_sums;  // where sums are split, of at most as many parts as there are pairs
};

// Fills a batch, with places in the workspace (null: sizes only); the bytes it takes.
int64_t place(const std::vector<Group>& shapes, bool precise, char* base, Batch* b, Extra* extra) {
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        char* p = base ? base + at : nullptr;
        at += round_up(bytes, 256);
        return p;
    };
    *b = Batch{};
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
        const int64_t n = s.rows * s.cols;
        c.item = round_up(std::max<int64_t>(kItem, (n + kMostItems - 1) / kMostItems), kItem);
        c.items = (int)((n + c.item - 1) / c.item);
        c.items_before = b->items;
        b->matrices += c.count;
        b->items += c.count * c.items;
    }
    extra->squares = reinterpret_cast<double*>(take((int64_t)b->items * sizeof(double)));
    extra->tickets = reinterpret_cast<unsigned int*>(take(kTickets * sizeof(unsigned int)));
    int parts[kMostClasses];
    const int64_t pieces = split_gram(*b, kMostPairs, parts);  // (no fewer than where there are fewer pairs)
    extra->part_sums = reinterpret_cast<float*>(take(pieces * kPartFloats * sizeof(float)));
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
cudaError_t first(const Batch& b, const Streams& s, const Update& u, const Extra& extra, double eps, void* stream) {
    MICA_STEP(launch_after(momentum_kernel<T, kMuon>, b.items, 256, 0, stream, b, s, u, extra.squares));
    return launch_after(first_kernel<T, kMuon>, b.items, 256, 0, stream, b, s, u, (const double*)extra.squares, eps,
                        extra.tickets, kTickets);
}

template <typename O, bool kMuon>
cudaError_t last(const Muon& call, const Batch& b, const Schedules& s, const std::vector<Group>& shapes, int from, int sms,
                 void* stream) {
    ApplyLast<O, kMuon> p{};
    p.b = b;
    p.s = s.apply;
    p.from = from;
    int k = 0;
    for (const Group& shape : shapes)
        for (int32_t i : shape.which) p.out[k++] = static_cast<O*>(call.out[i]);
    p.decay = (float)(1.0 - call.hp.lr * call.hp.weight_decay);
    p.skip = (call.hp.flags & MICA_STEP_SKIP_NONFINITE) != 0;
    p.factor = call.d_factor;
    return launch_gemm<__half>(p, s.apply.pieces, 2 * most_pairs(sms), stream);
}

cudaError_t run(const Muon& call, const std::vector<Group>& shapes, char* workspace, int sms, void* stream) {
    Batch b;
    Extra extra;
    place(shapes, (call.ns->flags & MICA_NS_PRECISE) != 0, workspace, &b, &extra);
    if (!maps(&b)) return cudaErrorInvalidValue;
    Schedules deals{};
    schedules(b, sms, &deals);
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
        MICA_STEP((call.in_dtype == MICA_F16 ? first<__half, true>(b, s, u, extra, eps, stream)
                                             : first<float, true>(b, s, u, extra, eps, stream)));
    else
        MICA_STEP((call.in_dtype == MICA_F16   ? first<__half, false>(b, s, u, extra, eps, stream)
                   : call.in_dtype == MICA_BF16 ? first<__nv_bfloat16, false>(b, s, u, extra, eps, stream)
                                                : first<float, false>(b, s, u, extra, eps, stream)));
    for (int step = 0; step < call.ns->steps; ++step) {
        const double* c = call.ns->coefficients + 3 * step;
        const int from = step & 1;
        Gram g{};
        g.b = b;
        g.s = deals.gram;
        g.part_sums = extra.part_sums;
        g.tickets = extra.tickets;
        g.from = from;
        MICA_STEP(launch_gemm<__half>(g, deals.gram.pieces, 2 * most_pairs(sms), stream));
        Poly p{};
        p.b = b;
        p.s = deals.poly;
        p.ca = (float)(c[0] * kScale);
        p.cb = (float)c[1];
        p.cc = (float)(c[2] / kScale);
        MICA_STEP(launch_gemm<__half>(p, deals.poly.pieces, 2 * most_pairs(sms), stream));
        if (step + 1 < call.ns->steps) {
            ApplyMiddle a{};
            a.b = b;
            a.s = deals.apply;
            a.from = from;
            MICA_STEP(launch_gemm<__half>(a, deals.apply.pieces, 2 * most_pairs(sms), stream));
        } else {
            MICA_STEP((call.m                         ? last<float, true>(call, b, deals, shapes, from, sms, stream)
                       : call.out_dtype == MICA_F16 ? last<__half, false>(call, b, deals, shapes, from, sms, stream)
                                                      : last<__nv_bfloat16, false>(call, b, deals, shapes, from, sms, stream)));
        }
    }
    return cudaSuccess;
}

}  // namespace

int64_t muon_workspace(const int64_t* rows, const int64_t* cols, int32_t T, uint32_t flags) {
    int64_t most = 0;
    for (const auto& shapes : batches_of(rows, cols, T)) {
        Batch b;
        Extra extra;
        most = std::max(most, place(shapes, (flags & MICA_NS_PRECISE) != 0, nullptr, &b, &extra));
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
