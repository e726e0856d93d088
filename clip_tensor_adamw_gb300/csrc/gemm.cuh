// A matrix product on the tensor cores whose operands, tiles and epilogue a policy gives: what the losses from hidden states
// (linear.cu) and the orthogonalisation (muon.cu) are made of.
//
// A pair of CTAs takes a tile of 256 x 256 sums, 64 steps of the summed dimension at a time: each CTA holds 128 rows of the
// tile and loads half of both operands, and tcgen05.mma of the pair multiplies both halves with one another. The grid is one
// pair for two SMs; pairs take pieces of work in turn. One warp loads stages by TMA, one issues products, and eight empty the
// accumulators, of which TMEM holds two, so that a tile's epilogue runs under the next tile's products.
//
// An operand is K-major (the summed dimension contiguous) or MN-major; either way a stage is boxes of 64 x 64 elements with
// 128-byte swizzle, so that one tensor map serves a matrix in both roles and nothing is transposed: only the step from one
// product of 16 to the next differs, 32 bytes or 2 KB. Elements outside the matrix are read as zeros.
//
// A policy P is the kernel's parameter, with
//   Deal deal(int pair, int pairs) const            how the work is dealt to one of the pairs; computed once a thread
//   bool piece(Deal&, Piece*) const                 the pair's next piece of work; false when there are no more
//   kAhead                                          the work is known from the parameter alone, and the first piece is looked
//                                                   up while the kernel before still runs (1 to 2 us, most of it misses);
//                                                   otherwise void prefetch() const does what it can
//   kJoins                                          tiles may be split, and the kernel joins their sums itself: each warp
//                                                   leaves its part's in `part_sums` (kPartFloats for each part), and the one
//                                                   that comes last, by `tickets` (16 for each tile, zeros before and after),
//                                                   adds them up in their order; the epilogue's bool wants(int c) says which
//                                                   chunks are worth it
//   struct Epilogue                                 what becomes of a piece's sums, made for each piece by each of its threads:
//     Epilogue(const P&, const Deal&, const Piece&, const Place&)
//     void chunk(int c, float (&v)[32])             columns [32 c, 32 c + 32) of the thread's row of its half, in order
//     void done()
#pragma once

#include <atomic>

#include "elem.cuh"
#include "mma.cuh"
#include "stream.cuh"

namespace mica {
namespace {

constexpr int kHalf = 128, kTile = 2 * kHalf;  // rows and columns: of a CTA, of a pair
constexpr int kDepth = 64;                     // the summed dimension of a stage
constexpr int kStages = 6;
constexpr int kTakers = 8;                     // warps that empty the accumulators
constexpr int kGemmThreads = (kTakers + 2) * 32;
enum GemmRole { kLoader = kTakers, kMultiplier };
constexpr int kOperandBytes = kHalf * kDepth * 2, kBoxBytes = 64 * kDepth * 2;
constexpr int kStagingBytes = 32 * 32 * 4;     // of a warp
constexpr int kGemmShared = 1024 + kStages * 2 * kOperandBytes + kTakers * kStagingBytes;

// Set (OR-ed) by a kernel whose bounded wait gave up; read and cleared by the host (read_gemm_status).
__device__ unsigned int g_gemm_status;
std::atomic<bool> g_gemm_launched{false};  // in this process; until then nothing can have set it

// An operand: its map, the coordinate of its third dimension, and whether its rows run along the summed dimension.
struct Operand {
    const CUtensorMap* map;
    int z;
    bool k_major;
};

// Stages [from, to) of the tile whose first row and column are m0 and n0.
struct Piece {
    Operand a, b;
    int m0, n0;
    int columns;  // of the tile, a multiple of 64 up to 256: the products take as long as there are
    int from, to;
    int tile;   // for the epilogue, as the policy likes
    int part;   // >= 0: part of a split tile
    int parts;  // kJoins: how many it has (then `part` counts from 0), from `first` on among all parts
    int first;
    int slot;   // the tile's place among all
    int low;    // > 0: both operands are sums of two matrices, the second (the rounding's rest) `low` further on in z: the
    int depth;  // products of stages [0, depth) of high and high, high and low, low and high follow one another
};

// Where a taker stands: its row of the tile, its half's first column, the warp's staging buffer.
struct Place {
    int row, first_column, lane;
    unsigned char* staging;
};

struct GemmBarriers {
    uint64_t full[kStages];          // (leader) a stage's operands have come, in both CTAs
    uint64_t used[kStages];          // the products of a stage are done
    uint64_t sum_full[2], sum_empty[2];  // a tile's sums are in TMEM; (leader) both CTAs have taken them
    uint32_t tmem;
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void load_box3_for_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 at;\n\t"
        "mapa.shared::cluster.u32 at, %5, 0;\n\t"
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [at];\n\t}" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// A CTA's half of a stage's operand: 64 or 128 rows (or columns) from `at` on, by 64 of the summed dimension from k on.
__device__ __forceinline__ void load_operand(unsigned char* dst, const Operand& o, int at, int k, int z, bool both, uint64_t* bar) {
    load_box3_for_pair(dst, o.map, o.k_major ? k : at, o.k_major ? at : k, z, bar);
    if (both) load_box3_for_pair(dst + kBoxBytes, o.map, o.k_major ? k : at + 64, o.k_major ? at + 64 : k, z, bar);
}

// A tile's columns where `left` are left of the matrix.
__host__ __device__ inline int columns_of(int left, int most) { return left < most ? (left + 63) & ~63 : most; }

// The descriptor of either kind of operand: 128-byte swizzle, groups of 8 lines of 128 bytes 1 KB apart; boxes of 64 columns
// kBoxBytes apart, which counts for MN-major operands only.
__device__ __forceinline__ uint64_t operand_descriptor(uint32_t at) {
    return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)(kBoxBytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// float32 sums of bfloat16 (or binary16) products, 256 x columns
template <typename T>
__device__ __forceinline__ uint32_t instruction(bool a_k_major, bool b_k_major, int columns) {
    constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | (a_k_major ? 0u : 1u << 15) | (b_k_major ? 0u : 1u << 16) |
           (uint32_t)(columns / 8) << 17 |
           (kTile / 16) << 24;
}

// 32 columns of the thread's row of TMEM
__device__ __forceinline__ void load_sums32(uint32_t at, float (&f)[32]) {
    uint32_t v[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
          "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
}

constexpr int64_t kPartFloats = (int64_t)kTile * kTile;  // of a part's sums

// Where a warp leaves its share of a part's sums.
template <typename P>
__device__ __forceinline__ float* part_of(const P& p, const Piece& q, int part, int rank, int warp) {
    return p.part_sums + (int64_t)(q.first + part) * kPartFloats + (rank * kTakers + warp) * (kPartFloats / (2 * kTakers));
}
// Whether the warp is the last of `parts` to get here; it leaves the ticket at 0.
__device__ __forceinline__ bool comes_last(unsigned int* ticket, int parts, int lane) {
    __threadfence();
    __syncwarp();
    unsigned int before = 0;
    if (lane == 0) {
        before = atomicAdd(ticket, 1u);
        if (before == (unsigned)parts - 1) *ticket = 0u;
    }
    before = __shfl_sync(~0u, before, 0);
    __threadfence();
    return before == (unsigned)parts - 1;
}

template <typename T, typename P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ P p) {
    extern __shared__ unsigned char raw[];
    __shared__ GemmBarriers bar;
    unsigned char* a_stage = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    unsigned char* b_stage = a_stage + kStages * kOperandBytes;
    unsigned char* staging = b_stage + kStages * kOperandBytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)rank_of_cta(), pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sum_full[i], 1);
            mbar_init(&bar.sum_empty[i], 2 * kTakers);
        }
        mbar_fence_init();
    }
    if (warp == kMultiplier) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bar.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bar.tmem);
    typename P::Deal deal;
    Piece q;
    bool ok = true, more = false;
    if constexpr (P::kAhead) {
        deal = p.deal(pair, pairs);
        more = p.piece(deal, &q);
        if (warp == kLoader && lane == 0 && more) {
            prefetch_map(q.a.map);
            prefetch_map(q.b.map);
        }
    }
    if constexpr (!P::kAhead) {
        if (warp == kLoader && lane == 0) p.prefetch();
    }
    wait_prerequisite();
    allow_dependents();
    if constexpr (!P::kAhead) {
        deal = p.deal(pair, pairs);
        more = p.piece(deal, &q);
    }

    if (warp == kLoader) {
        if (lane == 0) {
            Turn<kStages> turn;
            for (; ok && more; more = p.piece(deal, &q))
                for (int k = q.from; k < q.to; ++k, turn.next()) {
                    const int s = turn.at;
                    if (!(ok = mbar_wait_idle(&bar.used[s], turn.round ^ 1))) break;
                    const bool both = q.columns > 128;
                    if (rank == 0) mbar_arrive_expect_tx(&bar.full[s], 2 * (kOperandBytes + (both ? 2 : 1) * kBoxBytes));
                    int az = q.a.z, bz = q.b.z, at = k;
                    if (q.low && k >= q.depth) {
                        if (k < 2 * q.depth) bz += q.low, at -= q.depth;
                        else az += q.low, at -= 2 * q.depth;
                    }
                    load_operand(a_stage + s * kOperandBytes, q.a, q.m0 + rank * kHalf, at * kDepth, az, true, &bar.full[s]);
                    load_operand(b_stage + s * kOperandBytes, q.b, q.n0 + rank * (q.columns / 2), at * kDepth, bz, both,
                                 &bar.full[s]);
                }
            // Every copy has landed when the last products are done. Where a wait gave up they are given 2 ms.
            for (int i = 0; !ok && i < 200; ++i) __nanosleep(10000);
        }
    } else if (warp == kMultiplier) {  // issued by one thread of the leader, in code that the whole warp runs alike
        if (rank == 0) {
            const bool one = elect_one();
            const uint64_t a0 = operand_descriptor(smem_u32(a_stage)), b0 = operand_descriptor(smem_u32(b_stage));
            Turn<kStages> turn;
            Turn<2> sums;
            for (; ok && more; more = p.piece(deal, &q)) {
                const int b = sums.at;
                const uint32_t how = instruction<T>(q.a.k_major, q.b.k_major, q.columns);
                const uint32_t a_step = (q.a.k_major ? 32 : 2048) >> 4, b_step = (q.b.k_major ? 32 : 2048) >> 4;
                if (!(ok = mbar_wait_idle(&bar.sum_empty[b], sums.round ^ 1))) break;
                fence_after();
                for (int k = q.from; k < q.to; ++k, turn.next()) {
                    const int s = turn.at;
                    if (!(ok = mbar_wait_idle(&bar.full[s], turn.round))) break;
                    fence_after();
                    if (one) {
                        const uint64_t a = a0 + (uint32_t)s * (kOperandBytes >> 4), b1 = b0 + (uint32_t)s * (kOperandBytes >> 4);
#pragma unroll
                        for (int d = 0; d < kDepth / 16; ++d)
                            multiply(tmem + b * kTile, a + d * a_step, b1 + d * b_step, how, k > q.from || d > 0);
                        commit(&bar.used[s]);
                        if (k == q.to - 1) commit(&bar.sum_full[b]);
                    }
                }
                sums.next();
            }
        }
    } else {
        const int quarter = warp % 4, half = warp / 4;
        Place place{rank * kHalf + quarter * 32 + lane, 0, lane, staging + warp * kStagingBytes};
        Turn<2> sums;
        for (; more; more = p.piece(deal, &q)) {
            const int b = sums.at, chunks = q.columns / 64;
            place.first_column = half * (q.columns / 2);
            const uint32_t own = tmem + ((uint32_t)quarter << 21) + b * kTile + place.first_column;
            typename P::Epilogue epilogue(p, deal, q, place);
            if (!(ok = mbar_wait_idle(&bar.sum_full[b], sums.round))) break;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                float v[32];
                __syncwarp();  // (TMEM is read by the whole warp at once, whose lanes an epilogue's edges part)
                load_sums32(own + c * 32, v);
                if (c == chunks - 1) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader(&bar.sum_empty[b]);
                }
                if constexpr (P::kJoins) {
                    if (q.parts > 1) {
                        if (!epilogue.wants(c)) continue;
                        float* out = part_of(p, q, q.part, rank, warp) + c * 1024 + lane;
#pragma unroll
                        for (int e = 0; e < 32; ++e) out[e * 32] = v[e];
                        continue;
                    }
                }
                epilogue.chunk(c, v);
            }
            if constexpr (P::kJoins) {
                if (q.parts > 1) {
                    if (epilogue.wants(0) && comes_last(p.tickets + (q.slot * 2 + rank) * kTakers + warp, q.parts, lane))
#pragma unroll 1
                        for (int c = 0; c < chunks && epilogue.wants(c); ++c) {
                            float v[32] = {};
                            for (int part = 0; part < q.parts; ++part) {
                                const float* in = part_of(p, q, part, rank, warp) + c * 1024 + lane;
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] += __ldcg(in + e * 32);
                            }
                            epilogue.chunk(c, v);
                        }
                    sums.next();
                    continue;
                }
            }
            epilogue.done();
            sums.next();
        }
    }
    if (!ok) atomicOr(&g_gemm_status, p.kStatus);
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's products have read this CTA's shared memory, its arrivals have landed
    fence_after();
    if (warp == kMultiplier) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------------------------------------------------------------
// splitting a long sum
// ------------------------------------------------------------------------------------------------------------------------

// `whole` tiles one after another, then the rest (fewer than there are pairs) in `parts` along the summed dimension.
struct SplitDeal {
    int tiles, stages, whole, parts, pieces;
    int next, pairs;  // the pair's next piece; and then every pairs-th
};

// The number of parts is the one that makes the rest shortest by this count, in stages: rounds of parts, each with a part's
// stages and kPartCost for filling and emptying it; and what joining takes, kJoinCost and a quarter of a stage for each part
// (512 KB written and read). 48 tiles of 786 stages on 76 pairs: 1 part 221 us, 3 parts (2 rounds) 150 us.
constexpr int kPartCost = 6, kJoinCost = 12, kLeastStages = 4, kMostRounds = 2;
__host__ __device__ inline SplitDeal split_deal(int tiles, int stages, int pair, int pairs) {
    SplitDeal d{tiles, stages, tiles / pairs * pairs, 1, tiles, pair, pairs};
    const int rest = tiles - d.whole;
    if (rest == 0) return d;
    int best = stages + kPartCost;
    for (int rounds = 1; rounds <= kMostRounds; ++rounds) {
        int parts = rounds * pairs / rest;
        if (parts > stages / kLeastStages) parts = stages / kLeastStages;
        if (parts < 2) continue;
        const int cost = rounds * ((stages + parts - 1) / parts + kPartCost) + kJoinCost + rest * parts / 4;
        if (cost < best) {
            best = cost;
            d.parts = parts;
        }
    }
    d.pieces = d.whole + rest * d.parts;
    return d;
}

// The next piece's tile, stages and part; false when there are no more.
__device__ __forceinline__ bool split_piece(SplitDeal& d, Piece* q) {
    const int i = d.next;
    if (i >= d.pieces) return false;
    d.next += d.pairs;
    if (i < d.whole || d.parts == 1) {
        *q = Piece{{}, {}, 0, 0, kTile, 0, d.stages, i, -1, 1, 0, 0, 0, 0};
        return true;
    }
    const int k = i - d.whole, part = k % d.parts;
    *q = Piece{{}, {}, 0, 0, kTile, (int)((int64_t)d.stages * part / d.parts), (int)((int64_t)d.stages * (part + 1) / d.parts),
               d.whole + k / d.parts, k, 1, 0, 0, 0, 0};
    return true;
}

// ------------------------------------------------------------------------------------------------------------------------
// from a row to a thread, to coalesced accesses
// ------------------------------------------------------------------------------------------------------------------------

// 32 rows x 32 float32 of a warp, a row to a lane, turned to four columns of a row at a time, eight lanes to a row: x[i] is
// row 4 i + lane / 8, columns 4 (lane % 8) on. Through shared memory, whose 16-byte units change places so that no two lanes of
// a phase meet.
__device__ __forceinline__ void by_columns(unsigned char* staging, int lane, const float (&v)[32], float4 (&x)[8]) {
    float4* s = reinterpret_cast<float4*>(staging);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) s[lane * 8 + (j ^ (lane & 7))] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    const int j = lane % 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + lane / 8;
        x[i] = s[row * 8 + (j ^ (row & 7))];
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    else
        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// 32 rows x 32 elements of 16 bits of a warp, a row to a lane, turned to eight columns of a row at a time, four lanes to a row:
// x[i] is row 8 i + lane / 4, columns 8 (lane % 4) on.
__device__ __forceinline__ void by_columns16(unsigned char* staging, int lane, const uint32_t (&v)[16], uint4 (&x)[4]) {
    uint4* s = reinterpret_cast<uint4*>(staging);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        s[lane * 4 + (j ^ ((lane >> 1) & 3))] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    const int j = lane % 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + lane / 4;
        x[i] = s[row * 4 + (j ^ ((row >> 1) & 3))];
    }
}

// Eight elements of 16 bits to a row, of which `there` are in the matrix; wide: rows are aligned for one store.
__device__ __forceinline__ void store8(unsigned short* at, uint4 x, int there, bool wide) {
    if (wide && there >= 8) {
        *reinterpret_cast<uint4*>(at) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < there) at[i] = (unsigned short)(w[i / 2] >> (i % 2 * 16));
}

// The warp's 32 x 32 elements of 16 bits at (row0, col0) of a matrix whose first `rows` x `cols` are written.
__device__ __forceinline__ void store_block(unsigned short* to, int64_t ld, int rows, int cols, int row0, int col0, int lane,
                                            bool wide, unsigned char* staging, const uint32_t (&v)[16]) {
    uint4 x[4];
    by_columns16(staging, lane, v, x);
    const int row = row0 + lane / 4, col = col0 + lane % 4 * 8;
    unsigned short* at = to + row * ld + col;
    if (wide && row0 + 32 <= rows && col0 + 32 <= cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(at + i * 8 * ld) = x[i];
        return;
    }
    if (!wide) {  // a column to a lane, so that a row's stores are contiguous
        const unsigned short* s = reinterpret_cast<const unsigned short*>(staging);
        if (col0 + lane >= cols) return;
        at = to + row0 * ld + col0 + lane;
#pragma unroll 1
        for (int r0 = 0; r0 < 32 && row0 + r0 < rows; r0 += 16) {
            unsigned short e[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) e[r] = s[(r0 + r) * 32 + ((lane / 8 ^ ((r >> 1) & 3)) * 8) + lane % 8];
#pragma unroll
            for (int r = 0; r < 16; ++r, at += ld)
                if (row0 + r0 + r < rows) *at = e[r];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (row + i * 8 < rows && col < cols) store8(at + i * 8 * ld, x[i], cols - col, true);
}

// Four values to a row of O, the first at `at`, of which `there` are in the matrix; wide: rows are aligned for one store.
template <typename O>
__device__ __forceinline__ void store4(O* at, float4 v, int there, bool wide) {
    if (wide && there >= 4) {
        if constexpr (sizeof(O) == 4)
            *reinterpret_cast<float4*>(at) = v;
        else
            *reinterpret_cast<uint2*>(at) = make_uint2(pack2<O>(v.x, v.y), pack2<O>(v.z, v.w));
        return;
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < there) at[i] = narrow<O>(f[i]);
}
template <typename O>
__device__ __forceinline__ float4 load4(const O* at, int there, bool wide) {
    if (wide && there >= 4) {
        if constexpr (sizeof(O) == 4) {
            return *reinterpret_cast<const float4*>(at);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(at);
            const O* e = reinterpret_cast<const O*>(&u);
            return make_float4(widen(e[0]), widen(e[1]), widen(e[2]), widen(e[3]));
        }
    }
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < there ? widen(at[i]) : 0.0f;
    return make_float4(f[0], f[1], f[2], f[3]);
}

// ------------------------------------------------------------------------------------------------------------------------
// the host side
// ------------------------------------------------------------------------------------------------------------------------

// A map of `count` matrices of rows x cols elements of 16 bits, one after another; false where the driver refuses it.
bool matrix_map(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t cols, int64_t rows, int64_t ld,
                int64_t count) {
    const Encode fn = encode_fn();
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(count > 1 ? ld * rows : ld) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)kDepth, 1}, one[3] = {1, 1, 1};
    return fn && fn(map, type, 3, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pieces: how many there can be at most
template <typename T, typename P>
cudaError_t launch_gemm(const P& p, int64_t pieces, int sms, void* stream) {
    const auto kernel = gemm_kernel<T, P>;
    g_gemm_launched = true;
    // once for each device (a kernel's attributes are the device's, and the call takes as long as a third of a launch)
    static std::atomic<uint64_t> set{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
    if (!(set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmShared);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
    return launch_after(kernel, 2 * (pieces < pairs ? pieces : pairs), kGemmThreads, kGemmShared, stream, p);
}

cudaError_t read_gemm_status(unsigned int* status) {
    *status = 0;
    if (!g_gemm_launched) return cudaSuccess;
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gemm_status, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_gemm_status, &zero, sizeof zero);
    }
    *status = v;
    return e;
}

}  // namespace
}  // namespace mica
