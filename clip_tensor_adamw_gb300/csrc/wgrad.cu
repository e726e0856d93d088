// A linear layer's weight gradient from its input's 8-bit checkpoint: dw = add + x^T dy, on the tensor cores.
//
// A pair of CTAs takes a tile of 256 outputs (dy's columns, the rows of the accumulator) x 256 features (the checkpoint's
// columns), 64 tokens at a time. Each CTA holds 128 of the outputs and decodes 128 of the features; tcgen05.mma of the pair
// multiplies both halves with one another, so that dy and the codes come from L2 once for two SMs (one CTA alone would
// take 80 bytes a clock, more than an SM gets).
//
// A code times its block's power of two is exact in bfloat16 (7 bits), and by the format in binary16 too, so decoding adds
// no rounding and the products are exact. The tensor cores' additions are truncated: their sums leave TMEM every 512 tokens
// (kChunkStages stages) and are added in registers. A float32 gradient's error, of its norm, at 16,384 tokens: 1.8e-7 with
// bfloat16 and 4.3e-7 with binary16 operands (8.6e-7 with 1,024 tokens a visit, 1.1e-5 with none; 7.6e-7 for a product in
// float32). 1,024 tokens a visit would take 3% less.
//
// Both operands are MN-major: a stage is [64 tokens][64 columns] boxes with 128-byte swizzle, as dy lies in memory and as
// the codes do, so nothing is transposed. dy comes by TMA; the codes come by TMA into a stage of their own, from which
// sixteen warps, four groups of four that take stages in turn, decode them into the operand. The same warps empty TMEM, a
// chunk behind. Three more warps load codes, load dy, and issue the products.
//
// What bounds it: 16,384 x 1,600 x 6,400 bfloat16 takes 299 to 308 us, 1,110 TFLOP/s, the tensor pipe 54% active; without the
// decoding it would take some 240 us. A stage moves 96 KB through an SM's shared memory (the products read 48, dy and codes
// are written with 24, codes read with 8, operands written with 16), 750 clocks' worth against the products' 512. Beside
// that, tiles of 256 cover 1,792 features where there are 1,600 (12% more products), and nineteen warps leave a thread 96
// registers, of which its sums take 64: 92 to 120 bytes are spilled. Two groups of eight decoding warps took 11% longer.
//
// Whole tiles are dealt to the pairs in turn; what remains for the last round is split along the tokens so that every pair
// has a share, whose sums a second kernel joins in a fixed order.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "packed.cuh"
#include "pipe.cuh"
#include "plan.h"
#include "stream.cuh"
#include "train.h"

namespace mica {
namespace {

constexpr int kHalf = 128, kTile = 2 * kHalf;  // outputs, and features: of a CTA, of a pair
constexpr int kDepth = 64;                     // tokens of a stage
constexpr int kDepths = 5;                     // stages
constexpr int kChunkStages = 8;                // stages between two visits to the accumulator
constexpr int kWorkers = 512, kWorkerWarps = kWorkers / 32, kThreads2 = kWorkers + 96;
constexpr int kGroups = 4, kGroupWarps = kWorkerWarps / kGroups;  // of workers: they decode stages in turn
static_assert(kGroups <= kDepths, "a group would miss two phases of a stage's barriers");
constexpr int kColumns = kTile * kHalf / kWorkers;  // of the accumulator, that a worker sums up
enum Role { kCodes = kWorkerWarps, kDy, kProducts };              // the other warps
constexpr int kOperandBytes = kDepth * kHalf * 2, kCodeBytes = kDepth * kHalf, kBoxBytes = kDepth * 128;
constexpr int kSharedBytes = 1024 + kDepths * (2 * kOperandBytes + kCodeBytes);

// Set (OR-ed) by a kernel whose bounded wait gave up; read and cleared by the host (read_wgrad_status).
__device__ unsigned int g_wgrad_status;
std::atomic<bool> g_wgrad_launched{false};  // in this process; until then nothing can have set it
enum : unsigned int { kStatusWgrad = 0x80u };

// How the work is dealt: `whole` tiles one after another, then `split` tiles in `parts` along the tokens.
struct Deal {
    int pairs, feature_tiles, tiles, whole, parts, stages;
};

// A pair's i-th piece of work: a tile's stages [from, to); piece >= 0: part of a split tile, whose sums go to the workspace.
struct Piece {
    int tile, from, to, piece;
};

__host__ __device__ inline int pieces_of(const Deal& d) { return d.whole + (d.tiles - d.whole) * d.parts; }

__device__ __forceinline__ Piece piece_at(const Deal& d, int i) {
    if (i < d.whole) return Piece{i, 0, d.stages, -1};
    const int k = i - d.whole, part = k % d.parts;
    return Piece{d.whole + k / d.parts, (int)((int64_t)d.stages * part / d.parts),
                 (int)((int64_t)d.stages * (part + 1) / d.parts), d.parts > 1 ? k : -1};
}

struct Barriers {
    uint64_t codes_full[kDepths], codes_empty[kDepths];  // the codes of a stage have come; the workers have read them
    uint64_t ready[kDepths];                             // (leader) dy has come and the codes are decoded, in both CTAs
    uint64_t used[kDepths];                              // the products of a stage are done
    uint64_t sum_full[2], sum_empty[2];                  // a chunk's sums are in TMEM; (leader) both CTAs have taken them
    uint32_t tmem;
    alignas(16) uint32_t steps[kDepths][kDepth];  // a token's four blocks of 32 features
};

__device__ __forceinline__ uint32_t rank_of_cta() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on the leader's barrier.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 at;\n\t"
        "mapa.shared::cluster.u32 at, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [at];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
// One lane of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Four bytes, or zeros, to shared memory without waiting for them; a thread's arrival on `bar` once all of its have landed.
__device__ __forceinline__ void copy4(uint32_t* dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// The same, completing on the leader's barrier.
__device__ __forceinline__ void load_box_for_pair(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 at;\n\t"
        "mapa.shared::cluster.u32 at, %4, 0;\n\t"
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[at];\n\t}" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// The descriptor of an MN-major operand with 128-byte swizzle: boxes of 64 columns kBoxBytes apart, groups of 8 tokens 1 KB.
__device__ __forceinline__ uint64_t operand(uint32_t at) {
    return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)(kBoxBytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// float32 sums of bfloat16 (or binary16) products, both operands MN-major, 256 x 256
template <typename T>
__host__ __device__ constexpr uint32_t instruction() {
    constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | 1u << 15 | 1u << 16 | (kTile / 8) << 17 | (kTile / 16) << 24;
}
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t how, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(how), "r"((uint32_t)add)
        : "memory");
}
// The barrier (in both CTAs) completes when every product so far is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of the thread's row of TMEM
__device__ __forceinline__ void load_sums(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A block's step in both halves of a register, from a token's four stored exponents (byte `b` of them). 255 gives an
// infinity, whose product with the block's codes, all 0, is a NaN.
template <typename T>
__device__ __forceinline__ uint32_t step_pair(uint32_t four, int b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        return __byte_perm(four, 0, 0x4040u | b | b << 8) << 7;
    } else {
        const __half2 s = __float2half2_rn(__uint_as_float(__byte_perm(four, 0, 0x4440u | b) << 23));
        return *reinterpret_cast<const uint32_t*>(&s);
    }
}

// The codes in bytes 0 and 2 of w as 16-bit floats times the step:
//   bfloat16: 128 + (q & 127) and 128 + (q & 128) have the bits 0x4300 | those, and their difference is q
//   binary16: 1024 + (q + 128) has the bits 0x6400 | (q ^ 128)
template <typename T>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t step) {
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const uint32_t a = (w & 0x007F007Fu) | 0x43004300u, c = (w & 0x00800080u) | 0x43004300u;
        asm("{\n\t.reg .b32 d;\n\tsub.rn.bf16x2 d, %1, %2;\n\tmul.rn.bf16x2 %0, d, %3;\n\t}"
            : "=r"(r)
            : "r"(a), "r"(c), "r"(step));
    } else {
        const uint32_t a = (w & 0x00FF00FFu) ^ 0x64806480u;
        asm("{\n\t.reg .b32 d;\n\tsub.rn.f16x2 d, %1, %2;\n\tmul.rn.f16x2 %0, d, %3;\n\t}"
            : "=r"(r)
            : "r"(a), "r"(0x64806480u), "r"(step));  // 1152
    }
    return r;
}

// Sixteen codes of a token, all of one block, to the two 16-byte pieces of its row that the swizzle puts them in. Of each
// four features the middle ones change places, which write_dw undoes: so a pair takes a mask and not a permutation.
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename T>
__device__ __forceinline__ void decode(uint32_t at, uint4 codes, uint32_t step) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = decode_pair<T>(w[i], step);
        o[2 * i + 1] = decode_pair<T>(w[i] >> 8, step);
    }
    store_shared(at, o[0], o[1], o[2], o[3]);
    store_shared(at ^ 16, o[4], o[5], o[6], o[7]);
}
// The feature of an operand's column.
__host__ __device__ constexpr int feature_of(int column) {
    return column % 4 == 1 ? column + 1 : column % 4 == 2 ? column - 1 : column;
}

// dw[i + c][j] = add + the sum of feature c, eight features' loads at a time
template <typename O, int kCount>
__device__ __forceinline__ void write_dw(const Wgrad& w, int64_t i, int64_t j, const float (&sum)[kCount]) {
    if (j >= w.n) return;
    const int there = (int)(w.x.cols - i < kCount ? w.x.cols - i : kCount);
    const O* add = static_cast<const O*>(w.add) + i * w.ld_add + j;
    O* dw = static_cast<O*>(w.dw) + i * w.ld_dw + j;
#pragma unroll
    for (int c0 = 0; c0 < kCount; c0 += 8) {
        float a[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) a[c] = w.add && c0 + c < there ? widen(add[(c0 + c) * w.ld_add]) : 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c0 + c < there) dw[(c0 + c) * w.ld_dw] = narrow<O>(sum[feature_of(c0 + c)] + a[c]);
    }
}

template <typename T, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads2, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap codes_map, const __grid_constant__ CUtensorMap dy_map, Wgrad w, Deal deal,
                 float* partial) {
    extern __shared__ unsigned char raw[];
    __shared__ Barriers bar;
    unsigned char* base = raw + (1024 - smem_u32(raw) % 1024) % 1024;
    unsigned char* dy_stage = base;
    unsigned char* x_stage = base + kDepths * kOperandBytes;
    unsigned char* code_stage = base + 2 * kDepths * kOperandBytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)rank_of_cta(), pair = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDepths; ++i) {
            mbar_init(&bar.codes_full[i], 1 + 32);
            mbar_init(&bar.codes_empty[i], kGroupWarps);
            mbar_init(&bar.ready[i], 2 * kGroupWarps + 1);
            mbar_init(&bar.used[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sum_full[i], 1);
            mbar_init(&bar.sum_empty[i], 2 * kWorkerWarps);
        }
        mbar_fence_init();
    }
    if (warp == kProducts) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bar.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bar.tmem);
    wait_prerequisite();
    allow_dependents();

    const int all = pieces_of(deal);
    bool ok = true;
    if (warp == kCodes) {  // loads codes and steps
        const uint8_t* steps = reinterpret_cast<const uint8_t*>(w.x.steps);
        Turn<kDepths> turn;
        int queued = 0;
        for (int i = pair; i < all && ok; i += deal.pairs) {
            const Piece p = piece_at(deal, i);
            const int i0 = p.tile % deal.feature_tiles * kTile + rank * kHalf;
            for (int k = p.from; k < p.to; ++k, turn.next()) {
                const int s = turn.at;
                if (!(ok = mbar_wait_idle(&bar.codes_empty[s], turn.round ^ 1))) break;
                if (queued < kDepths) ++queued;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.codes_full[s], kCodeBytes);
                    load_box(code_stage + s * kCodeBytes, &codes_map, i0, k * kDepth, &bar.codes_full[s]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int64_t t = (int64_t)k * kDepth + lane + u * 32;
                    const bool there = t < w.x.rows && i0 < w.x.cols;
                    copy4(&bar.steps[s][lane + u * 32], there ? steps + t * w.x.ld_s + i0 / kBlock : steps, there);
                }
                arrive_copied(&bar.codes_full[s]);
                __syncwarp();
            }
        }
        // no copy is left in flight when the CTA ends
        drain(bar.codes_full, turn, queued);
    } else if (warp == kDy) {  // loads dy
        if (lane == 0) {
            Turn<kDepths> turn;
            for (int i = pair; i < all && ok; i += deal.pairs) {
                const Piece p = piece_at(deal, i);
                const int j0 = p.tile / deal.feature_tiles * kTile + rank * kHalf;
                for (int k = p.from; k < p.to; ++k, turn.next()) {
                    const int s = turn.at;
                    if (!(ok = mbar_wait_idle(&bar.used[s], turn.round ^ 1))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&bar.ready[s], 2 * kOperandBytes);
                    load_box_for_pair(dy_stage + s * kOperandBytes, &dy_map, j0, k * kDepth, &bar.ready[s]);
                    load_box_for_pair(dy_stage + s * kOperandBytes + kBoxBytes, &dy_map, j0 + 64, k * kDepth, &bar.ready[s]);
                }
            }
            // Every copy has landed when the last products are done. Where a wait gave up they are given 2 ms.
            for (int i = 0; !ok && i < 200; ++i) __nanosleep(10000);
        }
    } else if (warp == kProducts) {  // issued by one thread of the leader, in code that the whole warp runs alike
        if (rank == 0) {
            const bool one = elect_one();
            const uint64_t dy0 = operand(smem_u32(dy_stage)), x0 = operand(smem_u32(x_stage));
            Turn<kDepths> turn;
            Turn<2> sums;
            for (int i = pair; i < all && ok; i += deal.pairs) {
                const Piece p = piece_at(deal, i);
                int within = 0;  // the chunk
                for (int k = p.from; k < p.to; ++k, turn.next()) {
                    const int s = turn.at, b = sums.at;
                    if (within == 0 && !(ok = mbar_wait_idle(&bar.sum_empty[b], sums.round ^ 1))) break;
                    if (!(ok = mbar_wait_idle(&bar.ready[s], turn.round))) break;
                    fence_after();
                    const uint32_t at = (uint32_t)s * (kOperandBytes >> 4);
                    const bool last = ++within == kChunkStages || k == p.to - 1;
                    if (one) {
#pragma unroll
                        for (int d = 0; d < kDepth / 16; ++d)  // 16 tokens are 2 KB further on
                            multiply(tmem + b * kTile, dy0 + (at + d * (2048 >> 4)), x0 + (at + d * (2048 >> 4)), instruction<T>(),
                                     within > 1 || d > 0);
                        commit(&bar.used[s]);
                        if (last) commit(&bar.sum_full[b]);
                    }
                    if (last) {
                        sums.next();
                        within = 0;
                    }
                }
            }
        }
    } else {  // the workers
        // A thread decodes 2 x 16 codes of two tokens, in the order of the halves that puts a store's 8 lanes (two tokens) on
        // different banks; and sums up one row and kColumns columns of the accumulator.
        const int quarter = warp % 4, first_column = warp / 4 * kColumns, group = warp / kGroupWarps;
        const uint32_t own = tmem + ((uint32_t)quarter << 21) + first_column;
        const int in_group = threadIdx.x % (kWorkers / kGroups), token = in_group / 4, part = in_group % 4, odd = token % 2;
        const uint32_t from = smem_u32(code_stage) + token * kHalf + part * 16;
        const uint32_t to = smem_u32(x_stage) + token * 128 + ((part * 2) ^ (token % 8)) * 16;
        Turn<kDepths> turn;
        Turn<2> sums;
        int whose = 0;  // group's turn it is
        for (int i = pair; i < all && ok; i += deal.pairs) {
            const Piece p = piece_at(deal, i);
            const int j0 = p.tile / deal.feature_tiles * kTile + rank * kHalf, i_tile = p.tile % deal.feature_tiles * kTile;
            float sum[kColumns];
#pragma unroll
            for (int c = 0; c < kColumns; ++c) sum[c] = 0.0f;
            auto take = [&]() {  // the oldest such chunk's sums
                const int b = sums.at;
                if (!mbar_wait_idle(&bar.sum_full[b], sums.round)) return false;
                sums.next();
                fence_after();
#pragma unroll
                for (int c = 0; c < kColumns; c += 16) {
                    uint32_t v[16];
                    load_sums(own + b * kTile + c, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[c + e] += __uint_as_float(v[e]);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(&bar.sum_empty[b]);
                return true;
            };
            int waiting = 0;  // chunks whose operands are in place and whose sums have not been taken
            int within = 0;        // the chunk
            for (int k = p.from; k < p.to; ++k, turn.next(), whose = (whose + 1) % kGroups) {
                if (whose == group) {
                    const int s = turn.at;
                    constexpr int kApart = kWorkers / kGroups / 4, kTokens = kDepth / kApart;  // of a thread
                    // The order matters: a group takes every kGroups-th stage of a ring of kDepths, so it has not seen
                    // whether the stage's last codes (another group's) have come, and a wait by parity passes on the phase
                    // before the last too. When the products of those codes are done, the codes had come, and the second
                    // wait can only mean this stage's. The first is safe by itself: products end in order, and the group's
                    // own last stage waited for later ones than this barrier's phase before.
                    if (!(ok = mbar_wait_idle(&bar.used[s], turn.round ^ 1))) break;
                    if (!(ok = mbar_wait_idle(&bar.codes_full[s], turn.round))) break;
#pragma unroll
                    for (int u = 0; u < kTokens; ++u) {
                        const uint32_t steps = bar.steps[s][token + u * kApart];
                        uint4 codes[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            codes[h] = load_shared(from + s * kCodeBytes + u * kApart * kHalf + (h ^ odd) * 64);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            decode<T>(to + s * kOperandBytes + u * kApart * 128 + (h ^ odd) * kBoxBytes, codes[h],
                                      step_pair<T>(steps, (h ^ odd) * 2 + part / 2));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.codes_empty[s]);
                        arrive_leader(&bar.ready[s]);
                    }
                }
                // the groups empty TMEM at different times, so that the others go on decoding
                if (++within == kChunkStages) {
                    if (waiting && !(ok = take())) break;
                    waiting = 1;
                    within = 0;
                }
            }
            if (within) ++waiting;
            while (ok && waiting-- > 0) ok = take();
            if (!ok) break;
            // lanes hold neighbouring outputs, so a feature's stores are contiguous
            const int j = j0 + quarter * 32 + lane;
            if (p.piece < 0) {
                write_dw<O>(w, i_tile + first_column, j, sum);
            } else {
                float* out = partial + ((int64_t)p.piece * 2 + rank) * kHalf * kTile + threadIdx.x;
#pragma unroll
                for (int c = 0; c < kColumns; ++c) out[c * kWorkers] = sum[c];
            }
        }
    }
    if (!ok) atomicOr(&g_wgrad_status, kStatusWgrad);
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's products have read this CTA's shared memory, its arrivals have landed
    fence_after();
    if (warp == kProducts)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the parts of split tiles (none where there are no tokens): a CTA takes 8 of a worker's columns.
template <typename O>
__global__ void __launch_bounds__(kWorkers) wgrad_join_kernel(Wgrad w, Deal deal, const float* partial) {
    wait_prerequisite();
    allow_dependents();
    constexpr int kSome = 8, kCtas = kColumns / kSome;
    const int c0 = blockIdx.x % kCtas * kSome, rank = blockIdx.x / kCtas % 2, k = blockIdx.x / (2 * kCtas);
    const int tile = deal.whole + k, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float sum[kSome] = {};
    for (int part = 0; part < deal.parts; ++part) {
        const float* in = partial + (((int64_t)k * deal.parts + part) * 2 + rank) * kHalf * kTile + threadIdx.x;
#pragma unroll
        for (int c = 0; c < kSome; ++c) sum[c] += __ldcg(in + (c0 + c) * kWorkers);
    }
    write_dw<O>(w, (int64_t)(tile % deal.feature_tiles) * kTile + warp / 4 * kColumns + c0,
                (int64_t)(tile / deal.feature_tiles) * kTile + rank * kHalf + warp % 4 * 32 + lane, sum);
}

// dy with its rows at 16-byte boundaries, for TMA: 8 elements to a thread.
__global__ void __launch_bounds__(256) align_rows_kernel(const unsigned short* dy, int64_t ld, int64_t rows, int64_t n,
                                                         unsigned short* out, int64_t ld_out) {
    wait_prerequisite();
    allow_dependents();
    const int64_t per = ld_out / 8;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < rows * per; q += (int64_t)gridDim.x * 256) {
        const int64_t row = q / per, col = q % per * 8;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = col + 2 * i;
            const uint32_t lo = c < n ? dy[row * ld + c] : 0u, hi = c + 1 < n ? dy[row * ld + c + 1] : 0u;
            v[i] = lo | hi << 16;
        }
        *reinterpret_cast<uint4*>(out + row * ld_out + col) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

Deal deal_of(int64_t tokens, int64_t features, int64_t n, int sms) {
    Deal d{};
    d.pairs = sms / 2 < 1 ? 1 : sms / 2;
    d.feature_tiles = (int)((features + kTile - 1) / kTile);
    d.tiles = (int)((n + kTile - 1) / kTile) * d.feature_tiles;
    d.stages = (int)((tokens + kDepth - 1) / kDepth);
    d.whole = d.tiles / d.pairs * d.pairs;
    const int rest = d.tiles - d.whole;
    d.parts = 1;
    if (rest) {
        d.parts = d.pairs / rest;
        // a chunk at least: 509 tokens of 27 tiles take 16 us whole and 23 us with the second kernel that two parts cost
        if (d.parts > d.stages / kChunkStages) d.parts = d.stages / kChunkStages;
        if (d.parts < 1) d.parts = 1;
    }
    if (d.stages == 0) d.whole = 0, d.parts = 0;  // nothing to add up: the join alone writes every tile
    return d;
}

bool rows_aligned(const void* dy, int64_t ld) { return reinterpret_cast<uintptr_t>(dy) % 16 == 0 && ld % 8 == 0 && ld > 0; }

int64_t partial_bytes(const Deal& d) {
    return d.parts > 1 ? (int64_t)(d.tiles - d.whole) * d.parts * kTile * kTile * sizeof(float) : 0;
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encode_fn() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (Encode) nullptr;
        }
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t cols, int64_t rows, int64_t stride_bytes,
            uint32_t box_cols, CUtensorMapSwizzle swizzle) {
    const Encode fn = encode_fn();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride_bytes};
    const cuuint32_t box[2] = {box_cols, (cuuint32_t)kDepth}, one[2] = {1, 1};
    return fn && fn(map, type, 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename... A>
cudaError_t launch_after(K kernel, int64_t ctas, int threads, size_t shared, void* stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, typename O>
cudaError_t launch_typed(const Wgrad& w, const Deal& d, float* partial, void* stream) {
    if (d.stages) {
        CUtensorMap codes, dy;
        const auto type = std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const int64_t padded = (w.x.cols + kBlock - 1) / kBlock * kBlock;
        if (!encode(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.x.codes, padded, w.x.rows, w.x.ld, kHalf,
                    CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode(&dy, type, w.dy, w.n, w.x.rows, w.ld_dy * 2, 64, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        const auto kernel = wgrad_kernel<T, O>;
        g_wgrad_launched = true;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
        const int all = pieces_of(d), pairs = all < d.pairs ? all : d.pairs;
        if (e == cudaSuccess)
            e = launch_after(kernel, 2 * (int64_t)pairs, kThreads2, kSharedBytes, stream, codes, dy, w, d, partial);
        if (e != cudaSuccess) return e;
    }
    if (d.parts == 1) return cudaSuccess;
    return launch_after(wgrad_join_kernel<O>, (int64_t)(d.tiles - d.whole) * 2 * (kColumns / 8), kWorkers, 0, stream, w, d,
                        (const float*)partial);
}

template <typename T>
cudaError_t launch_into(const Wgrad& w, const Deal& d, float* partial, void* stream) {
    return w.dw_dtype == MICA_F32   ? launch_typed<T, float>(w, d, partial, stream)
           : w.dw_dtype == MICA_F16 ? launch_typed<T, __half>(w, d, partial, stream)
                                    : launch_typed<T, __nv_bfloat16>(w, d, partial, stream);
}

}  // namespace

int64_t wgrad_workspace(int64_t tokens, int64_t features, int64_t n, const void* dy, int64_t ld_dy, int sms) {
    if (features == 0 || n == 0) return 0;
    return partial_bytes(deal_of(tokens, features, n, sms)) + (rows_aligned(dy, ld_dy) ? 0 : tokens * ((n + 7) / 8 * 8) * 2);
}

int launch_wgrad(const Wgrad& in, void* workspace, int sms, void* stream) {
    Wgrad w = in;
    const Deal d = deal_of(w.x.rows, w.x.cols, w.n, sms);
    float* partial = static_cast<float*>(workspace);
    if (d.stages && !rows_aligned(w.dy, w.ld_dy)) {
        unsigned short* copy = reinterpret_cast<unsigned short*>(static_cast<char*>(workspace) + partial_bytes(d));
        const int64_t ld = (w.n + 7) / 8 * 8, threads = w.x.rows * (ld / 8), ctas = (threads + 255) / 256;
        const cudaError_t e = launch_after(align_rows_kernel, ctas < (1 << 16) ? ctas : (1 << 16), 256, 0, stream,
                                           static_cast<const unsigned short*>(w.dy), w.ld_dy, w.x.rows, w.n, copy, ld);
        if (e != cudaSuccess) return (int)e;
        w.dy = copy;
        w.ld_dy = ld;
    }
    return (int)(w.dy_dtype == MICA_F16 ? launch_into<__half>(w, d, partial, stream)
                                        : launch_into<__nv_bfloat16>(w, d, partial, stream));
}

int read_wgrad_status(unsigned int* status) {
    *status = 0;
    if (!g_wgrad_launched) return (int)cudaSuccess;
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_wgrad_status, sizeof v);
    if (e != cudaSuccess) return (int)e;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wgrad_status, &zero, sizeof zero);
    }
    *status = v;
    return (int)e;
}

}  // namespace mica
