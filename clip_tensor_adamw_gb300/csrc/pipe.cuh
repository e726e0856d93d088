// TMA bulk copies and mbarriers whose waits are bounded, for the kernels that pipeline through shared memory.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mica {
namespace {

constexpr uint32_t kMaxPolls = 1u << 22;  // try_wait rounds before a wait gives up (each round may suspend a while)

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Waits until the barrier's phase of parity `parity` has completed; false if it has not after kMaxPolls rounds.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, uint32_t max_polls = kMaxPolls) {
    const uint32_t addr = smem_u32(bar);
    for (uint32_t i = 0; i < max_polls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}
// The same for warps that wait often and long: each round suspends for up to a millisecond, so that the waiting warps take
// few of the SM's issue slots; up to some 4 s.
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
    for (uint32_t i = 0; i < 4096; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity), "r"(1000000)
            : "memory");
        if (done) return true;
    }
    return false;
}
// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned, completing on `bar`.
__device__ __forceinline__ void bulk_copy_g2s(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(smem_dst)),
                 "l"(gmem_src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// The same with an L2 cache policy (an evict-last policy from l2_keep_policy keeps the lines for a later reader).
__device__ __forceinline__ void bulk_copy_g2s_hint(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar,
                                                   uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
            "r"(smem_u32(smem_dst)),
        "l"(gmem_src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// A place in a ring of kCount stages: the stage and how often the ring has been around, mod 2. A stage's `full` barrier is
// waited on with parity `round`, its `empty` barrier with `round ^ 1` (which is through at once the first time around).
template <int kCount>
struct Turn {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next() {
        if (++at == kCount) {
            at = 0;
            round ^= 1;
        }
    }
};

// Waits for the last copies queued, up to a ring's.
template <int kCount>
__device__ __forceinline__ void drain(uint64_t* full, const Turn<kCount>& turn, int queued) {
    for (int q = 0; q < kCount; ++q) {  // stages before `at` were filled in this round, the others in the last
        if (q < turn.at) mbar_wait(&full[q], turn.round);
        else if (queued == kCount) mbar_wait(&full[q], turn.round ^ 1);
    }
}

}  // namespace
}  // namespace mica
