// The instructions that the tensor-core kernels share: clusters, TMA boxes, tcgen05 products of a pair of CTAs, and their
// host side (tensor maps, launches as programmatic dependents).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pipe.cuh"
#include "plan.h"
#include "stream.cuh"

namespace mica {
namespace {

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

// The driver's encoder of tensor maps, or null.
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

// A matrix of 16-bit elements with its rows at 16-byte boundaries, for TMA: 8 elements to a thread.
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

bool rows_aligned(const void* dy, int64_t ld) { return reinterpret_cast<uintptr_t>(dy) % 16 == 0 && ld % 8 == 0 && ld > 0; }

}  // namespace
}  // namespace mica
