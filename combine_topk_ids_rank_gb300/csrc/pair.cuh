// pair.cuh -- inline PTX of the persistent products (layer_small.cu,
// gemm_int8.cu, expert_product.cuh) beside ptx.cuh: the electing branch, clusters, parked waits.
#pragma once

#include "ptx.cuh"

namespace moe {
namespace ptx {

// True in one lane of a fully active warp.  Inside the branch the compiler
// knows that one thread runs, and tcgen05 and TMA instructions are issued
// straight from uniform registers: 9 to 40 cycles a small tensor-core product
// against 56 to 207 under a plain `lane == 0` (measured, M = 128, N = 16).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// cp_async16 with zeros instead of the source's bytes (nothing is read).
__device__ __forceinline__ void cp_async16_zero(void *smem_dst, const void *gmem_src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, 0;" ::"r"(smem_u32(smem_dst)),
                 "l"(gmem_src)
                 : "memory");
}

// ---- clusters ---------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Barrier of all threads of the cluster (memory ordered at cluster scope), in
// two halves and as one.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// Address in CTA `rank` of the cluster of this CTA's shared memory at `p`.
__device__ __forceinline__ uint32_t cluster_smem(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

// One arrival on a barrier of any CTA of the cluster, released at CTA scope:
// for what only the arriving CTA's own SM goes on to touch -- the tensor core
// of each SM of a pair reads and writes that SM's shared and tensor memory,
// whichever CTA issued the product.  (A release at cluster scope took about
// 1300 cycles an arrival and 15 % of the 8-bit product's time.)
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(
                     cluster_addr)
                 : "memory");
}

// ---- waits of kernels with many waiting warps ---------------------------------

// mbar_wait_timed whose probes suspend the warp in hardware for up to kParkNs
// (it wakes when the phase completes) instead of coming back at once: probes
// go through the queue that the working warps' loads, stores and shuffles use.  Gives up
// early where *failed is set.
constexpr uint32_t kParkNs = 20000;
__device__ __forceinline__ bool mbar_park(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                          const volatile int *failed = nullptr) {
    auto probe = [&] {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kParkNs)
            : "memory");
        return done != 0;
    };
    if (probe()) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 4; ++i)
            if (probe()) return true;
        if (globaltimer_ns() - t0 > limit_ns || (failed != nullptr && *failed)) return false;
    }
}

}  // namespace ptx
}  // namespace moe
