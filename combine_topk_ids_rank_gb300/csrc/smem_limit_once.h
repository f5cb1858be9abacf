// smem_limit_once.h -- raise_smem_limit for kernels that always ask for the
// same size.  Internal to libmoe_a2a.so.
#pragma once

#include "smem_limit.h"

#include <cuda.h>

#include <atomic>

namespace moe {

// Unique id of the current CUDA context (never reused, so a context made
// after a device reset has another), 0 if it cannot be told.
inline unsigned long long context_id() {
    using GetCurrent = CUresult (*)(CUcontext *);
    using GetId = CUresult (*)(CUcontext, unsigned long long *);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *a = nullptr, *b = nullptr;
        cudaDriverEntryPointQueryResult qa, qb;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &a, 12000, cudaEnableDefault,
                                             &qa) == cudaSuccess &&
            cudaGetDriverEntryPointByVersion("cuCtxGetId", &b, 12000, cudaEnableDefault, &qb) ==
                cudaSuccess &&
            qa == cudaDriverEntryPointSuccess && qb == cudaDriverEntryPointSuccess) {
            get_current = reinterpret_cast<GetCurrent>(a);
            get_id = reinterpret_cast<GetId>(b);
        }
    });
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (get_current == nullptr || get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr ||
        get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// raise_smem_limit for a kernel that always asks for the same `bytes`: once
// per context (`done` remembers the last one, one variable per kernel); the
// query of the live value costs about as much as a launch.
template <typename Kernel>
inline cudaError_t raise_smem_limit_once(Kernel *func, size_t bytes,
                                         std::atomic<unsigned long long> &done) {
    const unsigned long long id = context_id();
    if (id != 0 && done.load(std::memory_order_acquire) == id) return cudaSuccess;
    const cudaError_t err = raise_smem_limit(func, bytes);
    if (err == cudaSuccess) done.store(id, std::memory_order_release);
    return err;
}

}  // namespace moe
