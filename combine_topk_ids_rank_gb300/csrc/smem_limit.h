// smem_limit.h -- a kernel's dynamic shared-memory limit, raised and never
// lowered.  Internal to libmoe_a2a.so.
//
// cudaFuncAttributeMaxDynamicSharedMemorySize is one value per kernel and
// context for the whole process, while each handle prepares the kernels for
// its own row size.  Setting it to a handle's own size would take it below
// what an earlier handle of a larger size launches with, and that handle's
// next launch would be refused.  So the limit only ever grows: the live
// value is read (correct also after the context was reset) and raised when
// it is below the size asked for, under one lock so that concurrent handles
// cannot lower each other's raise.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace moe {

inline cudaError_t raise_smem_limit(const void *func, size_t bytes) {
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    cudaFuncAttributes fa;
    cudaError_t err = cudaFuncGetAttributes(&fa, func);
    if (err != cudaSuccess) return err;
    if ((size_t)fa.maxDynamicSharedSizeBytes >= bytes) return cudaSuccess;
    return cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename Kernel>
inline cudaError_t raise_smem_limit(Kernel *func, size_t bytes) {
    return raise_smem_limit(reinterpret_cast<const void *>(func), bytes);
}

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
