// entry.h -- what the C entry points of the operators share (moe_ops.cpp,
// moe_products.cpp): checks and statuses.  Internal to libmoe_a2a.so.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "moe_a2a.h"

namespace moe {

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A CUDA call failed: clear the runtime's last error, so that the caller's
// next CUDA call does not report it again.
inline int cuda_failed() {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
}

inline bool sm_count(int *sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// A launcher's result as a status; nothing is thrown through the C entries.
template <typename Launch>
int launched(Launch &&launch) {
    try {
        return launch() == cudaSuccess ? MOE_OK : cuda_failed();
    } catch (...) {
        return cuda_failed();
    }
}

}  // namespace moe
