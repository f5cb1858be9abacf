// tensor_map.h -- tensor maps of the tiled TMA loads, encoded on the host.
// Internal to libmoe_a2a.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

namespace moe {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    });
    return fn;
}

// Matrix of `rows` x `cols` bf16 values or bytes (row-major, cols contiguous),
// boxes of box_rows x 128 bytes with the 128-byte swizzle; rows and columns
// past the end read as zero.
inline bool make_map(CUtensorMap *m, const void *base, long long rows, int cols, int box_rows,
                     bool bytes) {
    EncodeTiled enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const int esize = bytes ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * esize};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / esize), (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for `n` > 2 extents (innermost first) with the strides of all but
// the first in elements.
inline bool make_map_nd(CUtensorMap *m, const void *base, int n, const long long *extent,
                        const long long *stride, const int *box_extent, bool bytes) {
    EncodeTiled enc = tensor_map_encoder();
    if (enc == nullptr || n > 5) return false;
    const int esize = bytes ? 1 : 2;
    cuuint64_t dims[5], strides[4];
    cuuint32_t box[5], estr[5];
    for (int i = 0; i < n; ++i) {
        dims[i] = (cuuint64_t)extent[i];
        box[i] = (cuuint32_t)box_extent[i];
        estr[i] = 1;
        if (i > 0) strides[i - 1] = (cuuint64_t)stride[i] * esize;
    }
    return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n,
               const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
