// moe_products.cpp -- C entry points of the experts' products and of the block
// quantiser (include/moe_a2a.h): argument checks on the host, then one launch.
#include "entry.h"
#include "product.h"

#include "moe_a2a.h"

namespace {

using namespace moe;

// Extents that every product takes: 32-bit coordinates, and twice the number of tiles.
// `wide`: columns of all groups together.
bool extents_ok(int64_t groups, int64_t rows, int64_t lanes, int64_t wide, int64_t depth) {
    if (rows > kProductMaxExtent || lanes > kProductMaxExtent || wide > kProductMaxExtent ||
        depth > kProductMaxDepth || groups * lanes > kProductMaxExtent ||
        groups * depth > kProductMaxExtent)
        return false;
    // (the smallest tiles of a call with many; a group may end with one that is not full)
    return (lanes + 127) / 128 * (wide / 128 + groups) <= INT32_MAX / 2;
}

ProductParams params(const int32_t *counts, const int32_t *offsets, void *out, void *scratch,
                     int groups, int rows, int lanes, int cols, int depth, int nmax) {
    ProductParams p = {};
    p.counts = counts;
    p.offsets = offsets;
    p.out = out;
    p.header = static_cast<StreamHeader *>(scratch);
    p.part = reinterpret_cast<float *>(static_cast<char *>(scratch) + kStreamHeaderBytes);
    p.G = groups;
    p.M = rows;
    p.lanes = lanes;
    p.cols = cols;
    p.depth = depth;
    p.nmax = nmax;
    return p;
}

// The checks of pointers that the ragged products share.
int check_ragged(const void *a, const void *b, const int32_t *offsets, const void *out,
                 uintptr_t out_align, const void *scratch, size_t scratch_bytes) {
    if (a == nullptr || b == nullptr || offsets == nullptr || out == nullptr ||
        scratch == nullptr || !aligned(a, 16) || !aligned(b, 16) || !aligned(offsets, 4) ||
        !aligned(out, out_align) || !aligned(scratch, 256))
        return MOE_ERR_INVALID_ARG;
    if (scratch_bytes < moe_gemm_ragged_scratch_bytes()) return MOE_ERR_CAPACITY;
    return MOE_OK;
}

bool ragged_shape_ok(int groups, int rows, int N, int hidden, bool grads) {
    return groups >= 0 && groups <= kProductMaxGroups && rows >= 0 && N >= 1 && hidden >= 8 &&
           hidden % 8 == 0 && (!grads || N % 8 == 0);
}

}  // namespace

extern "C" {

int moe_quantize_blocks_fp8(const void *d_x, int32_t bf16, int32_t groups, int32_t rows,
                            int32_t hidden, int64_t row_stride, int32_t block_rows,
                            const int32_t *d_counts, void *d_q, float *d_scale, void *stream) {
    const int vec = bf16 ? 8 : 4;  // elements of a 16-byte load
    if (groups < 0 || rows < 0 || hidden < 16 || hidden % 16 != 0 ||
        hidden > kProductMaxExtent || rows > kProductMaxExtent || row_stride < hidden ||
        row_stride % vec != 0 ||
        (block_rows != 1 && block_rows != kScaleBlock) ||
        (d_counts != nullptr && block_rows != 1))
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    if (d_x == nullptr || d_q == nullptr || d_scale == nullptr || !aligned(d_x, 16) ||
        !aligned(d_q, 16) || !aligned(d_scale, 4) || !aligned(d_counts, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    QuantBlocksParams p;
    p.x = d_x;
    p.q = static_cast<uint8_t *>(d_q);
    p.scale = d_scale;
    p.counts = d_counts;
    p.row_stride = row_stride;
    p.groups = groups;
    p.rows = rows;
    p.H = hidden;
    p.block_rows = block_rows;
    p.bf16 = bf16 != 0;
    return launched([&] {
        return launch_quantize_blocks(p, sms, static_cast<cudaStream_t>(stream));
    });
}

size_t moe_gemm_fp8_scratch_bytes(int32_t rows) {
    if (rows < 1) return 0;
    return kStreamHeaderBytes + product_part_bytes(product_nmax(rows));
}

int moe_gemm_fp8(const void *d_xq, const float *d_x_scale, const void *d_wq,
                 const float *d_w_scale, const int32_t *d_counts, const int32_t *d_offsets,
                 int32_t groups, int32_t rows, int32_t N, int32_t hidden, void *d_out,
                 void *d_scratch, size_t scratch_bytes, void *stream) {
    if (groups < 0 || groups > kProductMaxGroups || rows < 0 || N < 1 || hidden < 16 ||
        hidden % 16 != 0 || (d_counts != nullptr && d_offsets != nullptr) ||
        !extents_ok(groups, d_offsets != nullptr ? rows : (int64_t)groups * rows, N,
                    d_offsets != nullptr ? rows : (int64_t)groups * rows, hidden))
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    if (d_xq == nullptr || d_x_scale == nullptr || d_wq == nullptr || d_w_scale == nullptr ||
        d_out == nullptr || d_scratch == nullptr || !aligned(d_xq, 16) || !aligned(d_wq, 16) ||
        !aligned(d_x_scale, 4) || !aligned(d_w_scale, 4) || !aligned(d_counts, 4) ||
        !aligned(d_offsets, 4) || !aligned(d_out, 2) || !aligned(d_scratch, 256))
        return MOE_ERR_INVALID_ARG;
    if (scratch_bytes < moe_gemm_fp8_scratch_bytes(rows)) return MOE_ERR_CAPACITY;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    ProductParams p = params(d_counts, d_offsets, d_out, d_scratch, groups, rows, N, 0, hidden,
                             product_nmax(rows));
    p.x_scale = d_x_scale;
    p.w_scale = d_w_scale;
    return launched([&] {
        return launch_gemm_fp8(p, d_xq, d_wq, sms, static_cast<cudaStream_t>(stream));
    });
}

size_t moe_gemm_ragged_scratch_bytes(void) {
    return kStreamHeaderBytes + product_part_bytes(kProductMaxCols);
}

int moe_gemm_ragged(const void *d_x, const void *d_w, const int32_t *d_offsets, int32_t groups,
                    int32_t rows, int32_t N, int32_t hidden, void *d_out, void *d_scratch,
                    size_t scratch_bytes, void *stream) {
    if (!ragged_shape_ok(groups, rows, N, hidden, false) ||
        !extents_ok(groups, rows, N, rows, hidden))
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    const int bad = check_ragged(d_x, d_w, d_offsets, d_out, 2, d_scratch, scratch_bytes);
    if (bad != MOE_OK) return bad;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    const ProductParams p = params(nullptr, d_offsets, d_out, d_scratch, groups, rows, N, 0,
                                   hidden, kProductMaxCols);
    return launched([&] {
        return launch_gemm_ragged(p, d_x, d_w, sms, static_cast<cudaStream_t>(stream));
    });
}

int moe_gemm_ragged_input_grad(const void *d_dy, const void *d_w, const int32_t *d_offsets,
                               int32_t groups, int32_t rows, int32_t N, int32_t hidden,
                               void *d_dx, void *d_scratch, size_t scratch_bytes, void *stream) {
    if (!ragged_shape_ok(groups, rows, N, hidden, true) ||
        !extents_ok(groups, rows, hidden, rows, N))
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    const int bad = check_ragged(d_dy, d_w, d_offsets, d_dx, 2, d_scratch, scratch_bytes);
    if (bad != MOE_OK) return bad;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    const ProductParams p = params(nullptr, d_offsets, d_dx, d_scratch, groups, rows, hidden, 0,
                                   N, kProductMaxCols);
    return launched([&] {
        return launch_gemm_ragged_input_grad(p, d_dy, d_w, sms, static_cast<cudaStream_t>(stream));
    });
}

int moe_gemm_ragged_weight_grad(const void *d_dy, const void *d_x, const int32_t *d_offsets,
                                int32_t groups, int32_t rows, int32_t N, int32_t hidden,
                                int32_t fp32, int32_t accumulate, void *d_dw, void *d_scratch,
                                size_t scratch_bytes, void *stream) {
    if (!ragged_shape_ok(groups, rows, N, hidden, true) || (accumulate && !fp32) ||
        !extents_ok(groups, rows, N, (int64_t)groups * hidden, 1))
        return MOE_ERR_INVALID_ARG;
    if (groups == 0) return MOE_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums of nothing
        if (accumulate) return MOE_OK;
        if (d_dw == nullptr || !aligned(d_dw, 16)) return MOE_ERR_INVALID_ARG;
        const size_t bytes = (size_t)groups * N * hidden * (fp32 ? 4 : 2);
        return cudaMemsetAsync(d_dw, 0, bytes, st) == cudaSuccess ? MOE_OK : cuda_failed();
    }
    const int bad = check_ragged(d_dy, d_x, d_offsets, d_dw, 16, d_scratch, scratch_bytes);
    if (bad != MOE_OK) return bad;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    ProductParams p = params(nullptr, d_offsets, d_dw, d_scratch, groups, rows, N, hidden, 0,
                             kProductMaxCols);
    p.f32 = fp32 != 0;
    p.accumulate = accumulate != 0;
    return launched([&] { return launch_gemm_ragged_weight_grad(p, d_dy, d_x, sms, st); });
}

}  // extern "C"
