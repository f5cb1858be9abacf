// product.h -- parameter blocks and host launchers of the experts' products
// (gemm_fp8.cu, gemm_ragged.cu) and of the block quantiser
// (quantize_blocks.cu).  Internal to libmoe_a2a.so.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "layer.h"

namespace moe {

// Values along k and output channels that share a scale of the 8-bit product.
constexpr int kScaleBlock = 128;

// Block quantiser: rows of `groups` planes of `rows` rows each.
struct QuantBlocksParams {
    const void *x;          // fp32 or bf16, row r of the planes at r * row_stride
    uint8_t *q;             // e4m3 [groups][rows][H]
    float *scale;           // [groups][ceil(rows / block_rows)][ceil(H / 128)]
    const int32_t *counts;  // [groups] rows in use, or null (all); block_rows = 1 only
    long long row_stride;
    int groups, rows, H;
    int block_rows;         // 1 or 128
    int bf16;
};
cudaError_t launch_quantize_blocks(const QuantBlocksParams &p, int num_sms, cudaStream_t st);

// The products.  Each is a sum over k of A[lane][k] * B[column][k]: the lanes
// are output channels (or, for the gradient of the maps, their rows), the
// columns rows of tokens (or the maps' columns).
constexpr int kProductMaxGroups = 1024;
// 32-bit coordinates, with room for rounding up to whole tiles
constexpr int kProductMaxExtent = INT32_MAX - (1 << 24);
// of k, where tiles are cut along it: the blocks of all cut tiles are numbered with 32 bits
constexpr int kProductMaxDepth = 1 << 28;
static_assert((long long)kStreamMaxCtas * 5 / 4 * 2 * (kProductMaxDepth / 64) <= INT32_MAX,
              "numbers of blocks (twice that in between)");
constexpr int kProductMaxCols = 256;  // columns of a tile, at most

struct ProductParams {
    const int32_t *counts;   // [G] rows in use of each plane, or null
    const int32_t *offsets;  // [G + 1] first row of each group, or null (planes)
    const float *x_scale, *w_scale;  // 8-bit product
    const void *a, *b;       // gradient of the maps: dy and x
    void *out;
    StreamHeader *header;
    float *part;             // [CTAs][2][nmax][128]
    int G;
    int M;                   // rows of a plane, or (offsets) all rows
    int lanes, cols, depth;  // extents: lanes; maps' columns (gradient of the maps); k
    int nmax;                // columns that a part has room for
    int f32, accumulate;     // gradient of the maps: type, added to what is there
};

// Columns a part of the 8-bit product needs for M rows of tokens (a group of
// kProductTurnFrom tokens or more may have tiles of kProductMaxCols channels; for fewer
// tokens as columns are faster: 32 groups of 4096 x 2048, 32 tokens each 49 and 54 us, 33
// tokens 55 and 54, 64 tokens 60 and 55, 128 tokens 77 and 59).
constexpr int kProductTurnFrom = 33;
inline int product_nmax(int M) {
    if (M >= kProductTurnFrom) return kProductMaxCols;
    int n = 16;
    while (n < M) n *= 2;
    return n;
}

inline size_t product_part_bytes(int nmax) {
    return (size_t)kStreamMaxCtas * 2 * (size_t)nmax * 128 * sizeof(float);
}

cudaError_t launch_gemm_fp8(ProductParams p, const void *xq, const void *wq, int num_sms,
                            cudaStream_t st);
// x [M][depth], w [G][lanes][depth]
cudaError_t launch_gemm_ragged(ProductParams p, const void *x, const void *w, int num_sms,
                               cudaStream_t st);
// dy [M][depth], w [G][depth][lanes]
cudaError_t launch_gemm_ragged_input_grad(ProductParams p, const void *dy, const void *w,
                                          int num_sms, cudaStream_t st);
// dy [M][lanes], x [M][cols]
cudaError_t launch_gemm_ragged_weight_grad(ProductParams p, const void *dy, const void *x,
                                           int num_sms, cudaStream_t st);

}  // namespace moe
