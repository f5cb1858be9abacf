// layer.h -- parameter blocks and host launchers of the operators around
// dispatch and combine: the router gate (topk_gate.cu), the 8-bit integer
// row quantiser (quantize_int8.cu), the 8-bit integer product
// (gemm_int8.cu) and the whole layer for a few tokens (layer_small.cu).
// Internal to libmoe_a2a.so.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace moe {

// Router gate: one warp per token.
constexpr int kGateMaxExperts = 1024;
struct TopkGateParams {
    const void *logits;    // fp32 or bf16 [tokens][row_stride]
    int32_t *topk_ids;     // [tokens][K]
    float *topk_w;         // [tokens][K]
    long long tokens, row_stride;
    int E, K;
    int bf16;              // element type of the logits
    int sigmoid;           // 0: softmax, 1: sigmoid
    int renormalize;
    float scale;
};
cudaError_t launch_topk_gate(const TopkGateParams &p, int num_sms, cudaStream_t st);

// Row quantiser: rows of `groups` planes of `rows` rows each.
struct QuantInt8Params {
    const void *x;          // fp32 or bf16, row r of the planes at r * row_stride
    int8_t *q;              // [groups][rows][H]
    float *scale;           // [groups][rows]
    const int32_t *counts;  // [groups] rows in use, or null (all)
    long long row_stride;
    int groups, rows, H;
    int bf16;
};
cudaError_t launch_quantize_rows_int8(const QuantInt8Params &p, int num_sms, cudaStream_t st);

// Device memory that the two persistent kernels keep between their CTAs.
// The header is zero between calls (the kernels leave it so).
constexpr int kStreamMaxCtas = 192;      // CTAs of a persistent launch, at most
constexpr size_t kStreamHeaderBytes = 8192;
struct StreamHeader {
    uint32_t flags;                      // sticky MOE_DEVICE_FLAG_* bits
    int32_t done[2];                     // finished quarters of output tiles, by phase
    int32_t left;                        // CTAs that are through with the counters
    int32_t pad[12];
    int32_t merged[2][kStreamMaxCtas][4];  // finished parts of the cut tile that CTA c
                                           // began, by quarter of its rows (warp)
};
static_assert(sizeof(StreamHeader) <= kStreamHeaderBytes, "header");

// Whole layer for a few tokens.
constexpr int kLayerMaxTokens = 64;
struct LayerSmallParams {
    const uint16_t *x;         // bf16 [T][H]
    const int32_t *topk_ids;   // [T][K]
    const float *topk_w;       // [T][K]
    const void *w13, *w2;      // [E][2I][H], [E][H][I]
    const float *w13_scale, *w2_scale;  // [E][2I], [E][H] (8-bit formats)
    const uint16_t *residual;  // bf16 [T][H] or null
    uint16_t *out;             // bf16 [T][H]
    StreamHeader *header;
    uint16_t *act;             // bf16 [T * K][2][I]: the activations in two terms
    float *y;                  // [T * K][H]
    float *part;               // [CTAs][2][Nmax][128]
    int T, K, E, H, I;
    int format;                // MOE_FORMAT_*
    // set by the launcher
    int nmax, ring_bytes, kshift;
};
cudaError_t launch_layer_small(LayerSmallParams p, int num_sms, cudaStream_t st);

// 8-bit integer product, dense or grouped.
constexpr int kGemmInt8MaxGroups = 1024;
// Rows, channels and hidden size: 32-bit coordinates, with room for rounding up to
// whole tiles and for the evened width of a tile (rows + tiles, at most 2^23 of them).
constexpr int kGemmInt8MaxExtent = INT32_MAX - (1 << 24);
struct GemmInt8Params {
    const int8_t *xq;          // [G][M][H]
    const float *x_scale;      // [G][M]
    const int8_t *wq;          // [G][N][H]
    const float *w_scale;      // [G][N]
    const int32_t *counts;     // [G] or null
    uint16_t *out;             // bf16 [G][M][N]
    StreamHeader *header;
    float *part;               // [CTAs][2][nmax][128]
    int G, M, N, H;
    int nmax;                  // token columns of a tile, set by the launcher
};
int gemm_int8_nmax(int M);  // token columns a part needs for M rows
cudaError_t launch_gemm_int8(GemmInt8Params p, int num_sms, cudaStream_t st);

}  // namespace moe
