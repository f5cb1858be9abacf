// gemm_ragged.cu -- one linear map per expert over rows that stand one
// expert after another, and its gradients (expert_product.cuh).
//
// With rows offsets[e] <= m < offsets[e + 1] of expert e and maps W_e (N x H):
//   y[m][n]    = bf16_rn( sum_h x[m][h] * W_e[n][h] )
//   dx[m][h]   = bf16_rn( sum_n dy[m][n] * W_e[n][h] )
//   dW_e[n][h] = sum_m dy[m][n] * x[m][h]            (bf16 or fp32, or added to fp32)
// products of bf16 values summed in fp32.  Rows of no expert are not written;
// the dW_e of an expert without rows is zero.
#include "expert_product.cuh"

namespace moe {

using namespace product;

cudaError_t launch_gemm_ragged(ProductParams p, const void *x, const void *w, int num_sms,
                               cudaStream_t st) {
    CUtensorMap a, b, b8;
    if (!map_3d(&a, w, p.G, p.lanes, p.depth, 64, kTileRows, false) ||
        !map_2d(&b, x, p.M, p.depth, 64, kBigBox, false) ||
        !map_2d(&b8, x, p.M, p.depth, 64, kSmallBox, false))
        return cudaErrorInvalidValue;
    return launch<kForward>(p, a, b, b8, num_sms, st);
}

cudaError_t launch_gemm_ragged_input_grad(ProductParams p, const void *dy, const void *w,
                                          int num_sms, cudaStream_t st) {
    CUtensorMap a, b, b8;
    if (!map_3d(&a, w, p.G, p.depth, p.lanes, 64, 64, false) ||
        !map_2d(&b, dy, p.M, p.depth, 64, kBigBox, false) ||
        !map_2d(&b8, dy, p.M, p.depth, 64, kSmallBox, false))
        return cudaErrorInvalidValue;
    return launch<kInputGrad>(p, a, b, b8, num_sms, st);
}

cudaError_t launch_gemm_ragged_weight_grad(ProductParams p, const void *dy, const void *x,
                                           int num_sms, cudaStream_t st) {
    CUtensorMap a, b, out;
    if (!map_2d(&a, dy, p.M, p.lanes, 64, 64, false) ||
        !map_2d(&b, x, p.M, p.cols, 64, 64, false))
        return cudaErrorInvalidValue;
    p.a = dy;
    p.b = x;
    if (!map_3d(&out, p.out, p.G, p.lanes, p.cols, p.f32 ? 32 : 64, kBoxRows, false, p.f32 != 0))
        return cudaErrorInvalidValue;
    return launch<kWeightGrad>(p, a, b, out, num_sms, st);
}

}  // namespace moe
