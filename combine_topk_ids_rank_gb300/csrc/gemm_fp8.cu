// gemm_fp8.cu -- product of e4m3 codes with a scale for each block of 128
// codes of a token and one for each 128 x 128 block of the weights, dense,
// grouped over the experts' planes, or over rows that stand one group after
// another (expert_product.cuh).
//
// Operation, group g, token row m, channel n:
//   out[m][n] = bf16_rn( sum over blocks b of RN32(sx[m][b] * sw[g][n / 128][b]) * d_b ),
//   d_b = sum over h in block b of xq[m][h] * wq[g][n][h],
// the products of codes exact, the sums in fp32 (d_b as the tensor cores add,
// the outer sum by fused multiply-adds in ascending b).
#include "expert_product.cuh"

namespace moe {

cudaError_t launch_gemm_fp8(ProductParams p, const void *xq, const void *wq, int num_sms,
                            cudaStream_t st) {
    using namespace product;
    // Few tokens in every group (no tile is turned: 16 x 7168 x 4096 13.1 us, 16.1 with the
    // other kernel), or, as far as the host knows, in most of them (32 uneven groups of 4096 x
    // 2048: 30 tokens on average 52 us, 59 with the other; 39 tokens 54 and 55; 56 tokens 58 and
    // 58; 62 tokens 61 and 53), or so few tiles that narrower ones keep more SMs at work (333 x
    // 1000 x 1040: 9.7 us and 11.0; 600 x 2048 x 4096: 25.0 and 26.6).
    const long long tiles = ((long long)p.M + kTileRows - 1) / kTileRows *
                            ((p.lanes + kProductMaxCols - 1) / kProductMaxCols);
    const bool one = p.G == 1 && p.counts == nullptr && p.offsets == nullptr;
    const bool narrow = p.M < kProductTurnFrom || (p.offsets != nullptr && p.M / p.G < 48) ||
                        (one && tiles * 2 <= num_sms);
    CUtensorMap a, b, b8;
    const long long rows = p.offsets != nullptr ? p.M : (long long)p.G * p.M;
    if (!map_3d(&a, wq, p.G, p.lanes, p.depth, kAtom, narrow ? 64 : kTileRows, true) ||
        !map_2d(&b, xq, rows, p.depth, kAtom, kBigBox, true) ||
        !map_2d(&b8, xq, rows, p.depth, kAtom, kSmallBox, true))
        return cudaErrorInvalidValue;
    return narrow ? launch<kFp8Narrow>(p, a, b, b8, num_sms, st)
                  : launch<kFp8>(p, a, b, b8, num_sms, st);
}

}  // namespace moe
