// quantize_blocks.cu -- rows to e4m3 codes with one scale for each block of
// 1 x 128 values (activations) or 128 x 128 values (weights): the operands of
// the 8-bit floating-point product.
//
// Operation, per block with values x (bf16 or fp32):
//   amax = max |x|,  scale = max(RN32(amax / 448), 2^-126), 1 if amax = 0,
//   q = e4m3(RN32(x / scale)), to nearest, ties to even, saturating at 448.
// A block that holds a NaN or an infinity has scale NaN and zero codes, so
// whatever is computed from it is NaN.  The last blocks of a row (and of a
// column of tiles) are what is left.
//
// The quotients are the correctly rounded ones of fp8.cuh: one reciprocal a
// block and two remainder steps.  Memory bound: each value is read once and
// its code written once.  Sixteen lanes hold a row of a block, 8 values each.
#include "fp8.cuh"
#include "kernels.h"
#include "product.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kRowBlocks = 4;   // 1 x 128 blocks that a half-warp has in hand

__device__ __forceinline__ fp8::RowScale block_scale(float amax) {
    fp8::RowScale r;
    r.s = amax > 0.0f ? fmaxf(__fdiv_rn(amax, fp8::kMax), 0x1p-126f) : 1.0f;
    r.m = r.s < 0x1p-100f ? 0x1p100f : (r.s > 0x1p100f ? 0x1p-100f : 1.0f);
    r.sd = __fmul_rn(r.s, r.m);
    r.y = __frcp_rn(r.sd);
    return r;
}

// Eight values as loaded.
template <bool BF16>
struct Vec8 {
    uint4 v[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *x, long long at) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(x) +
                                                         at * (BF16 ? 2 : 4));
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) v[k] = __ldcs(p + k);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) v[k] = make_uint4(0, 0, 0, 0);
    }
    // bits of the largest |x| (NaN above infinity above every number)
    __device__ __forceinline__ uint32_t most() const {
        if (BF16) {  // two 16-bit lanes at a time
            const uint32_t k = 0x7fff7fffu;
            const uint32_t a = __vmaxu2(__vmaxu2(v[0].x & k, v[0].y & k),
                                        __vmaxu2(v[0].z & k, v[0].w & k));
            return max(a << 16, a & 0xffff0000u);
        } else {
            const uint32_t k = 0x7fffffffu;
            const uint4 w = v[BF16 ? 0 : 1];
            const uint32_t a = max(max(v[0].x & k, v[0].y & k), max(v[0].z & k, v[0].w & k));
            return max(a, max(max(w.x & k, w.y & k), max(w.z & k, w.w & k)));
        }
    }
    __device__ __forceinline__ uint2 codes(const fp8::RowScale &s) const {
        float f[8];
        if (BF16) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint4 b = v[BF16 ? 0 : 1];
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        }
        return s.m == 1.0f ? fp8::quantize8<false>(f, s) : fp8::quantize8<true>(f, s);
    }
};

__device__ __forceinline__ bool finite_bits(uint32_t m) { return m < 0x7f800000u; }

// Blocks of 1 x 128: a half-warp a block, kRowBlocks blocks of consecutive
// positions (row-major) at a time, their loads issued first.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantBlocksParams p) {
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 15;
    const int KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    const long long blocks = (long long)p.groups * p.rows * KB;
    const long long step = (long long)gridDim.x * (kThreads / 16) * kRowBlocks;
    // (both halves of a warp make the same number of rounds)
    long long b0 = ((long long)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kRowBlocks;
    const long long first = b0 - (threadIdx.x >> 4 & 1) * kRowBlocks;
    for (long long w0 = first; w0 < blocks; w0 += step, b0 += step) {
        Vec8<BF16> x[kRowBlocks];
        long long row[kRowBlocks];
        int col[kRowBlocks];
        bool live[kRowBlocks];
        long long r = b0 / KB;
        int kb = (int)(b0 - r * KB);
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i) {
            row[i] = r;
            col[i] = kb * kScaleBlock + lane * 8;
            live[i] = b0 + i < blocks;
            if (live[i] && p.counts != nullptr) {
                const long long g = r / p.rows;
                live[i] = r - g * p.rows < __ldg(p.counts + g);
            }
            if (live[i] && col[i] < p.H) x[i].load(p.x, r * p.row_stride + col[i]);
            else x[i].clear();
            if (++kb == KB) {
                kb = 0;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i) {
            uint32_t m = x[i].most();
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
            const bool finite = finite_bits(m);
            const fp8::RowScale s = block_scale(finite ? __uint_as_float(m) : 0.0f);
            if (!live[i]) continue;
            if (col[i] < p.H)
                *reinterpret_cast<uint2 *>(p.q + row[i] * p.H + col[i]) =
                    finite ? x[i].codes(s) : make_uint2(0, 0);
            if (lane == 0)
                p.scale[row[i] * KB + col[i] / kScaleBlock] =
                    finite ? s.s : __uint_as_float(0x7fc00000u);
        }
    }
}

// Blocks of 128 x 128: a CTA a block, 8 rows a half-warp.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_tiles_kernel(const QuantBlocksParams p) {
    __shared__ uint32_t red[2][kThreads / 32];
    ptx::grid_dependency_wait();
    constexpr int kRows = kScaleBlock / (kThreads / 16);
    const int lane = threadIdx.x & 15, sub = threadIdx.x >> 4;
    const int KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    const int RB = (p.rows + kScaleBlock - 1) / kScaleBlock;
    const long long blocks = (long long)p.groups * RB * KB;
    int turn = 0;
    for (long long b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const long long gr = b / KB, g = gr / RB;
        const int kb = (int)(b - gr * KB), r0 = (int)(gr - g * RB) * kScaleBlock;
        const int col = kb * kScaleBlock + lane * 8;
        Vec8<BF16> x[kRows];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * (kThreads / 16) + sub;
            if (r < p.rows && col < p.H) x[i].load(p.x, (g * p.rows + r) * p.row_stride + col);
            else x[i].clear();
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = max(m, x[i].most());
        m = __reduce_max_sync(kFull, m);
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, red[turn][w]);
        const bool finite = finite_bits(m);
        const fp8::RowScale s = block_scale(finite ? __uint_as_float(m) : 0.0f);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * (kThreads / 16) + sub;
            if (r < p.rows && col < p.H)
                *reinterpret_cast<uint2 *>(p.q + (g * p.rows + r) * p.H + col) =
                    finite ? x[i].codes(s) : make_uint2(0, 0);
        }
        if (threadIdx.x == 0) p.scale[b] = finite ? s.s : __uint_as_float(0x7fc00000u);
    }
}

}  // namespace

cudaError_t launch_quantize_blocks(const QuantBlocksParams &p, int num_sms, cudaStream_t st) {
    const long long KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    long long ctas;
    if (p.block_rows == 1) {
        const long long per = kThreads / 16 * kRowBlocks;
        ctas = ((long long)p.groups * p.rows * KB + per - 1) / per;
    } else {
        ctas = (long long)p.groups * ((p.rows + kScaleBlock - 1) / kScaleBlock) * KB;
    }
    const long long most = (long long)num_sms * 8;
    const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kThreads);
    if (p.block_rows == 1)
        return launch_pdl(p.bf16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>, grid,
                          block, 0, st, p);
    return launch_pdl(p.bf16 ? quantize_tiles_kernel<true> : quantize_tiles_kernel<false>, grid,
                      block, 0, st, p);
}

}  // namespace moe
