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
// The quotients come from one reciprocal a block and remainder steps (fp8.cuh
// explains them): two steps, which give the correctly rounded x / scale, for
// fp32; for bf16 one step, which leaves the same code for every pair of a bf16
// maximum and a bf16 value (128 x 128 pairs of significands and the binades in
// which a code is not zero; a test goes through all of them).
//
// Memory bound: each value is read once and its code written once.  Eight lanes
// hold a row of a block, 16 values each, so that a block's scale is computed
// once for 16 values of a lane.  32768 bf16 rows of 7168 take 118 us, 6.0 TB/s
// (sixteen lanes of 8 values: 210; three CTAs an SM instead of four: 123; the next
// blocks' loads in flight, or one division for four blocks: nothing gained); 16384
// rows as fp32 95 us, 6.2 TB/s; as 128 x 128 blocks 55 us in bf16, 96 us in fp32.
#include "fp8.cuh"
#include "kernels.h"
#include "product.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kRowLanes = 8;    // lanes of a row of a block, 16 values each
constexpr int kRowBlocks = 4;   // 1 x 128 blocks that such lanes have in hand

__device__ __forceinline__ fp8::RowScale block_scale(float amax) {
    fp8::RowScale r;
    r.s = amax > 0.0f ? fmaxf(__fdiv_rn(amax, fp8::kMax), 0x1p-126f) : 1.0f;
    r.m = r.s < 0x1p-100f ? 0x1p100f : (r.s > 0x1p100f ? 0x1p-100f : 1.0f);
    r.sd = __fmul_rn(r.s, r.m);
    r.y = __frcp_rn(r.sd);
    return r;
}

// Two quotients -> two codes without their signs (they are the values').
template <bool BF16, bool SCALED>
__device__ __forceinline__ uint32_t code2(float a, float b, const fp8::RowScale &r) {
    x2::f2 xs = x2::pack(a, b);
    if (SCALED) xs = x2::mul(xs, x2::pack(r.m, r.m));
    const x2::f2 y = x2::pack(r.y, r.y), nsd = x2::pack(-r.sd, -r.sd);
    x2::f2 q = x2::mul(xs, y);
    q = x2::fma(x2::fma(q, nsd, xs), y, q);
    if (!BF16) q = x2::fma(x2::fma(q, nsd, xs), y, q);
    float qa, qb;
    x2::unpack(q, qa, qb);
    return fp8::cvt2(qa, qb);
}

// Sixteen values of a row of a block as loaded: 16-byte chunks `lane`,
// `lane` + 8, ... of the block's row.
template <bool BF16>
struct Vec16 {
    static constexpr int kChunks = BF16 ? 2 : 4, kPer = BF16 ? 8 : 4;  // values of a chunk
    uint4 v[kChunks];
    // (the chunks below `cols` of the row at x + at; zeros past them)
    __device__ __forceinline__ void load(const void *x, long long at, int lane, int cols) {
        const uint4 *p =
            reinterpret_cast<const uint4 *>(static_cast<const char *>(x) + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
            v[k] = (lane + k * kRowLanes) * kPer < cols ? __ldcs(p + lane + k * kRowLanes)
                                                        : make_uint4(0, 0, 0, 0);
    }
    // bits of the largest |x| (NaN above infinity above every number)
    __device__ __forceinline__ uint32_t most() const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            if (BF16) {  // two 16-bit lanes at a time
                const uint32_t a = 0x7fff7fffu;
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[k].x & a, v[k].y & a),
                                         __vmaxu2(v[k].z & a, v[k].w & a)));
            } else {
                const uint32_t a = 0x7fffffffu;
                m = max(m, max(max(v[k].x & a, v[k].y & a), max(v[k].z & a, v[k].w & a)));
            }
        }
        return BF16 ? max(m << 16, m & 0xffff0000u) : m;
    }
    template <bool SCALED>
    __device__ __forceinline__ void store_as(uint8_t *q, const fp8::RowScale &s, int lane,
                                             int cols) const {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            const int at = lane + k * kRowLanes;
            if (at * kPer >= cols) continue;
            if (BF16) {
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c[i] = code2<true, SCALED>(__uint_as_float(w[i] << 16),
                                               __uint_as_float(w[i] & 0xffff0000u), s);
                uint2 o;  // the high bytes of the values hold their signs
                o.x = ((c[0] | c[1] << 16) & 0x7f7f7f7fu) |
                      (__byte_perm(w[0], w[1], 0x7531) & 0x80808080u);
                o.y = ((c[2] | c[3] << 16) & 0x7f7f7f7fu) |
                      (__byte_perm(w[2], w[3], 0x7531) & 0x80808080u);
                reinterpret_cast<uint2 *>(q)[at] = o;
            } else {
                const uint32_t lo = code2<false, SCALED>(__uint_as_float(w[0]),
                                                         __uint_as_float(w[1]), s);
                const uint32_t hi = code2<false, SCALED>(__uint_as_float(w[2]),
                                                         __uint_as_float(w[3]), s);
                const uint32_t sign = __byte_perm(__byte_perm(w[0], w[1], 0x0073),
                                                  __byte_perm(w[2], w[3], 0x0073), 0x5410);
                reinterpret_cast<uint32_t *>(q)[at] =
                    ((lo | hi << 16) & 0x7f7f7f7fu) | (sign & 0x80808080u);
            }
        }
    }
    // the codes of a block with maximum bits `m`, to the row at q
    __device__ __forceinline__ void store(uint8_t *q, uint32_t m, const fp8::RowScale &s, int lane,
                                          int cols) const {
        if (m >= 0x7f800000u) {
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int at = lane + k * kRowLanes;
                if (at * kPer >= cols) continue;
                if (BF16) reinterpret_cast<uint2 *>(q)[at] = make_uint2(0, 0);
                else reinterpret_cast<uint32_t *>(q)[at] = 0;
            }
        } else if (s.m == 1.0f) {
            store_as<false>(q, s, lane, cols);
        } else {
            store_as<true>(q, s, lane, cols);
        }
    }
};

__device__ __forceinline__ float scale_of(uint32_t m, const fp8::RowScale &s) {
    return m < 0x7f800000u ? s.s : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ fp8::RowScale scale_from(uint32_t m) {
    return block_scale(m < 0x7f800000u ? __uint_as_float(m) : 0.0f);
}

// Blocks of 1 x 128: kRowLanes lanes a block, kRowBlocks consecutive blocks
// (row-major) at a time, their loads issued first.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 2)
    quantize_rows_kernel(const QuantBlocksParams p) {
    ptx::grid_dependency_wait();
    constexpr int kTeams = kThreads / kRowLanes;
    const int lane = threadIdx.x % kRowLanes, team = threadIdx.x / kRowLanes;
    const int KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    const long long blocks = (long long)p.groups * p.rows * KB;
    const long long step = (long long)gridDim.x * kTeams * kRowBlocks;
    const long long step_r = step / KB;
    const int step_k = (int)(step - step_r * KB);
    long long b = ((long long)blockIdx.x * kTeams + team) * kRowBlocks;
    long long r0 = b / KB;
    int k0 = (int)(b - r0 * KB);
    // (the teams of a warp make the same number of rounds)
    const int behind = team % (32 / kRowLanes) * kRowBlocks;
    for (; b - behind < blocks; b += step) {
        Vec16<BF16> x[kRowBlocks];
        long long row[kRowBlocks];
        int col[kRowBlocks];
        bool live[kRowBlocks];
        long long r = r0;
        int kb = k0;
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i) {
            row[i] = r;
            col[i] = kb * kScaleBlock;
            live[i] = b + i < blocks;
            if (live[i] && p.counts != nullptr) {
                const long long g = r / p.rows;
                live[i] = r - g * p.rows < __ldg(p.counts + g);
            }
            x[i].load(p.x, r * p.row_stride + col[i], lane, live[i] ? p.H - col[i] : 0);
            if (++kb == KB) {
                kb = 0;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i) {
            uint32_t m = x[i].most();
#pragma unroll
            for (int o = kRowLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
            const fp8::RowScale s = scale_from(m);
            if (!live[i]) continue;
            x[i].store(p.q + row[i] * p.H + col[i], m, s, lane, p.H - col[i]);
            if (lane == 0) p.scale[row[i] * KB + col[i] / kScaleBlock] = scale_of(m, s);
        }
        r0 += step_r;
        k0 += step_k;
        if (k0 >= KB) {
            k0 -= KB;
            ++r0;
        }
    }
}

// Blocks of 128 x 128: a CTA a block, 4 rows a team of lanes.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_tiles_kernel(const QuantBlocksParams p) {
    __shared__ uint32_t red[2][kThreads / 32];
    ptx::grid_dependency_wait();
    constexpr int kTeams = kThreads / kRowLanes, kRows = kScaleBlock / kTeams;
    const int lane = threadIdx.x % kRowLanes, team = threadIdx.x / kRowLanes;
    const int KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    const int RB = (p.rows + kScaleBlock - 1) / kScaleBlock;
    const long long blocks = (long long)p.groups * RB * KB;
    int turn = 0;
    for (long long b = blockIdx.x; b < blocks; b += gridDim.x, turn ^= 1) {
        const long long gr = b / KB, g = gr / RB;
        const int kb = (int)(b - gr * KB), r0 = (int)(gr - g * RB) * kScaleBlock + team;
        const int col = kb * kScaleBlock;
        Vec16<BF16> x[kRows];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            x[i].load(p.x, (g * p.rows + r0 + i * kTeams) * p.row_stride + col, lane,
                      r0 + i * kTeams < p.rows ? p.H - col : 0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) m = max(m, x[i].most());
        m = __reduce_max_sync(kFull, m);
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, red[turn][w]);
        const fp8::RowScale s = scale_from(m);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (r0 + i * kTeams < p.rows)
                x[i].store(p.q + (g * p.rows + r0 + i * kTeams) * p.H + col, m, s, lane,
                           p.H - col);
        if (threadIdx.x == 0) p.scale[b] = scale_of(m, s);
    }
}

}  // namespace

cudaError_t launch_quantize_blocks(const QuantBlocksParams &p, int num_sms, cudaStream_t st) {
    const long long KB = (p.H + kScaleBlock - 1) / kScaleBlock;
    long long ctas;
    if (p.block_rows == 1) {
        const long long per = kThreads / kRowLanes * kRowBlocks;
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
