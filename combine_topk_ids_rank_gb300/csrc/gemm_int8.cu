// gemm_int8.cu -- product of 8-bit integer codes with one scale per token
// and one per output channel, dense or grouped over the experts' planes.
//
// Operation, group g, token row m < counts[g] (all M without counts), channel n:
//   out[g][m][n] = bf16_rn( (sum_h xq[g][m][h] * wq[g][n][h]) * sx[g][m] * sw[g][n] ),
// two fp32 multiplies and one narrowing after the sum.  Rows past a count
// are neither read for a result nor written.
//
// sm_103a has no 8-bit integer product on its 5th-generation tensor cores
// (.kind::i8 is refused for this target), so the codes are widened to f16,
// which holds every 8-bit integer, and multiplied there: the products are
// exact, and the fp32 sums are exact integers as long as they stay within
// 2^24 in magnitude; past that each addition rounds to 24 bits.  Both
// operands stay 8 bits wide in memory, in L2 and on the way to the SM.
//
// GB300 design (stream.cuh: weights are the A operand, 128 channels a tile,
// up to 256 tokens the columns): persistent CTAs, one per SM.  Whole waves
// of tiles go round robin; what is left over is cut evenly by k.
//   warps 0-3: epilogue (tensor-memory lane quadrants);
//   warps 4-7: widen a stage's 128 weight rows into tensor memory, which the
//     products read as their A operand;
//   warps 8-15: widen the token rows into f16 tiles in shared memory, half a
//     k-block (64 codes) at a time;
//   warp 16: producer (TMA, 128-byte swizzle); warp 17: MMA issuer.
#include "kernels.h"
#include "ptx.cuh"
#include "smem_limit.h"
#include "stream.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

#include "moe_a2a.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

using namespace stream;

constexpr int kWeightWarp0 = 4, kTokenWarp0 = 8, kTokenWarps = 8;
constexpr int kProducerWarp = 16, kMmaWarp = 17, kThreads = 18 * 32;
constexpr int kMaxCols = 256;           // tokens of a tile
constexpr int kTmemCols = 512;          // accumulators, then widened weights
constexpr int kSlots = 4, kSlotCols = kBlockK / 2;
constexpr int kWeightBytes = kTileRows * kBlockK;
constexpr int kMaxStages = 12, kMaxHalves = 8;
// dynamic shared memory: 227 KB a CTA less the static tables
constexpr size_t kMaxDynamic = (227 - 12) * 1024;
constexpr int kRowGroup = 16;           // row tiles of a raster group

struct Ring {
    int nmax;      // token rows a stage holds
    int box;       // rows of a token TMA box
    int stages;    // raw stages: 128 weight rows + nmax token rows of 128 codes
    int halves;    // widened token tiles: nmax rows of 64 f16
};

// The tiles of a call: groups in turn; in a group, blocks of kRowGroup row
// tiles, token tile outer and row tile inner.
struct Tiles {
    const int *first;   // [G + 1]
    const int *count;   // [G] token rows
    int G, M, N, rtiles, nmax;
    __device__ int token_tiles(int c) const { return (c + nmax - 1) / nmax; }
    __device__ int width(int c) const {  // token rows of a tile: even, multiple of 16
        const int k = token_tiles(c);
        return ((c + k - 1) / k + 15) / 16 * 16;
    }
    __device__ void of(int t, int &g, int &r, int &m0, int &rows) const {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= t) lo = mid; else hi = mid - 1;
        }
        g = lo;
        const int c = count[g], k = token_tiles(c), w = width(c);
        const int u = t - first[g], block = u / (kRowGroup * k);
        const int in = min(kRowGroup, rtiles - block * kRowGroup);
        const int v = u - block * kRowGroup * k;
        m0 = v / in * w;
        r = block * kRowGroup + v % in;
        rows = min(w, c - m0);
    }
};

// The work of a CTA in order: its parts of the cut tiles, then whole tiles.
struct Work {
    Segments segs;
    int tile, tiles, step, blocks;
    __device__ Work(const Cut &ct, int cut_tiles, int tiles_, int blocks_, int cta, int ctas)
        : segs(ct, cta, blocks_), tile(cut_tiles + cta), tiles(tiles_), step(ctas),
          blocks(blocks_) {}
    __device__ bool next(Segment &s) {
        if (segs.next(s)) return true;
        if (tile >= tiles) return false;
        s.tile = tile;
        s.k0 = 0;
        s.k1 = blocks;
        tile += step;
        return true;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const GemmInt8Params p,
                     const Ring ring) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t raw_full[kMaxStages], raw_free[kMaxStages];
    __shared__ uint64_t wide_full[kSlots], wide_free[kSlots];
    __shared__ uint64_t half_full[kMaxHalves], half_free[kMaxHalves];
    __shared__ uint64_t acc_full[2], acc_free[2], drained;
    __shared__ int s_first[kGemmInt8MaxGroups + 1], s_count[kGemmInt8MaxGroups];
    __shared__ float s_sx[kMaxCols];
    __shared__ uint32_t s_taddr;
    __shared__ int s_last;
    __shared__ volatile int s_failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;

    const uint32_t base = ptx::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (base & 1023u)) & 1023u);
    const int raw_bytes = kWeightBytes + ring.nmax * kAtom, half_bytes = ring.nmax * kAtom;
    uint8_t *wide = smem + ring.stages * raw_bytes;  // raw_bytes: a multiple of 1024
    auto raw_w = [&](int s) { return smem + s * raw_bytes; };
    auto raw_x = [&](int s) { return smem + s * raw_bytes + kWeightBytes; };

    for (int g = tid; g < p.G; g += kThreads) {
        int c = p.M;
        if (p.counts != nullptr) c = min(max(__ldg(p.counts + g), 0), p.M);
        s_count[g] = c;
    }
    if (tid == 0) {
        for (int s = 0; s < ring.stages; ++s) {
            ptx::mbar_init(&raw_full[s], 1);
            ptx::mbar_init(&raw_free[s], 4 + kTokenWarps);
        }
        for (int q = 0; q < kSlots; ++q) {
            ptx::mbar_init(&wide_full[q], 4);
            ptx::mbar_init(&wide_free[q], 1);
        }
        for (int q = 0; q < ring.halves; ++q) {
            ptx::mbar_init(&half_full[q], kTokenWarps);
            ptx::mbar_init(&half_free[q], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_free[b], 4);
        }
        ptx::mbar_init(&drained, 1);
        ptx::fence_mbar_init();
        s_failed = 0;
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&s_taddr, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const int rtiles = (p.N + kTileRows - 1) / kTileRows;
    const Tiles T{s_first, s_count, p.G, p.M, p.N, rtiles, ring.nmax};
    if (warp == 0) {  // exclusive prefix of the groups' tiles
        int sum = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane, n = g < p.G ? T.token_tiles(s_count[g]) * rtiles : 0;
            int s = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            if (g < p.G) s_first[g] = sum + s - n;
            sum += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) s_first[p.G] = sum;
    }
    __syncthreads();

    const uint32_t taddr = s_taddr;
    const int tiles = s_first[p.G], blocks = (p.H + kBlockK - 1) / kBlockK;
    // Whole waves are dealt out as they are; the rest, and one wave more where
    // the rest is under a quarter of a wave (parts of a few k-blocks each cost
    // more than they balance), is cut by k.
    int waves = tiles / ctas;
    if (waves > 0 && tiles % ctas != 0 && tiles % ctas * 4 < ctas) --waves;
    const int cut_tiles = tiles - waves * ctas;
    const Cut ct = cut(cut_tiles, blocks, ctas, 4, ring.nmax <= 32 ? kAlone : 16);
    const int nacc = 2 * ring.nmax <= kMaxCols ? 2 : 1;  // accumulators
    const uint32_t slots_at = taddr + kMaxCols;

    if (warp == kProducerWarp) {
        if (ptx::elect_one()) {
            uint32_t n = 0;
            Work work(ct, cut_tiles, tiles, blocks, cta, ctas);
            Segment sg;
            while (!s_failed && work.next(sg)) {
                int g, r, m0, rows;
                T.of(sg.tile, g, r, m0, rows);
                const int boxes = (rows + ring.box - 1) / ring.box;
                const uint32_t bytes = kWeightBytes + boxes * ring.box * kAtom;
                for (int kb = sg.k0; kb < sg.k1; ++kb, ++n) {
                    const int s = (int)(n % ring.stages);
                    if (!ptx::mbar_wait_timed(&raw_free[s], ((n / ring.stages) & 1u) ^ 1u, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    ptx::mbar_arrive_expect_tx(&raw_full[s], bytes);
                    tc::tma_load_2d(raw_w(s), &map_w, kb * kBlockK, g * p.N + r * kTileRows,
                                    &raw_full[s]);
                    for (int b = 0; b < boxes; ++b)
                        tc::tma_load_2d(raw_x(s) + b * ring.box * kAtom, &map_x, kb * kBlockK,
                                        g * p.M + m0 + b * ring.box, &raw_full[s]);
                }
            }
            // copies still in flight land before shared memory goes away
            const uint32_t from = n > (uint32_t)ring.stages ? n - ring.stages : 0u;
            for (uint32_t k = from; k < n; ++k)
                ptx::mbar_wait_timed(&raw_full[k % ring.stages], (k / ring.stages) & 1u, kWaitNs);
        }
    } else if (warp == kMmaWarp) {
        if (ptx::elect_one()) {
            uint32_t n = 0, h = 0, it = 0;
            Work work(ct, cut_tiles, tiles, blocks, cta, ctas);
            Segment sg;
            for (; !s_failed && work.next(sg); ++it) {
                int g, r, m0, rows;
                T.of(sg.tile, g, r, m0, rows);
                const uint32_t idesc = tc::idesc_f16_f32(kTileRows, (rows + 15) / 16 * 16);
                const uint32_t b = it % nacc, d = taddr + b * ring.nmax;
                if (!ptx::mbar_wait_timed(&acc_free[b], ((it / nacc) & 1u) ^ 1u, kWaitNs)) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                for (int kb = sg.k0; kb < sg.k1 && !s_failed; ++kb, ++n) {
                    const uint32_t q = n % kSlots, a = slots_at + q * kSlotCols;
                    if (!ptx::mbar_wait_timed(&wide_full[q], (n / kSlots) & 1u, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    for (int hh = 0; hh < 2; ++hh, ++h) {
                        const uint32_t s = h % ring.halves;
                        if (!ptx::mbar_wait_timed(&half_full[s], (h / ring.halves) & 1u, kWaitNs)) {
                            s_failed = 1;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint64_t bd = tc::smem_desc_sw128(ptx::smem_u32(wide + s * half_bytes));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_f16_ta(d, a + 32 * hh + 8 * kk, bd + 2 * kk, idesc,
                                           kb != sg.k0 || hh != 0 || kk != 0);
                        tc::commit(&half_free[s]);
                    }
                    tc::commit(&wide_free[q]);
                }
                tc::commit(&acc_full[b]);
            }
            tc::commit(&drained);  // before tensor memory is freed
            ptx::mbar_wait_timed(&drained, 0, kWaitNs);
        }
    } else if (warp >= kWeightWarp0 && warp < kTokenWarp0) {
        // Thread l of the four warps owns weight row l of the tile = lane l.
        const int row = tid - kWeightWarp0 * 32;
        Work work(ct, cut_tiles, tiles, blocks, cta, ctas);
        Segment sg;
        uint32_t n = 0;
        while (!warp_flag(&s_failed) && work.next(sg)) {
            bool ok = true;
            for (int kb = sg.k0; kb < sg.k1 && ok; ++kb, ++n) {
                const uint32_t s = n % ring.stages, q = n % kSlots;
                ok = ptx::mbar_wait_timed(&raw_full[s], (n / ring.stages) & 1u, kWaitNs) &&
                     ptx::mbar_wait_timed(&wide_free[q], ((n / kSlots) & 1u) ^ 1u, kWaitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint8_t *src = raw_w(s) + row * kAtom;
                const uint32_t dst = slots_at + q * kSlotCols + ((uint32_t)(row & ~31) << 16);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            src + (((4 * hh + c) ^ (row & 7)) << 4));
                        int8_to_f16(v.x, w[8 * c + 0], w[8 * c + 1]);
                        int8_to_f16(v.y, w[8 * c + 2], w[8 * c + 3]);
                        int8_to_f16(v.z, w[8 * c + 4], w[8 * c + 5]);
                        int8_to_f16(v.w, w[8 * c + 6], w[8 * c + 7]);
                    }
                    tc::st_32x32(dst + 32 * hh, w);
                }
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_free[s]);
                    mbar_arrive(&wide_full[q]);
                }
            }
        }
    } else if (warp >= kTokenWarp0 && warp < kTokenWarp0 + kTokenWarps) {
        // Warp w takes the 16-code chunk w % 4 of a half and every second block
        // of 32 rows: 8 consecutive lanes read (and write) 8 different 16-byte
        // columns of the swizzled rows, so no bank is hit twice.
        const int w = warp - kTokenWarp0, c = w & 3;
        Work work(ct, cut_tiles, tiles, blocks, cta, ctas);
        Segment sg;
        uint32_t n = 0, h = 0;
        while (!warp_flag(&s_failed) && work.next(sg)) {
            int g, r, m0, rows;
            T.of(sg.tile, g, r, m0, rows);
            const int cols = (rows + 15) / 16 * 16;
            bool ok = true;
            for (int kb = sg.k0; kb < sg.k1 && ok; ++kb, ++n) {
                const uint32_t s = n % ring.stages;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait_timed(&raw_full[s],
                                                                  (n / ring.stages) & 1u, kWaitNs));
                for (int hh = 0; hh < 2 && ok; ++hh, ++h) {
                    const uint32_t q = h % ring.halves;
                    ok = __all_sync(0xffffffffu,
                                    ptx::mbar_wait_timed(&half_free[q],
                                                         ((h / ring.halves) & 1u) ^ 1u, kWaitNs));
                    if (!ok) break;
                    const uint8_t *src = raw_x(s);
                    uint8_t *dst = wide + q * half_bytes;
                    for (int row = (w >> 2) * 32 + lane; row < cols; row += 64) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            src + row * kAtom + (((4 * hh + c) ^ (row & 7)) << 4));
                        uint4 a, b;
                        int8_to_f16(v.x, a.x, a.y);
                        int8_to_f16(v.y, a.z, a.w);
                        int8_to_f16(v.z, b.x, b.y);
                        int8_to_f16(v.w, b.z, b.w);
                        uint8_t *to = dst + row * kAtom;
                        *reinterpret_cast<uint4 *>(to + (((2 * c) ^ (row & 7)) << 4)) = a;
                        *reinterpret_cast<uint4 *>(to + (((2 * c + 1) ^ (row & 7)) << 4)) = b;
                    }
                    ptx::fence_proxy_async_smem();  // read next by the tensor cores
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&half_full[q]);
                }
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                if (lane == 0) mbar_arrive(&raw_free[s]);
            }
        }
    } else if (warp < 4) {
        Work work(ct, cut_tiles, tiles, blocks, cta, ctas);
        Segment sg;
        for (uint32_t it = 0; work.next(sg); ++it) {
            const uint32_t b = it % nacc;
            const bool ok = ptx::mbar_wait_timed(&acc_full[b], (it / nacc) & 1u, kWaitNs);
            if (epi_any(!ok || s_failed)) {  // (all four warps leave together)
                s_failed = 1;
                break;
            }
            tc::fence_after_sync();
            int g, r, m0, rows;
            T.of(sg.tile, g, r, m0, rows);
            const uint32_t acc = taddr + b * ring.nmax + ((uint32_t)(tid & ~31) << 16);
            const bool whole = sg.k0 == 0 && sg.k1 == blocks;
            const Parts parts(whole ? Cut(1, 1, blocks) : ct, whole ? 0 : sg.tile, blocks);
            auto part_of = [&](int c) {
                return p.part + ((size_t)(2 * c + parts.slot(c)) * p.nmax) * kTileRows + tid;
            };
            for (int i = tid; i < rows; i += 128)
                s_sx[i] = __ldg(p.x_scale + (size_t)g * p.M + m0 + i);
            if (!whole) {
                float *to = part_of(cta);
                for (int n0 = 0; n0 < rows; n0 += 16) {
                    uint32_t v[16];
                    tc::ld_32x16(acc + n0, v);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (n0 + i < rows) __stcg(to + (n0 + i) * kTileRows, __uint_as_float(v[i]));
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_free[b]);
                __threadfence();
                epi_sync();
                if (tid == 0) {
                    int *m = &p.header->merged[0][parts.c0][0];
                    s_last = atomicAdd(m, 1) == parts.count() - 1;
                    if (s_last) *m = 0;  // for the next call
                }
                epi_sync();
                if (!s_last) continue;
                __threadfence();
            } else {
                epi_sync();
            }
            const int chan = r * kTileRows + tid;
            const bool live = chan < p.N;
            const float sw = live ? __ldg(p.w_scale + (size_t)g * p.N + chan) : 0.0f;
            uint16_t *out = p.out + ((size_t)g * p.M + m0) * p.N + chan;
            for (int n0 = 0; n0 < rows; n0 += 16) {
                float v[16];
                if (whole) {
                    uint32_t u[16];
                    tc::ld_32x16(acc + n0, u);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                    for (int c = parts.c0; c <= parts.c1; ++c) {
                        const float *from = part_of(c);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < rows) v[i] += __ldcg(from + (n0 + i) * kTileRows);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (n0 + i < rows && live) {
                        const __nv_bfloat16 o = __float2bfloat16_rn(
                            __fmul_rn(__fmul_rn(v[i], s_sx[n0 + i]), sw));
                        out[(size_t)(n0 + i) * p.N] = *reinterpret_cast<const uint16_t *>(&o);
                    }
                }
            }
            if (whole) {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_free[b]);
            }
            epi_sync();  // s_sx is free again
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && s_failed) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_WAIT_TIMEOUT);
    if (warp == kMmaWarp) tc::tmem_dealloc(taddr, kTmemCols);
}

}  // namespace

int gemm_int8_nmax(int M) {
    if (M <= 16) return 16;
    const int n = (M + 31) / 32 * 32;  // whole TMA boxes
    return n < kMaxCols ? n : kMaxCols;
}

cudaError_t launch_gemm_int8(GemmInt8Params p, int num_sms, cudaStream_t st) {
    if (p.G < 1 || p.G > kGemmInt8MaxGroups || p.M < 1 || p.N < 1 || p.H < 16 || p.H % 16 != 0)
        return cudaErrorInvalidValue;
    Ring ring;
    p.nmax = gemm_int8_nmax(p.M);
    ring.nmax = p.nmax;
    ring.box = p.nmax < 32 ? 16 : 32;
    const int raw = kWeightBytes + ring.nmax * kAtom, half = ring.nmax * kAtom;
    const int room = (int)kMaxDynamic - 1024;
    // at least two widened halves, then raw stages, then more halves
    ring.halves = ring.nmax > 128 ? 2 : 4;
    ring.stages = (room - ring.halves * half) / raw;
    if (ring.stages > kMaxStages) ring.stages = kMaxStages;
    if (ring.stages < 2) return cudaErrorInvalidValue;
    const size_t smem = 1024 + (size_t)ring.stages * raw + (size_t)ring.halves * half;
    CUtensorMap mx, mw;
    if (!make_map(&mx, p.xq, (long long)p.G * p.M, p.H, ring.box, true) ||
        !make_map(&mw, p.wq, (long long)p.G * p.N, p.H, kTileRows, true))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = raise_smem_limit_once(gemm_int8_kernel, kMaxDynamic, raised);
    if (err != cudaSuccess) return err;
    const int grid = num_sms < kStreamMaxCtas ? num_sms : kStreamMaxCtas;
    gemm_int8_kernel<<<grid, kThreads, smem, st>>>(mx, mw, p, ring);
    return cudaGetLastError();
}

}  // namespace moe
