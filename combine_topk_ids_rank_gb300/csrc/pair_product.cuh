// pair_product.cuh -- the persistent product of the experts' maps that
// gemm_fp8.cu and gemm_ragged.cu instantiate:
//   D[lane][column] = sum_k A[lane][k] * B[column][k],
// per group g, on pairs of CTAs (cta_group::2): 256 lanes (128 a CTA) by up to
// 256 columns a tile, one CTA per SM.
//
//   op          lanes              columns        k
//   kFp8        output channels    tokens         hidden size, 8-bit codes with block scales
//   kForward    output channels    tokens         hidden size
//   kInputGrad  hidden size        tokens         output channels
//   kWeightGrad output channels    hidden size    tokens
//
// Groups are ragged along the tokens: the columns of the first three (a tile is
// as wide as its group needs, a multiple of 16, so that a group of few tokens
// costs its weights and little else), k of the last one.
//
// Both operands come by TMA with the 128-byte swizzle, 128 bytes of k (or 64
// rows of k where k is not the innermost extent: MN-major tiles) a stage.
// Warps of a CTA:
//   0-7  epilogue: tensor-memory lanes 32 (w mod 4), half of the tile's columns;
//   8    producer;
//   9    of CTA 0: issues the products of the pair;
//   10   kFp8: fetches the scales; kWeightGrad: clears what a last block of k
//        holds of the next group's rows;
//   11   none (registers are handed over by four warps at a time).
// Sums.  The tensor cores add in fp32 with truncation (measured on bf16 normal
// values against 64 bits: 4.7e-7 of the result's norm after 512 products, 2.1e-6
// after 2048, 9.1e-6 after 8192), so what is kept in 32 bits (kWeightGrad) leaves
// tensor memory every 512 rows of k and is summed to nearest in registers.  The
// 8-bit product leaves it every 128 codes, where its scales change.  The two
// accumulators of 256 columns take turns meanwhile.
//
// Split.  Whole waves of tiles go round robin, those with the most work first.
// What is left over is cut by k: into equal ranges of the line of all blocks
// (tokens as columns), or each tile into equal parts (kWeightGrad).  The parts
// go through memory; the CTA that finishes last adds them in ascending k, so the
// order of the additions does not depend on timing.
#pragma once

#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "product.h"
#include "smem_limit_once.h"
#include "stream.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

#include "moe_a2a.h"

namespace moe {
namespace product {

using namespace stream;

enum Op { kFp8, kForward, kInputGrad, kWeightGrad };

constexpr int kEpiWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kHelpWarp = 10;
constexpr int kThreads = 12 * 32;
// Registers: 384 threads start with 168 each (64512); the epilogue's 256 go to 208, the
// other 128 to 88, which is 64512 again.
constexpr int kStartRegs = 168, kEpiRegs = 208, kOtherRegs = 88;
static_assert(kEpiWarps * 32 * kEpiRegs + (kThreads - kEpiWarps * 32) * kOtherRegs <=
                  kThreads * kStartRegs, "more registers than the block starts with");
constexpr int kPairLanes = 2 * kTileRows;
constexpr int kMaxCols = kProductMaxCols;
constexpr int kStep = 16, kSteps = kMaxCols / 2 / kStep;  // columns an epilogue warp reads at once
constexpr int kLaneBytes = kTileRows * kAtom;             // A of a stage
constexpr int kPanelBytes = 64 * kAtom;                   // 64 lanes or columns by 64 rows of k
constexpr int kMaxStages = 12;
constexpr int kRowGroup = 8;                              // lane tiles of a raster group
constexpr int kBigBox = 64, kSmallBox = 8;                // rows of the token boxes
constexpr int kScaleSlots = 4, kScaleRun = 4;             // runs of 4 blocks' scales
constexpr int kDynamic = 193 * 1024;                      // 227 KB less the static tables
constexpr int kClasses = 64;
constexpr int kGradRun = 8;       // blocks of 64 rows of k that stay in tensor memory
constexpr int kMinPart = 4;       // blocks of k that make a part worth its way through memory

constexpr int tiles_of(int cols) { return (cols + kMaxCols - 1) / kMaxCols; }
// Columns of a tile: evened out over the group's tiles, a multiple of 16.
__device__ __forceinline__ int width_of(int cols) {
    const int k = tiles_of(cols);
    return k <= 1 ? (cols + 15) / 16 * 16 : ((cols + k - 1) / k + 15) / 16 * 16;
}

// Blocks [k0, k1) of k of a tile of a pair's work.  The tile is summed over
// `parts` pairs from p0 on; pair c keeps its part in slot 0 unless it is p0.
struct Seg {
    int g, l, c0, cols, k0, k1;
    bool turned;  // tokens are the lanes
    int p0, parts, slot0;
    __device__ bool whole() const { return parts == 1; }
    __device__ int slot(int c) const { return c == p0 ? slot0 : 0; }
};

// Turned tiles (kFp8).  A group with many tokens has them as the lanes and 256
// channels as the columns: a lane then has one scale for a block and 128 columns,
// in a register, where tokens as columns need one read of shared memory for four
// products.  (There are as many tiles either way.)
//
// The work of a call, in shared memory (the roles keep few registers of it).
// Tiles: groups in `order`; in a group, blocks of kRowGroup lane tiles, column
// tile outer and lane tile inner.  `waves` tiles of each pair are whole; the
// `rest` tiles behind them are cut.
struct Plan {
    int first[kProductMaxGroups + 1];   // tiles of the groups before, in this order
    int count[kProductMaxGroups];       // tokens of a group
    int start[kProductMaxGroups];       // its first row
    uint16_t order[kProductMaxGroups];
    int hist[kClasses];
    int turn_from;                      // tokens that make a group's tiles turned
    int waves, rest, share, blocks;     // share: pairs for each of the rest (kWeightGrad)
    int parts, grain, q, more;          // the cut of the rest (tokens as columns)

    // Columns of the tiles of a group of `c` tokens.
    __device__ int width(int c) const { return c >= turn_from ? kMaxCols : width_of(c); }

    template <bool KRAGGED>
    __device__ void tile(int t, const ProductParams &p, Seg &s) const {
        int lo = 0, hi = p.G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= t) lo = mid; else hi = mid - 1;
        }
        s.g = order[lo];
        const int ltiles = (p.lanes + kPairLanes - 1) / kPairLanes;
        const int c = KRAGGED ? p.cols : count[s.g], k = tiles_of(c), u = t - first[lo];
        const int w = KRAGGED ? width_of(c) : width(c), block = u / (kRowGroup * k);
        s.turned = !KRAGGED && c >= turn_from;
        const int in = min(kRowGroup, ltiles - block * kRowGroup);
        const int v = u - block * kRowGroup * k;
        const int m = v / in;
        s.l = block * kRowGroup + v - m * in;
        s.c0 = m * w;
        s.cols = min(w, c - s.c0);
    }
    __device__ Cut cut() const {
        Cut c(0, 0, grain);
        c.parts = parts;
        c.q = q;
        c.more = more;
        return c;
    }
};

// A pair's way through it: its parts of the cut tiles, which are the last ones,
// then a tile of each whole wave, to and fro.
template <bool KRAGGED>
struct Work {
    const Plan &plan;
    int u, end;  // blocks of the cut tiles' line (kWeightGrad: end 0 once they are done)
    int wave;
    __device__ explicit Work(const Plan &plan_) : plan(plan_), u(0), end(1), wave(0) {
        if constexpr (!KRAGGED) {
            const Segments sg(plan.cut(), blockIdx.x >> 1, plan.blocks);
            u = sg.u;
            end = sg.end;
        }
    }
    __device__ int blocks_of(int g) const {
        return KRAGGED ? (plan.count[g] + 63) / 64 : plan.blocks;
    }
    __device__ bool next(const ProductParams &p, Seg &s) {
        const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
        s.p0 = pair;
        s.parts = 1;
        s.slot0 = 0;
        if constexpr (KRAGGED) {
            if (end != 0) {
                end = 0;
                const int share = plan.share, t = pair / share, part = pair - t * share;
                if (t < plan.rest) {
                    plan.tile<KRAGGED>(plan.waves * pairs + t, p, s);
                    const int b = blocks_of(s.g), n = min(share, max(1, b / kMinPart));
                    if (part < n) {
                        s.k0 = (int)((long long)b * part / n);
                        s.k1 = (int)((long long)b * (part + 1) / n);
                        s.p0 = t * share;
                        s.parts = n;
                        return true;
                    }
                }
            }
        } else if (u < end) {
            const int blocks = plan.blocks, t = u / blocks;
            plan.tile<KRAGGED>(plan.waves * pairs + t, p, s);
            s.k0 = u - t * blocks;
            s.k1 = min(s.k0 + end - u, blocks);
            u += s.k1 - s.k0;
            if (s.k0 != 0 || s.k1 != blocks) {
                const Parts pt(plan.cut(), t, blocks);
                s.p0 = pt.c0;
                s.parts = pt.count();
                s.slot0 = pt.slot0;
            }
            return true;
        }
        if (wave >= plan.waves) return false;
        plan.tile<KRAGGED>(wave * pairs + (wave & 1 ? pairs - 1 - pair : pair), p, s);
        ++wave;
        s.k0 = 0;
        s.k1 = blocks_of(s.g);
        return true;
    }
};

// Where tiles of `width` columns put an operand's half of a stage.
template <Op OP>
__device__ __forceinline__ int half_bytes_of(int width) {
    return OP == kWeightGrad ? (width / 2 + 63) / 64 * kPanelBytes : width / 2 * kAtom;
}

template <Op OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_b8, const ProductParams p) {
    constexpr bool KRAGGED = OP == kWeightGrad;
    constexpr bool A_MN = OP == kInputGrad || OP == kWeightGrad, B_MN = OP == kWeightGrad;
    constexpr int kBlock = OP == kFp8 ? kAtom : kAtom / 2;  // extent of k in a stage
    constexpr int kScaleFloats = OP == kFp8 ? kScaleSlots * kScaleRun * kMaxCols : 4;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float s_scale[kScaleFloats];
    // (full, acc_free: CTA 0's, both CTAs arrive; empty, acc_full: either's own)
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages];
    __shared__ uint64_t acc_full[2], acc_free[2], sc_full[kScaleSlots], sc_free[kScaleSlots];
    __shared__ uint64_t drained;
    __shared__ Plan plan;
    __shared__ uint32_t s_taddr;
    __shared__ volatile int s_failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_rank(), pairs = gridDim.x >> 1;
    const uint32_t base = ptx::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (base & 1023u)) & 1023u);

    if (warp == kMmaWarp) tc::tmem_alloc_pair(&s_taddr, 2 * kMaxCols);
    if (tid < kMaxStages) {
        ptx::mbar_init(&full[tid], KRAGGED ? 2 : 1);
        ptx::mbar_init(&empty[tid], 1);
        ptx::mbar_init(&tail[tid], 1);
        if (tid < kScaleSlots) {
            ptx::mbar_init(&sc_full[tid], 1);
            ptx::mbar_init(&sc_free[tid], kEpiWarps);
        }
        if (tid < 2) {
            ptx::mbar_init(&acc_full[tid], 1);
            ptx::mbar_init(&acc_free[tid], 2 * kEpiWarps);
        }
        if (tid == 0) {
            ptx::mbar_init(&drained, 1);
            s_failed = 0;
        }
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
        if (!B_MN) tc::prefetch_map(&map_b8);
    }
    if (tid < kClasses) plan.hist[tid] = 0;
    // (a turned tile's rows are stored 8 channels at a time)
    if (tid == 0)
        plan.turn_from = OP == kFp8 && p.lanes % 8 == 0 &&
                                 reinterpret_cast<uintptr_t>(p.out) % 16 == 0
                             ? kProductTurnFrom : INT32_MAX;
    ptx::grid_dependency_wait();  // nothing of the caller's memory is touched before
    for (int g = tid; g < p.G; g += kThreads) {
        int at = 0, c = p.M;
        if (p.offsets != nullptr) {  // in bounds whatever they hold
            at = min(max(__ldg(p.offsets + g), 0), p.M);
            c = min(max(__ldg(p.offsets + g + 1), at), p.M) - at;
        } else {
            at = g * p.M;
            if (p.counts != nullptr) c = min(max(__ldg(p.counts + g), 0), p.M);
        }
        plan.start[g] = at;
        plan.count[g] = c;
        if (p.G == 1) plan.order[g] = 0;
    }
    tc::fence_before_sync();
    __syncthreads();
    // the pair's barriers are set up before either arrives on the other's
    ptx::cluster_arrive();
    const int ltiles = (p.lanes + kPairLanes - 1) / kPairLanes;
    // groups by the work of a tile, stable: its columns, or (to a half power of two)
    // its blocks of k
    const auto class_of = [&](int g) {
        if (!KRAGGED) return plan.width(plan.count[g]) / 16;
        const int b = (plan.count[g] + 63) / 64;
        if (b < 2) return b;
        const int e = 31 - __clz(b);
        return min(kClasses - 1, 2 * e + (b >> (e - 1) & 1));
    };
    if (p.G > 1) {
        for (int g = tid; g < p.G; g += kThreads) atomicAdd(&plan.hist[class_of(g)], 1);
        __syncthreads();
        for (int mine = warp; mine < kClasses; mine += kThreads / 32) {
            if (plan.hist[mine] == 0) continue;
            int at = 0;
            for (int w = mine + 1; w < kClasses; ++w) at += plan.hist[w];
            for (int g0 = 0; g0 < p.G; g0 += 32) {
                const bool hit = g0 + lane < p.G && class_of(g0 + lane) == mine;
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                if (hit) plan.order[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(g0 + lane);
                at += __popc(m);
            }
        }
        __syncthreads();
    }
    if (warp == 0) {  // exclusive prefix of the groups' tiles
        int sum = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            int n = 0;
            if (g < p.G) n = tiles_of(KRAGGED ? p.cols : plan.count[plan.order[g]]) * ltiles;
            int s = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            if (g < p.G) plan.first[g] = sum + s - n;
            sum += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) plan.first[p.G] = sum;
    }
    __syncthreads();

    const uint32_t taddr = s_taddr;
    const int tiles = plan.first[p.G], blocks = KRAGGED ? 0 : (p.depth + kBlock - 1) / kBlock;
    // the widest tile decides how many stages the ring has
    int widest = 16;
    if (KRAGGED) {
        widest = width_of(p.cols);
    } else if (p.G == 1) {
        widest = max(16, plan.width(plan.count[0]));
    } else {
        for (int w = 2; w <= kMaxCols / 16; ++w)
            if (plan.hist[w] != 0) widest = 16 * w;
    }
    const int half_bytes = half_bytes_of<OP>(widest), stage_bytes = kLaneBytes + half_bytes;
    const int stages = min(kMaxStages, (kDynamic - 1024) / stage_bytes);
    auto a_of = [&](uint32_t s) { return smem + s * stage_bytes; };
    auto b_of = [&](uint32_t s) { return smem + s * stage_bytes + kLaneBytes; };
    if (tid == 0) {
        // Whole waves are dealt out as they are; the rest (and one wave more where the
        // rest is under a quarter of a wave) is cut.
        int waves = tiles / pairs, rest = tiles - waves * pairs;
        if (!KRAGGED && waves > 0 && rest != 0 && rest * 4 < pairs) --waves;
        rest = tiles - waves * pairs;
        plan.waves = waves;
        plan.rest = rest;
        plan.share = rest ? max(1, pairs / rest) : 1;
        plan.blocks = blocks;
        if constexpr (!KRAGGED) {
            const Cut ct = widest <= 32 ? cut<true>(rest, blocks, pairs, 4 + widest / 16)
                                        : cut<false>(rest, blocks, pairs, 4 + widest / 16);
            plan.parts = ct.parts;
            plan.grain = ct.grain;
            plan.q = ct.q;
            plan.more = ct.more;
        }
    }
    __syncthreads();
    Work<KRAGGED> work(plan);
    Seg sg;
    ptx::cluster_wait();
    tc::fence_after_sync();
    // blocks of k whose products one accumulator takes
    constexpr int kRun = OP == kFp8 ? 1 : (OP == kWeightGrad ? kGradRun : INT32_MAX);
    // rows of k of a block (kWeightGrad: fewer than 64 in a group's last one)
    auto rows_of = [&](int g, int kb) { return KRAGGED ? min(64, plan.count[g] - kb * 64) : 64; };

    // (each in the branch of its own roles: where the two paths met, the smaller
    // number would hold)
    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kProducerWarp) {
            if (ptx::elect_one()) {
                Turn st(stages);
                uint32_t issued = 0, tails = 0, tail_parity = 0;
                while (!s_failed && work.next(p, sg)) {
                    const int half = (sg.cols + 15) / 16 * 8;  // columns of this CTA
                    const int a0 = sg.l * kPairLanes + rank * kTileRows, b0 = sg.c0 + rank * half;
                    const int at = plan.start[sg.g];
                    // bytes of this CTA and of the pair; turned: boxes of 64 tokens
                    uint32_t bytes = kLaneBytes + half_bytes_of<OP>(2 * half);
                    uint32_t both = 2 * bytes;
                    if (OP == kFp8 && sg.turned)
                        both = 2 * kLaneBytes + (sg.cols + 63) / 64 * kPanelBytes;
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int s = (int)st.at;
                        if (!ptx::mbar_park(&empty[s], st.parity ^ 1u, kWaitNs)) {
                            s_failed = 1;
                            break;
                        }
                        // A last block with rows of the next group lands on a barrier of this
                        // CTA; the helper clears those rows and arrives in the producer's place.
                        const bool last = KRAGGED && rows_of(sg.g, kb) < 64;
                        uint32_t bar = ptx::cluster_smem(&full[s], 0);
                        if (last) {
                            ptx::mbar_arrive_expect_tx(&tail[s], bytes);
                            if (tails >> s & 1u) tail_parity ^= 1u << s;
                            tails |= 1u << s;
                            bar = ptx::cluster_smem(&tail[s], rank);
                        } else if (rank == 0) {
                            ptx::mbar_arrive_expect_tx(&full[s], both);
                            issued |= 1u << s;
                        } else if (KRAGGED) {
                            ptx::mbar_arrive_pair(bar);
                        }
                        uint8_t *a = a_of(s), *b = b_of(s);
                        if (OP == kFp8 && sg.turned) {
                            for (int c = rank * kTileRows; c < sg.cols && c < (rank + 1) * kTileRows;
                                 c += kBigBox)
                                tc::tma_load_2d_pair(a + c % kTileRows * kAtom, &map_b, kb * kBlock,
                                                     at + sg.c0 + c, bar);
                            tc::tma_load_3d_pair(b, &map_a, kb * kBlock, a0, sg.g, bar);
                            continue;
                        }
                        if constexpr (OP == kFp8 || OP == kForward) {
                            tc::tma_load_3d_pair(a, &map_a, kb * kBlock, a0, sg.g, bar);
                        } else if constexpr (OP == kInputGrad) {
                            tc::tma_load_3d_pair(a, &map_a, a0, kb * 64, sg.g, bar);
                            tc::tma_load_3d_pair(a + kPanelBytes, &map_a, a0 + 64, kb * 64, sg.g,
                                                 bar);
                        } else {
                            tc::tma_load_2d_pair(a, &map_a, a0, at + kb * 64, bar);
                            tc::tma_load_2d_pair(a + kPanelBytes, &map_a, a0 + 64, at + kb * 64,
                                                 bar);
                        }
                        if constexpr (B_MN) {
                            for (int c = 0; c < half; c += 64)
                                tc::tma_load_2d_pair(b + c / 64 * kPanelBytes, &map_b, b0 + c,
                                                     at + kb * 64, bar);
                        } else {
                            int c = 0;
                            for (; c + kBigBox <= half; c += kBigBox)
                                tc::tma_load_2d_pair(b + c * kAtom, &map_b, kb * kBlock,
                                                     at + b0 + c, bar);
                            for (; c < half; c += kSmallBox)
                                tc::tma_load_2d_pair(b + c * kAtom, &map_b8, kb * kBlock,
                                                     at + b0 + c, bar);
                        }
                    }
                }
                // copies still in flight land before shared memory goes away (CTA 1's
                // complete on CTA 0's barriers, and the pair ends together)
                for (int i = 0; i < stages; ++i, st.next()) {
                    const uint32_t s = st.at, over = st.parity ^ 1u;
                    if (issued >> s & 1u) ptx::mbar_park(&full[s], over, kWaitNs);
                    if (tails >> s & 1u) ptx::mbar_park(&tail[s], tail_parity >> s & 1u, kWaitNs);
                }
            }
        } else if (warp == kMmaWarp) {
            if (rank == 0 && ptx::elect_one()) {
                Turn st(stages), acc(2);
                constexpr uint32_t kMajor =
                    (A_MN ? tc::kIdescMnA : 0u) | (B_MN ? tc::kIdescMnB : 0u);
                // a step along k: 32 bytes, or 16 rows, in descriptor units of 16 bytes
                constexpr uint64_t kStepA = A_MN ? 128 : 2, kStepB = B_MN ? 128 : 2;
                while (!s_failed && work.next(p, sg)) {
                    const int n = sg.turned ? kMaxCols : (sg.cols + 15) / 16 * 16;
                    const uint32_t idesc = (OP == kFp8 ? tc::idesc_e4m3_f32(kPairLanes, n)
                                                       : tc::idesc_bf16_f32(kPairLanes, n)) |
                                           kMajor;
                    for (int kb = sg.k0; kb < sg.k1 && !s_failed; acc.next()) {
                        const uint32_t d = taddr + acc.at * kMaxCols;
                        if (!ptx::mbar_park(&acc_free[acc.at], acc.parity ^ 1u, kWaitNs)) {
                            s_failed = 1;
                            break;
                        }
                        tc::fence_after_sync();
                        const int from = kb, to = kRun < sg.k1 - kb ? kb + kRun : sg.k1;
                        for (; kb < to; ++kb, st.next()) {
                            if (!ptx::mbar_park(&full[st.at], st.parity, kWaitNs)) {
                                s_failed = 1;
                                break;
                            }
                            tc::fence_after_sync();
                            const uint32_t as = ptx::smem_u32(a_of(st.at));
                            const uint32_t bs = ptx::smem_u32(b_of(st.at));
                            const uint64_t ad = A_MN ? tc::smem_desc_mn_sw128(as, kPanelBytes)
                                                     : tc::smem_desc_sw128(as);
                            const uint64_t bd = B_MN ? tc::smem_desc_mn_sw128(bs, kPanelBytes)
                                                     : tc::smem_desc_sw128(bs);
                            const int steps = (rows_of(sg.g, kb) + 15) / 16;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                if (KRAGGED && kk >= steps) break;
                                const bool add = kb != from || kk != 0;
                                const uint64_t ak = ad + kk * kStepA, bk = bd + kk * kStepB;
                                if (OP == kFp8) tc::mma_f8_pair(d, ak, bk, idesc, add);
                                else tc::mma_bf16_pair(d, ak, bk, idesc, add);
                            }
                            tc::commit_pair(&empty[st.at]);
                        }
                        tc::commit_pair(&acc_full[acc.at]);
                    }
                }
                tc::commit_pair(&drained);  // before tensor memory is freed
                ptx::mbar_park(&drained, 0, kWaitNs);
            }
        } else if (warp == kHelpWarp) {
            if constexpr (OP == kFp8) {
                // Products of the tokens' scales and the channels', four blocks of k
                // (a run) at a time: for each column, or, turned, for each lane and each
                // half of the columns.
                Turn sc(kScaleSlots);
                const int KB = blocks, NB = (p.lanes + kScaleBlock - 1) / kScaleBlock;
                const bool vec = KB % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scale) % 16 == 0;
                bool ok = true;
                while (ok && !warp_flag(&s_failed) && work.next(p, sg)) {
                    const int nb = 2 * sg.l + (sg.turned ? 0 : rank);
                    const float *sw = p.w_scale + ((size_t)sg.g * NB + min(nb, NB - 1)) * KB;
                    const float *sw1 = nb + 1 < NB ? sw + KB : sw;
                    const int first = sg.turned ? rank * kTileRows : 0;
                    const float *sx = p.x_scale +
                                      ((size_t)plan.start[sg.g] + sg.c0 + first + lane) * KB;
                    // tokens from this lane's first one on
                    const int left = min(sg.cols - first, sg.turned ? kTileRows : kMaxCols) - lane;
                    for (int kb = sg.k0 & ~3; kb < sg.k1; kb += kScaleRun, sc.next()) {
                        float x[kMaxCols / 32][kScaleRun], w[kScaleRun], w1[kScaleRun];
#pragma unroll
                        for (int j = 0; j < kMaxCols / 32; ++j) {
                            const float *from = sx + (size_t)(32 * j) * KB + kb;
#pragma unroll
                            for (int i = 0; i < kScaleRun; ++i) x[j][i] = 0.0f;
                            if (32 * j >= left) continue;
                            if (vec) {
                                const float4 f = __ldg(reinterpret_cast<const float4 *>(from));
                                x[j][0] = f.x, x[j][1] = f.y, x[j][2] = f.z, x[j][3] = f.w;
                            } else {
#pragma unroll
                                for (int i = 0; i < kScaleRun; ++i)
                                    if (kb + i < KB) x[j][i] = __ldg(from + i);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kScaleRun; ++i) {
                            w[i] = kb + i < KB ? __ldg(sw + kb + i) : 0.0f;
                            w1[i] = sg.turned && kb + i < KB ? __ldg(sw1 + kb + i) : 0.0f;
                        }
                        ok = __all_sync(0xffffffffu,
                                        ptx::mbar_park(&sc_free[sc.at], sc.parity ^ 1u, kWaitNs));
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        float *to = s_scale + sc.at * kScaleRun * kMaxCols + lane;
#pragma unroll
                        for (int j = 0; j < kMaxCols / 32; ++j) {
                            if (j < kTileRows / 32 || !sg.turned) {
#pragma unroll
                                for (int i = 0; i < kScaleRun; ++i)
                                    to[i * kMaxCols + 32 * j] = __fmul_rn(x[j][i], w[i]);
                            } else {
#pragma unroll
                                for (int i = 0; i < kScaleRun; ++i)
                                    to[i * kMaxCols + 32 * j] =
                                        __fmul_rn(x[j - kTileRows / 32][i], w1[i]);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_full[sc.at]);
                    }
                }
            } else if constexpr (KRAGGED) {
                Turn st(stages);
                uint32_t parity = 0;
                bool ok = true;
                while (ok && !warp_flag(&s_failed) && work.next(p, sg)) {
                    const int half = (sg.cols + 15) / 16 * 8, panels = 2 + (half + 63) / 64;
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int rows = rows_of(sg.g, kb);
                        if (rows == 64) continue;
                        ok = __all_sync(0xffffffffu, ptx::mbar_park(&tail[st.at],
                                                                    parity >> st.at & 1u, kWaitNs));
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        parity ^= 1u << st.at;
                        // up to the end of the last step of 16 rows (B's panels follow A's)
                        const int chunks = ((rows + 15) / 16 * 16 - rows) * (kAtom / 16);
                        for (int i = lane; i < panels * chunks; i += 32) {
                            const int panel = i / chunks, c = i - panel * chunks;
                            *reinterpret_cast<uint4 *>(a_of(st.at) + panel * kPanelBytes +
                                                       rows * kAtom + c * 16) = make_uint4(0, 0, 0, 0);
                        }
                        ptx::fence_proxy_async_smem();  // read next by the tensor cores
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_pair(ptx::cluster_smem(&full[st.at], 0));
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // Each warp finishes 32 lanes by half of the tile's columns by itself.
        const int q = warp & 3, hf = warp >> 2, row = q * 32 + lane;
        Turn acc(2), sc(kScaleSlots);
        bool ok = true;
        while (ok && work.next(p, sg)) {
            int s0, steps;  // this warp's steps of kStep columns of the tile
            if (OP == kFp8 && sg.turned) {  // channels that exist, if a token of the warp does
                s0 = hf * kSteps;
                const int chans = p.lanes - sg.l * kPairLanes - s0 * kStep;
                steps = rank * kTileRows + q * 32 < sg.cols
                            ? min(max((chans + kStep - 1) / kStep, 0), kSteps) : 0;
            } else {
                const int all = (sg.cols + kStep - 1) / kStep;
                s0 = hf ? (all + 1) / 2 : 0;
                steps = hf ? all / 2 : (all + 1) / 2;
            }
            const int n0 = s0 * kStep;
            x2::f2 sum[kSteps][kStep / 2];
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int j = 0; j < kStep / 2; ++j) sum[i][j] = 0ull;
            for (int kb = sg.k0; kb < sg.k1; acc.next()) {
                ok = ptx::mbar_park(&acc_full[acc.at], acc.parity, kWaitNs);
                const int run = kb % kScaleRun;
                if (OP == kFp8 && (run == 0 || kb == sg.k0))
                    ok = ok && ptx::mbar_park(&sc_full[sc.at], sc.parity, kWaitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t from = taddr + acc.at * kMaxCols + n0 + ((uint32_t)(q * 32) << 16);
                const float *scale = s_scale + (sc.at * kScaleRun + run) * kMaxCols;
                uint32_t u[2][kStep];
                const auto pair_of = [](const uint32_t *v) {
                    return x2::pack(__uint_as_float(v[0]), __uint_as_float(v[1]));
                };
                // (the loads of the next step are in flight)
                const auto read = [&](auto &&take) {
                    if (steps > 0) tc::ld_32x16(from, u[0]);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        if (i >= steps) break;
                        tc::wait_ld(u[i & 1]);
                        if (i + 1 < steps && i + 1 < kSteps)
                            tc::ld_32x16(from + (i + 1) * kStep, u[(i + 1) & 1]);
                        take(i, u[i & 1], sum[i]);
                    }
                };
                if constexpr (OP == kFp8) {
                    if (sg.turned) {
                        const float f = scale[hf * kTileRows + row];
                        const x2::f2 ff = x2::pack(f, f);
                        read([&](int, const uint32_t (&v)[kStep], x2::f2 (&t)[kStep / 2]) {
#pragma unroll
                            for (int j = 0; j < kStep / 2; ++j)
                                t[j] = x2::fma(pair_of(&v[2 * j]), ff, t[j]);
                        });
                    } else {
                        read([&](int i, const uint32_t (&v)[kStep], x2::f2 (&t)[kStep / 2]) {
                            const float4 *f = reinterpret_cast<const float4 *>(scale + n0 + i * kStep);
#pragma unroll
                            for (int j = 0; j < kStep / 4; ++j) {
                                const float4 f4 = f[j];
                                t[2 * j] = x2::fma(pair_of(&v[4 * j]), x2::pack(f4.x, f4.y), t[2 * j]);
                                t[2 * j + 1] = x2::fma(pair_of(&v[4 * j + 2]), x2::pack(f4.z, f4.w),
                                                       t[2 * j + 1]);
                            }
                        });
                    }
                } else {
                    read([&](int, const uint32_t (&v)[kStep], x2::f2 (&t)[kStep / 2]) {
#pragma unroll
                        for (int j = 0; j < kStep / 2; ++j)
                            t[j] = x2::add(t[j], pair_of(&v[2 * j]));
                    });
                }
                tc::fence_before_sync();
                __syncwarp();
                kb = kRun < sg.k1 - kb ? kb + kRun : sg.k1;
                if (lane == 0) {
                    ptx::mbar_arrive_pair(ptx::cluster_smem(&acc_free[acc.at], 0));
                    if (OP == kFp8 && (run == kScaleRun - 1 || kb == sg.k1))
                        mbar_arrive(&sc_free[sc.at]);
                }
                if (OP == kFp8 && (run == kScaleRun - 1 || kb == sg.k1)) sc.next();
            }
            if (!ok) break;
            if (steps == 0) continue;

            const int chan = sg.l * kPairLanes + rank * kTileRows + row;  // the lane's extent
            const bool live = chan < p.lanes;
            // Columns n .. n + 15 (of the tile) of this lane, tokens as columns: two
            // columns a word; neighbouring lanes exchange, so that the even lane stores
            // both lanes' values of the first column and the odd lane those of the second.
            uint16_t *const out16 = static_cast<uint16_t *>(p.out);
            const size_t tok0 = KRAGGED ? 0 : (size_t)plan.start[sg.g] + sg.c0;
            uint16_t *const out = out16 + tok0 * p.lanes + (chan & ~1);
            const bool words = p.lanes % 2 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
            const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
            auto pack_bf16 = [](x2::f2 v) {
                float a, b;
                x2::unpack(v, a, b);
                const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
                return *reinterpret_cast<const uint32_t *>(&o);
            };
            auto store = [&](int n, const x2::f2 (&v)[kStep / 2]) {
                if (OP == kFp8 && sg.turned) {  // a token's row, 8 channels at a time
                    const int tok = rank * kTileRows + row, at = sg.l * kPairLanes + n;
                    if (tok >= sg.cols) return;
                    uint16_t *o = out16 + (tok0 + tok) * p.lanes + at;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (at + 8 * h < p.lanes)
                            reinterpret_cast<uint4 *>(o)[h] =
                                make_uint4(pack_bf16(v[4 * h]), pack_bf16(v[4 * h + 1]),
                                           pack_bf16(v[4 * h + 2]), pack_bf16(v[4 * h + 3]));
                } else if constexpr (!KRAGGED) {
                    uint16_t *at = out + (size_t)(n + (lane & 1)) * p.lanes;
                    const int left = sg.cols - n - (lane & 1);
#pragma unroll
                    for (int j = 0; j < kStep / 2; ++j, at += 2 * (size_t)p.lanes) {
                        const uint32_t mine = pack_bf16(v[j]);
                        const uint32_t both =
                            __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
                        if (words) {
                            if (live && 2 * j < left) *reinterpret_cast<uint32_t *>(at) = both;
                        } else if (2 * j < left) {  // odd extent or address: rows start off a word
                            if ((chan & ~1) < p.lanes) at[0] = (uint16_t)both;
                            if ((chan | 1) < p.lanes) at[1] = (uint16_t)(both >> 16);
                        }
                    }
                } else if (live) {  // a row of the map's gradient, 8 columns at a time
                    const size_t at = ((size_t)sg.g * p.lanes + chan) * p.cols + sg.c0 + n;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (sg.c0 + n + 8 * h >= p.cols) break;
                        if (p.f32) {
                            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at +
                                                                   8 * h);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float4 f;
                                x2::unpack(v[4 * h + 2 * j], f.x, f.y);
                                x2::unpack(v[4 * h + 2 * j + 1], f.z, f.w);
                                if (p.accumulate) {
                                    const float4 old = o[j];
                                    f.x = old.x + f.x;
                                    f.y = old.y + f.y;
                                    f.z = old.z + f.z;
                                    f.w = old.w + f.w;
                                }
                                o[j] = f;
                            }
                        } else {
                            *reinterpret_cast<uint4 *>(out16 + at + 8 * h) =
                                make_uint4(pack_bf16(v[4 * h]), pack_bf16(v[4 * h + 1]),
                                           pack_bf16(v[4 * h + 2]), pack_bf16(v[4 * h + 3]));
                        }
                    }
                }
            };
            if (sg.whole()) {
                if (KRAGGED && p.accumulate && sg.k0 == sg.k1) continue;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    if (i >= steps) break;
                    store(n0 + i * kStep, sum[i]);
                }
                continue;
            }
            auto part_of = [&](int c) {
                return p.part + (size_t)(2 * (2 * c + rank) + sg.slot(c)) * p.nmax * kTileRows + row;
            };
            float *to = part_of(blockIdx.x >> 1) + n0 * kTileRows;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                if (i >= steps) break;
#pragma unroll
                for (int j = 0; j < kStep / 2; ++j) {
                    float a, b;
                    x2::unpack(sum[i][j], a, b);
                    __stcg(to + (i * kStep + 2 * j) * kTileRows, a);
                    __stcg(to + (i * kStep + 2 * j + 1) * kTileRows, b);
                }
            }
            // the warp's parts, then lane 0's fence and count; and the other way round: what
            // lane 0 finds counted, its fence, then the warp's reads (a shuffle orders no memory)
            __syncwarp();
            __threadfence();
            int last = 0;
            if (lane == 0) {
                int *m = &p.header->merged[hf][2 * sg.p0 + rank][q];
                last = atomicAdd(m, 1) == sg.parts - 1;
                if (last) *m = 0;  // for the next call
                __threadfence();
            }
            if (!__shfl_sync(0xffffffffu, last, 0)) continue;
            __syncwarp();
            for (int i = 0; i < steps; ++i) {
                const int n = n0 + i * kStep;
                float v[kStep];
#pragma unroll
                for (int j = 0; j < kStep; ++j) v[j] = 0.0f;
                for (int c = sg.p0; c < sg.p0 + sg.parts; ++c) {
                    const float *f = part_of(c) + (size_t)n * kTileRows;
#pragma unroll
                    for (int j = 0; j < kStep; ++j) v[j] += __ldcg(f + j * kTileRows);
                }
                x2::f2 o[kStep / 2];
#pragma unroll
                for (int j = 0; j < kStep / 2; ++j) o[j] = x2::pack(v[2 * j], v[2 * j + 1]);
                store(n, o);
            }
        }
    }

    __syncwarp();
    if (warp == kMmaWarp && rank != 0)  // CTA 0's products read this CTA's memory too
        ptx::mbar_park(&drained, 0, kWaitNs);
    __syncwarp();
    tc::fence_before_sync();
    ptx::cluster_sync();
    tc::fence_after_sync();
    // the output may be an input that the next kernel reads before it waits for this
    // one: the CTA's stores (all of them are before the barrier) are visible first
    if (tid == 0) __threadfence();
    if (tid == 0 && s_failed) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_WAIT_TIMEOUT);
    if (warp == kMmaWarp) tc::tmem_dealloc_pair(taddr, 2 * kMaxCols);
}

// Matrix of `rows` rows of `cols` values, boxes of box_cols x box_rows.
inline bool map_2d(CUtensorMap *m, const void *base, long long rows, long long cols, int box_cols,
                   int box_rows, bool bytes) {
    const long long ext[2] = {cols, rows}, str[2] = {1, cols};
    const int box[2] = {box_cols, box_rows};
    return make_map_nd(m, base, 2, ext, str, box, bytes);
}

// `groups` matrices one after another.
inline bool map_3d(CUtensorMap *m, const void *base, long long groups, long long rows,
                   long long cols, int box_cols, int box_rows, bool bytes) {
    const long long ext[3] = {cols, rows, groups}, str[3] = {1, cols, rows * cols};
    const int box[3] = {box_cols, box_rows, 1};
    return make_map_nd(m, base, 3, ext, str, box, bytes);
}

template <Op OP>
cudaError_t launch(const ProductParams &p, const CUtensorMap &a, const CUtensorMap &b,
                   const CUtensorMap &b8, int num_sms, cudaStream_t st) {
    int grid = num_sms < kStreamMaxCtas ? num_sms : kStreamMaxCtas;
    grid -= grid % 2;
    if (grid < 2) return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> raised{0};
    const cudaError_t err = raise_smem_limit_once(product_kernel<OP>, (size_t)kDynamic, raised);
    if (err != cudaSuccess) return err;
    return launch_pdl(product_kernel<OP>, dim3(grid), dim3(kThreads), (size_t)kDynamic, st, a, b,
                      b8, p);
}

}  // namespace product
}  // namespace moe
