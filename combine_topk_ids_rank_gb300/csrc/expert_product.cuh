// expert_product.cuh -- the persistent product of the experts' maps that
// gemm_fp8.cu and gemm_ragged.cu instantiate:
//   D[lane][column] = sum_k A[lane][k] * B[column][k],
// per group g, on the tensor cores (A is 128 tensor-memory lanes a CTA).
//
//   op          lanes              columns        k
//   kFp8        output channels    tokens         hidden size, 8-bit codes with block scales
//   kFp8Narrow  the same, for groups of few tokens
//   kForward    output channels    tokens         hidden size
//   kInputGrad  hidden size        tokens         output channels
//   kWeightGrad output channels    hidden size    tokens
//
// Groups are ragged along the tokens: the columns of the first three (a tile is
// as wide as its group needs, a multiple of 16, so that a group of few tokens
// costs its weights and little else), k of the last one.
//
// bf16: pairs of CTAs (cta_group::2), 256 lanes by up to 256 columns a tile.
// 8-bit: one CTA a tile, 128 lanes by up to 256 columns: its accumulators are
// read after every block of k, and two CTAs' meeting takes longer than that.  An
// accumulator's two halves of 128 columns are filled by an issuing warp each, read
// by four warps each and given back by themselves, so that no warp waits on a
// barrier whose phases it does not see one by one.
//
// Both operands come by TMA with the 128-byte swizzle, 128 bytes of k (or 64
// rows of k where k is not the innermost extent: MN-major tiles) a stage.
// Warps of a CTA:
//   0-7  epilogue: tensor-memory lanes 32 (w mod 4), half of the tile's columns;
//   8    producer; 8-bit: lists the CTA's tiles for the others as it goes;
//   9    (of CTA 0 of a pair) issues the products; 8-bit: of the first half;
//   10   8-bit: fetches the scales of tiles that are not turned; kWeightGrad:
//        clears what a last block of k holds of the next group's rows;
//   11   lists the pair's tiles, a few ahead (finding the next tile takes 1500 to
//        2000 cycles); 8-bit: issues the products of the second half.
// Sums.  The tensor cores add in fp32 with truncation (measured on bf16 normal
// values against 64 bits: 4.7e-7 of the result's norm after 512 products, 2.1e-6
// after 2048, 9.1e-6 after 8192; products of one sign lose 3.5e-5 after 8192 and 7.9e-4
// after 131072), so what is kept in 32 bits (kWeightGrad) leaves tensor memory every 512
// rows of k and is summed to nearest in registers, and what is rounded to bf16 at the
// end (kForward, kInputGrad) every 8192, where the loss is a hundredth of that rounding.
// The 8-bit product leaves it every 128 codes, where its scales change.  Two
// accumulators of 256 columns take turns meanwhile.
//
// Split.  Whole waves of tiles go round robin, those with the most work first.
// What is left over is cut by k: into equal ranges of the line of all blocks
// (tokens as columns), or each tile into equal parts (kWeightGrad).  The parts
// go through memory; the CTA that finishes last adds them in ascending k, so the
// order of the additions does not depend on timing.
//
// Bounds (device time of ten calls in a row; "stream": of thousands, which come to the power
// cap; operands of the calls of less than 20 us stand in L2, "cold": weights that do not).
//   kFp8, 8192 x 4096 x 7168: 195 us, 2460 TFLOP/s; stream 210.  The products alone take 154 us
//     (126 at the rate), with the epilogue's reads and meetings 182; its 256 additions a block
//     and SM sub-partition are the rest.  What holds the products themselves is not measured.
//     Pairs of CTAs: 337 us; reads in flight beside the additions: 197; each lane storing its
//     own row: 210.
//   kFp8, 32 planes of up to 1024 rows (12388 in all), 4096 x 2048: 125 us (57 at the memory's
//     rate): tiles of 16 blocks, 15% of their rows empty; lanes storing their own rows: 139.
//     (104, stream 107, with 9559 rows in all.)
//   kFp8Narrow, 16 x 7168 x 4096: 13.0 us, cold 13.8 (4.4): 2 us to the first load, the
//     chain along k, the last reads.  333 x 1000 x 1040: 9.6 us; with turned tiles 13.
//   kForward, 16384 rows of 32 groups, 4096 x 2048: one group 150 us (1840 TFLOP/s, the
//     power cap), even groups 162, uneven ones 186 (1480 TFLOP/s; 570 cycles a block where
//     the products need 420 on average: about 50 bytes a cycle and SM come from L2).
//     kInputGrad: 145, 171 and 183.  Prefetching weights into L2: 197.
//     Uneven ones in a stream: 202 and 203.
//   kForward, 8 rows of 128 groups, 1536 x 2048: 11.5 to 12 us, cold 14.0 (7.4).
//   kWeightGrad, the same 16384 rows: 162, 187 and 215 to 220 us, stream 226 to 235
//     (537 MB of output), fp32 278, added to fp32 448 (2.15 GB, 317 at the copy's
//     rate; each lane adding to its own row: 700):
//     even tiles have eight blocks at 0.87 of the dense rate; tiles of less than six wait
//     for the memory that takes their outputs.  Groups large and small in turn: 214 to 219.
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
#include "tiling.h"

#include "moe_a2a.h"

namespace moe {
namespace product {

using namespace stream;

constexpr int kEpiWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kHelpWarp = 10, kListWarp = 11;
constexpr int kThreads = 12 * 32;
// Registers: 384 threads start with 168 each (64512); the epilogue's 256 go to 200, the
// other 128 to 104, which is 64512 again.
constexpr int kStartRegs = 168, kEpiRegs = 200, kOtherRegs = 104;
static_assert(kEpiWarps * 32 * kEpiRegs + (kThreads - kEpiWarps * 32) * kOtherRegs <=
                  kThreads * kStartRegs, "more registers than the block starts with");
constexpr int kMaxCols = kProductMaxCols;
static_assert(kTileLanes == kTileRows && kTileCols == kMaxCols, "a tile's extents");
constexpr int kAccs = 2;                                  // accumulators of kMaxCols columns
constexpr int kStep = 16, kSteps = kMaxCols / 2 / kStep;  // columns an epilogue warp stores at once
constexpr int kLaneBytes = kTileRows * kAtom;             // A of a stage
constexpr int kPanelBytes = 64 * kAtom;                   // 64 lanes or columns by 64 rows of k
constexpr int kMaxStages = 12;
constexpr int kRowGroup = 8;                              // lane tiles of a raster group
constexpr int kBigBox = 64, kSmallBox = 8;                // rows of the token boxes
constexpr int kScaleSlots = 4, kScaleRun = 4;             // runs of 4 blocks' scales
constexpr int kSegs = 4;                                  // listed tiles
constexpr int kDynamic = 193 * 1024;                      // 227 KB less the static tables
constexpr int kBoxRows = 32, kBoxBytes = kBoxRows * kAtom;  // an output box of an epilogue warp
constexpr int kClasses = 64;
constexpr int kGradRun = 8;       // blocks of 64 rows of k that stay in tensor memory
constexpr int kRowRun = 128;      // (kForward, kInputGrad) blocks of 64 of k that do
// What a block of k takes at most, with much to spare (0.2 to 0.7 us): the limit of waits
// for whole tiles.
constexpr uint64_t kBlockNs = 4000;
constexpr int kMinPart = 4;       // blocks of k that make a part worth its way through memory
// kWeightGrad: a group's rows of up to this many bytes are fetched into L2 when its first
// tile is listed: all pairs come to a group at the same time, and then wait for memory.
// (Each CTA fetches its share of the grid, if it has a tile of the group: of a group with
// fewer tiles than pairs a part only.)
// (32 groups of 512 rows, 6 MB each: 187 us, 196 without; uneven groups up to 18 MB: 215 us,
// 216 without, 218 with those above 8 MB too.)
constexpr long long kAheadBytes = 8 << 20;
constexpr int kFp8Cols = 128;     // columns of an 8-bit tile that is not turned, at most

// Blocks [k0, k1) of k of a tile of a pair's (a CTA's) work: channel tile l, tokens
// (or the maps' columns) from c0 on.
struct Seg {
    int g, l, c0, cols, k0, k1;   // (g < 0: no more)
    int turned;                   // tokens are the lanes
    int whole, t;                 // the sum is whole; else t: the tile among the cut ones
    int p0, parts;                // (kWeightGrad)
};

// Turned tiles (kFp8).  A group with many tokens has them as the lanes, 128 a
// tile, and 256 channels as the columns: a lane then has one scale for a block and
// 128 columns, in a register, where tokens as columns need one read of shared
// memory for four products.
//
// Where no group has many tokens kFp8Narrow is launched: no turned tiles, and what
// the others take is fitted to narrow ones.
//
// The work of a call, in shared memory.  Tiles: groups in `order`; in a group,
// blocks of kRowGroup tiles along the channels (l), tile along the tokens (or the
// maps' columns) outer and l inner.  `waves` tiles of each pair are whole; the
// `rest` tiles behind them are cut.
template <Op OP>
struct Plan {
    static constexpr bool KRAGGED = OP == kWeightGrad;
    using Shape = product::Shape<OP>;

    int first[kProductMaxGroups + 1];   // tiles of the groups before, in this order
    int count[kProductMaxGroups];       // tokens of a group
    int start[kProductMaxGroups];       // its first row
    uint16_t order[kProductMaxGroups];
    uint16_t tally[kProductMaxGroups / 32][kClasses];  // groups of a class among 32 groups
    int base[kClasses];                 // groups of the classes above
    int sums[4], most_tokens;           // tiles by their widest form; the largest group
    int scan[kThreads / 32];
    Shape shape;
    int waves, rest, share, blocks;     // share: pairs for each of the rest (kWeightGrad)
    int parts, grain, q, more;          // the cut of the rest (tokens as columns)

    __device__ void tile(int t, const ProductParams &p, Seg &s) const {
        int lo = 0, hi = p.G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= t) lo = mid; else hi = mid - 1;
        }
        s.g = order[lo];
        const int c = KRAGGED ? p.cols : count[s.g], k = shape.mtiles(c), u = t - first[lo];
        s.turned = shape.turned(c);
        s.l = u;
        s.c0 = 0;
        s.cols = c;
        if (k > 1) {
            const int w = shape.stride(c), block = u / (kRowGroup * k);
            const int in = min(kRowGroup, shape.ltiles(c, p.lanes) - block * kRowGroup);
            const int v = u - block * kRowGroup * k;
            const int m = v / in;
            s.l = block * kRowGroup + v - m * in;
            s.c0 = m * w;
            s.cols = min(w, c - s.c0);
        }
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
template <Op OP>
struct Work {
    static constexpr bool KRAGGED = OP == kWeightGrad;
    const Plan<OP> &plan;
    int u, end;  // blocks of the cut tiles' line (kWeightGrad: end 0 once they are done)
    int wave;
    __device__ explicit Work(const Plan<OP> &plan_) : plan(plan_), u(0), end(1), wave(0) {
        if constexpr (!KRAGGED) {
            const Segments sg(plan.cut(), blockIdx.x / ctas_of(OP), plan.blocks);
            u = sg.u;
            end = sg.end;
        }
    }
    __device__ int blocks_of(int g) const {
        return KRAGGED ? (plan.count[g] + 63) / 64 : plan.blocks;
    }
    __device__ bool next(const ProductParams &p, Seg &s) {
        const int pair = blockIdx.x / ctas_of(OP), pairs = gridDim.x / ctas_of(OP);
        s.whole = 1;
        if constexpr (KRAGGED) {
            if (end != 0) {
                end = 0;
                const int share = plan.share, t = pair / share, part = pair - t * share;
                if (t < plan.rest) {
                    plan.tile(plan.waves * pairs + t, p, s);
                    const int b = blocks_of(s.g), n = min(share, max(1, b / kMinPart));
                    s.k0 = 0;
                    s.k1 = b;
                    if (n > 1 && part < n) {
                        s.k0 = (int)((long long)b * part / n);
                        s.k1 = (int)((long long)b * (part + 1) / n);
                        s.whole = 0;
                        s.p0 = t * share;
                        s.parts = n;
                    }
                    if (part < n) return true;
                }
            }
        } else if (u < end) {
            const int blocks = plan.blocks, t = u / blocks;
            plan.tile(plan.waves * pairs + t, p, s);
            s.k0 = u - t * blocks;
            s.k1 = min(s.k0 + end - u, blocks);
            u += s.k1 - s.k0;
            s.whole = s.k0 == 0 && s.k1 == blocks;
            s.t = t;
            return true;
        }
        if (wave >= plan.waves) {
            s.g = -1;
            return false;
        }
        plan.tile(wave * pairs + (wave & 1 ? pairs - 1 - pair : pair), p, s);
        ++wave;
        s.k0 = 0;
        s.k1 = blocks_of(s.g);
        return true;
    }
};

// The steps of kStep columns of a tile that one half of the epilogue's warps (and,
// in 8 bits, of an accumulator) takes.
constexpr int kHalfCols = kMaxCols / 2;
struct Half {
    int first, steps;
    // (grain: the first half has a multiple of so many steps, if there are as many)
    __device__ Half(bool turned, int cols, int h, int grain = 1) {
        const int all = (cols + kStep - 1) / kStep;
        if (grain > 1) {
            const int n = min(all, ((all + 1) / 2 + grain - 1) / grain * grain);
            first = h ? n : 0;
            steps = h ? all - n : n;
            return;
        }
        first = turned ? h * kSteps : (h ? (all + 1) / 2 : 0);
        steps = turned ? kSteps : (h ? all / 2 : (all + 1) / 2);
    }
};

// kFp8Narrow: blocks of k that half an accumulator holds side by side, 1 << shift of
// them (kFp8: one).  (A meeting of the issuer and the epilogue takes about 1000 cycles,
// whatever it is about.)
struct Sides {
    int shift;
    __device__ Sides(bool narrow, int cols) : shift(narrow ? (cols <= kMaxCols / 4 ? 2 : 1) : 0) {}
    __device__ bool first(int kb) const { return (kb & ((1 << shift) - 1)) == 0; }
    __device__ int next(int kb) const { return ((kb >> shift) + 1) << shift; }
    __device__ int col(int kb) const { return (kb & ((1 << shift) - 1)) * (kHalfCols >> shift); }
};

// Bytes that `cols` columns of a tile take of a CTA's stage.
template <Op OP>
__device__ __forceinline__ int col_bytes(int cols) {
    const int mine = cols / ctas_of(OP);
    return OP == kWeightGrad ? (mine + 63) / 64 * kPanelBytes : mine * kAtom;
}

// One more on a counter in memory: what this thread has seen written is released, and
// what others released there acquired.
__device__ __forceinline__ int count_up(int *p) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// 32 bytes of 16 neighbouring bf16 values or 8 fp32 values, 32-byte aligned.
__device__ __forceinline__ void store_256(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// This CTA's share of `bytes` bytes (a multiple of 16) from `p` on, into L2.
__device__ __forceinline__ void prefetch_share(const void *p, long long bytes) {
    const long long each = (bytes / gridDim.x + 127) / 128 * 128, at = each * blockIdx.x;
    if (at >= bytes) return;
    const uint32_t n = (uint32_t)(bytes - at < each ? bytes - at : each);
    const char *from = static_cast<const char *>(p) + at;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(n) : "memory");
}

template <Op OP>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_b8, const ProductParams p) {
    constexpr bool KRAGGED = OP == kWeightGrad;
    constexpr int kCtas = ctas_of(OP), kLanes = kCtas * kTileRows;
    constexpr bool PAIR = kCtas == 2;
    constexpr bool A_MN = OP == kInputGrad || OP == kWeightGrad, B_MN = OP == kWeightGrad;
    constexpr bool HELP = is_fp8(OP) || KRAGGED;
    constexpr int kBlock = is_fp8(OP) ? kAtom : kAtom / 2;  // extent of k in a stage
    constexpr int kScaleFloats = is_fp8(OP) ? kScaleSlots * kScaleRun * kFp8Cols : 4;
    // blocks of k whose products one accumulator takes
    constexpr int kRun = is_fp8(OP) ? 1 : (OP == kWeightGrad ? kGradRun : kRowRun);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) float s_scale[kScaleFloats];
    // (pairs.  full, acc_free: CTA 0's, both CTAs arrive; empty, acc_full: either's own)
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages];
    __shared__ uint64_t acc_full[kAccs][2], acc_free[kAccs][2];
    __shared__ uint64_t sc_full[kScaleSlots], sc_free[kScaleSlots];
    __shared__ uint64_t seg_full[kSegs], seg_free[kSegs], drained;
    __shared__ Seg segs[kSegs];
    __shared__ Plan<OP> plan;
    __shared__ uint32_t s_taddr;
    __shared__ volatile int s_failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = PAIR ? (int)ptx::cluster_rank() : 0;
    const uint32_t base = ptx::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (base & 1023u)) & 1023u);

    if (warp == kMmaWarp) {
        if (PAIR) tc::tmem_alloc_pair(&s_taddr, kAccs * kMaxCols);
        else tc::tmem_alloc(&s_taddr, kAccs * kMaxCols);
    }
    if (tid < kMaxStages) {
        ptx::mbar_init(&full[tid], KRAGGED ? kCtas : 1);
        ptx::mbar_init(&empty[tid], is_fp8(OP) ? 2 : 1);
        ptx::mbar_init(&tail[tid], 1);
        if (tid < kScaleSlots) {
            ptx::mbar_init(&sc_full[tid], 1);
            ptx::mbar_init(&sc_free[tid], kEpiWarps);
        }
        if (tid < kSegs) {  // read by the epilogue, the producer, the helper, the issuer
            ptx::mbar_init(&seg_full[tid], 1);
            ptx::mbar_init(&seg_free[tid], kEpiWarps + 1 + HELP + (rank == 0));
        }
        if (tid < kAccs) {
            for (int h = 0; h < 2; ++h) {
                ptx::mbar_init(&acc_full[tid][h], 1);
                ptx::mbar_init(&acc_free[tid][h], is_fp8(OP) ? kEpiWarps / 2 : kCtas * kEpiWarps);
            }
        }
        if (tid == 0) {
            ptx::mbar_init(&drained, is_fp8(OP) ? 2 : 1);
            s_failed = 0;
            plan.most_tokens = 0;
            for (int i = 0; i < 4; ++i) plan.sums[i] = 0;
        }
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
        if (!B_MN) tc::prefetch_map(&map_b8);
    }
    const int pairs = gridDim.x / kCtas, chunks = (p.G + 31) / 32;
    for (int i = tid; i < chunks * kClasses / 2; i += kThreads)
        reinterpret_cast<uint32_t *>(&plan.tally[0][0])[i] = 0;
    // (a turned tile's rows are stored 8 channels at a time)
    Shape<OP> shape;
    shape.turn_from = OP == kFp8 && p.lanes % 8 == 0 &&
                              reinterpret_cast<uintptr_t>(p.out) % 16 == 0
                          ? kProductTurnFrom : INT32_MAX;
    constexpr int kShift = is_fp8(OP) ? 7 : 8;
    static_assert(1 << kShift == (is_fp8(OP) ? kFp8Cols : kMaxCols), "columns of a tile");
    shape.shift = kShift;
    shape.even = !(KRAGGED && p.cols % 128 == 0);  // (every tile ends with a box)
    shape.thin = 0;
    __syncthreads();
    ptx::grid_dependency_wait();  // nothing of the caller's memory is touched before
    int sums[4] = {0, 0, 0, 0}, most = 0;
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
        plan.order[g] = (uint16_t)g;
        most = max(most, c);
        add_tiles(sums, shape, c, KRAGGED ? p.cols : c, p.lanes);
    }
    // (groups that this warp has none of leave the sums as they are)
    if (warp * 32 < p.G) {
        for (int i = 0; i < 4; ++i) {
            const int n = __reduce_add_sync(0xffffffffu, sums[i]);
            if (lane == 0) atomicAdd(&plan.sums[i], n);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) atomicMax(&plan.most_tokens, most);
    }
    tc::fence_before_sync();
    __syncthreads();
    // the pair's barriers are set up before either arrives on the other's
    if (PAIR) ptx::cluster_arrive();
    bool repeats = false;
    if (p.offsets != nullptr && could_repeat_too_many(shape, p.G, p.M, p.lanes)) {
        for (int g = tid; g < p.G; g += kThreads)
            repeats = repeats || __ldg(p.offsets + g + 1) < __ldg(p.offsets + g);
        repeats = __syncthreads_or(repeats);
    }
    const int tiles = settle(shape, plan.sums, repeats, pairs, p.lanes);
    // the widest tile decides how many stages the ring has
    const int blocks = KRAGGED ? 0 : (p.depth + kBlock - 1) / kBlock;
    int widest = max(16, KRAGGED ? shape.width(p.cols)
                                 : min(1 << shape.shift, (plan.most_tokens + 15) / 16 * 16));
    if (shape.turned(plan.most_tokens)) widest = kMaxCols;
    if (tid == kThreads - 1) {
        // Whole waves are dealt out as they are; the rest (and one wave more where the
        // rest is under a quarter of a wave) is cut.
        int waves = tiles / pairs, rest = tiles - waves * pairs;
        if (!KRAGGED && waves > 0 && rest != 0 && rest * 4 < pairs) --waves;
        rest = tiles - waves * pairs;
        plan.shape = shape;
        plan.waves = waves;
        plan.rest = rest;
        plan.blocks = blocks;
        if constexpr (KRAGGED) {
            plan.share = rest ? max(1, pairs / rest) : 1;
        } else {
            const Cut ct = widest <= 32 ? cut<true>(rest, blocks, pairs, 4 + widest / 16)
                                        : cut<false>(rest, blocks, pairs, 4 + widest / 16);
            plan.parts = ct.parts;
            plan.grain = ct.grain;
            plan.q = ct.q;
            plan.more = ct.more;
        }
    }
    // Groups by the work of a tile, stable: its columns, or (to a half power of two)
    // its blocks of k.  Where every pair has one tile at most the order is nothing.
    if (p.G > 1 && tiles > pairs) {
        const auto class_of = [&](int g) {
            if (!KRAGGED) return shape.width(plan.count[g]) / 16;
            const int b = (plan.count[g] + 63) / 64;
            if (b < 2) return b;
            const int e = 31 - __clz(b);
            return min(kClasses - 1, 2 * e + (b >> (e - 1) & 1));
        };
        // of 32 groups at a time (a warp's): those of a class, and the place among them
        constexpr int kTurns = (kProductMaxGroups / 32 + kThreads / 32 - 1) / (kThreads / 32);
        int cls[kTurns], place[kTurns];
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int chunk = warp + i * (kThreads / 32), g = chunk * 32 + lane;
            if (chunk >= chunks) break;
            cls[i] = g < p.G ? class_of(g) : kClasses;
            const unsigned same = __match_any_sync(0xffffffffu, cls[i]);
            place[i] = __popc(same & ((1u << lane) - 1u));
            if (place[i] == 0 && g < p.G) plan.tally[chunk][cls[i]] = (uint16_t)__popc(same);
        }
        __syncthreads();
        if (tid < kClasses) {
            int n = 0;
            for (int k = 0; k < chunks; ++k) {
                const int here = plan.tally[k][tid];
                plan.tally[k][tid] = (uint16_t)n;
                n += here;
            }
            plan.base[tid] = n;
        }
        __syncthreads();
        if (warp == 0) {  // the classes above: classes 63 - 2 lane and the next lower one
            const int hi = kClasses - 1 - 2 * lane, a = plan.base[hi], b = plan.base[hi - 1];
            int n = a + b;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o) n += v;
            }
            plan.base[hi] = n - a - b;
            plan.base[hi - 1] = n - b;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int chunk = warp + i * (kThreads / 32), g = chunk * 32 + lane;
            if (chunk < chunks && g < p.G)
                plan.order[plan.base[cls[i]] + plan.tally[chunk][cls[i]] + place[i]] = (uint16_t)g;
        }
        __syncthreads();
    }
    {  // exclusive prefix of the groups' tiles in this order
        const int each = (p.G + kThreads - 1) / kThreads, g0 = tid * each;
        const auto tiles_at = [&](int i) {
            return shape.tiles(KRAGGED ? p.cols : plan.count[plan.order[i]], p.lanes);
        };
        int n = 0;
        for (int i = g0; i < min(g0 + each, p.G); ++i) n += tiles_at(i);
        int sum = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) plan.scan[warp] = sum;
        sum -= n;
        if (p.G > 32 * each) {  // (else the first warp has all of them)
            __syncthreads();
            for (int w = 0; w < warp; ++w) sum += plan.scan[w];
        }
        for (int i = g0; i < min(g0 + each, p.G); ++i) {
            plan.first[i] = sum;
            sum += tiles_at(i);
        }
    }
    const uint32_t taddr = s_taddr;
    const int stage_bytes = kLaneBytes + col_bytes<OP>(widest);
    constexpr int boxes = KRAGGED ? kEpiWarps * kBoxBytes : 0;  // (at the end)
    const int stages = min(kMaxStages, (kDynamic - 1024 - boxes) / stage_bytes);
    auto a_of = [&](uint32_t s) { return smem + s * stage_bytes; };
    auto b_of = [&](uint32_t s) { return smem + s * stage_bytes + kLaneBytes; };
    __syncthreads();
    if (PAIR) ptx::cluster_wait();
    tc::fence_after_sync();
    // rows of k of a block (kWeightGrad: fewer than 64 in a group's last one)
    auto rows_of = [&](int g, int kb) { return KRAGGED ? min(64, plan.count[g] - kb * 64) : 64; };
    // A wait for as long as tiles take: for a free place in the list and for a tile that
    // comes to stand there, and the help warp's for a last block, since it passes over the
    // others.  (The other products' tiles of all of k end within kWaitNs: k of all groups
    // together has 32 bits, and fewer tiles than pairs are cut.)
    const uint64_t tiles_ns =
        kWaitNs + (KRAGGED ? (uint64_t)plan.most_tokens / 64 * kBlockNs * (kSegs + 1) : 0);
    const auto park_tiles = [&](uint64_t *bar, uint32_t parity) {
        return ptx::mbar_park(bar, parity, tiles_ns, &s_failed);
    };
    // the listed tiles in turn: waits for the next one, null behind the last (or on failure).
    // `far`: by a warp that may be ahead of the epilogue.
    const auto listed = [&](const Turn &sq, bool far) -> const Seg * {
        uint64_t *bar = &seg_full[sq.at];
        if (!(far ? park_tiles(bar, sq.parity) : ptx::mbar_park(bar, sq.parity, kWaitNs))) {
            s_failed = 1;
            return nullptr;
        }
        const Seg *s = &segs[sq.at];
        return s->g < 0 ? nullptr : s;
    };
    const auto arrive_first = [](uint64_t *bar) {  // on CTA 0's barrier
        if (PAIR) ptx::mbar_arrive_pair(ptx::cluster_smem(bar, 0));
        else mbar_arrive(bar);
    };

    // (setmaxnreg in the branch of its own roles: where two paths meet, the smaller
    // number holds)
    if (warp >= kEpiWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        Turn sq(kSegs);
        if (!is_fp8(OP) && warp == kListWarp) {
            if (ptx::elect_one()) {
                Work<OP> work(plan);
                int seen = -1;
                for (bool more = true; more && !s_failed; sq.next()) {
                    Seg s;
                    more = work.next(p, s);
                    if (KRAGGED && more && s.g != seen) {
                        seen = s.g;
                        const long long at = plan.start[s.g], n = plan.count[s.g];
                        const long long a = (long long)p.lanes * 2, b = (long long)p.cols * 2;
                        if (n * (a + b) <= kAheadBytes) {
                            prefetch_share(static_cast<const char *>(p.a) + at * a, n * a);
                            prefetch_share(static_cast<const char *>(p.b) + at * b, n * b);
                        }
                    }
                    if (!park_tiles(&seg_free[sq.at], sq.parity ^ 1u)) {
                        s_failed = 1;
                        break;
                    }
                    segs[sq.at] = s;
                    mbar_arrive(&seg_full[sq.at]);
                }
            }
        } else if (warp == kProducerWarp) {
            if (ptx::elect_one()) {
                Turn st(stages);
                uint32_t issued = 0, tails = 0, tail_parity = 0;
                const uint32_t full0 = PAIR ? ptx::cluster_smem(full, 0) : 0;
                Work<OP> work(plan);
                for (;;) {
                    const Seg *sp;
                    if (is_fp8(OP)) {  // lists the tiles itself (and alone writes the list)
                        Seg next;
                        next.g = -1;
                        const bool more = !s_failed && work.next(p, next);
                        if (!park_tiles(&seg_free[sq.at], sq.parity ^ 1u)) {
                            s_failed = 1;
                            break;
                        }
                        segs[sq.at] = next;
                        mbar_arrive(&seg_full[sq.at]);
                        sp = more ? &segs[sq.at] : nullptr;
                        sq.next();
                    } else {
                        sp = s_failed ? nullptr : listed(sq, true);
                    }
                    if (sp == nullptr) break;
                    const Seg sg = *sp;
                    if (!is_fp8(OP)) {
                        mbar_arrive(&seg_free[sq.at]);
                        sq.next();
                    }
                    // columns of this CTA; its first lane and column; the group's first row
                    const int half = (sg.cols + 15) / 16 * (16 / kCtas);
                    const bool thin = OP == kFp8Narrow && plan.shape.thin;
                    const int tall = OP == kFp8 && sg.turned ? kMaxCols : (thin ? 64 : kLanes);
                    const int a0 = sg.l * tall + rank * kTileRows;
                    const int at = plan.start[sg.g];
                    const int b0 = (KRAGGED ? 0 : at) + sg.c0 + rank * half;
                    int left = KRAGGED ? plan.count[sg.g] - sg.k0 * 64 : 64;  // rows of k
                    uint32_t bytes = kLaneBytes / (thin ? 2 : 1) + col_bytes<OP>(kCtas * half);
                    if (OP == kFp8 && sg.turned)  // boxes of 64 tokens, 256 channels
                        bytes = (sg.cols + 63) / 64 * kPanelBytes + 2 * kLaneBytes;
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int s = (int)st.at, k = kb * kBlock;
                        if (!ptx::mbar_park(&empty[s], st.parity ^ 1u, kWaitNs)) {
                            s_failed = 1;
                            break;
                        }
                        // A last block with rows of the next group lands on a barrier of this
                        // CTA; the helper clears those rows and arrives in the producer's place.
                        uint64_t *bar = &full[s];
                        uint32_t bar0 = full0 + 8 * s;
                        if (KRAGGED && left < 64) {
                            bar = &tail[s];
                            ptx::mbar_arrive_expect_tx(bar, bytes);
                            if (tails >> s & 1u) tail_parity ^= 1u << s;
                            tails |= 1u << s;
                            bar0 = ptx::cluster_smem(bar, rank);
                        } else if (rank == 0) {
                            ptx::mbar_arrive_expect_tx(bar, kCtas * bytes);
                            issued |= 1u << s;
                        } else if (KRAGGED) {
                            ptx::mbar_arrive_pair(bar0);
                        }
                        if (KRAGGED) left -= 64;
                        const auto load_2d = [&](uint8_t *to, const CUtensorMap *m, int x, int y) {
                            if (PAIR) tc::tma_load_2d_pair(to, m, x, y, bar0);
                            else tc::tma_load_2d(to, m, x, y, bar);
                        };
                        const auto load_3d = [&](uint8_t *to, const CUtensorMap *m, int x, int y) {
                            if (PAIR) tc::tma_load_3d_pair(to, m, x, y, sg.g, bar0);
                            else tc::tma_load_3d(to, m, x, y, sg.g, bar);
                        };
                        uint8_t *a = a_of(s), *b = b_of(s);
                        if (OP == kFp8 && sg.turned) {
                            for (int c = 0; c < sg.cols; c += kBigBox)
                                load_2d(a + c * kAtom, &map_b, k, b0 + c);
                            load_3d(b, &map_a, k, a0);
                            load_3d(b + kLaneBytes, &map_a, k, a0 + kTileRows);
                            continue;
                        }
                        if constexpr (OP == kFp8Narrow) {
                            load_3d(a, &map_a, k, a0);
                            if (!thin) load_3d(a + kPanelBytes, &map_a, k, a0 + 64);
                        } else if constexpr (OP == kFp8 || OP == kForward) {
                            load_3d(a, &map_a, k, a0);
                        } else if constexpr (OP == kInputGrad) {
                            load_3d(a, &map_a, a0, k);
                            load_3d(a + kPanelBytes, &map_a, a0 + 64, k);
                        } else {
                            load_2d(a, &map_a, a0, at + k);
                            load_2d(a + kPanelBytes, &map_a, a0 + 64, at + k);
                        }
                        if constexpr (B_MN) {
                            load_2d(b, &map_b, b0, at + k);
                            if (half > 64) load_2d(b + kPanelBytes, &map_b, b0 + 64, at + k);
                        } else {
                            int c = 0;
                            for (; c + kBigBox <= half; c += kBigBox)
                                load_2d(b + c * kAtom, &map_b, k, b0 + c);
                            for (; c < half; c += kSmallBox)
                                load_2d(b + c * kAtom, &map_b8, k, b0 + c);
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
        } else if (warp == kMmaWarp || (is_fp8(OP) && warp == kListWarp)) {
            if (rank == 0 && ptx::elect_one()) {
                const int h = warp == kMmaWarp ? 0 : 1;
                Turn st(stages), acc(kAccs);
                constexpr uint32_t kMajor =
                    (A_MN ? tc::kIdescMnA : 0u) | (B_MN ? tc::kIdescMnB : 0u);
                // a step along k: 32 bytes, or 16 rows, in descriptor units of 16 bytes
                constexpr uint64_t kStepA = A_MN ? 128 : 2, kStepB = B_MN ? 128 : 2;
                const uint32_t as = ptx::smem_u32(a_of(0)), bs = ptx::smem_u32(b_of(0));
                const uint64_t ad0 = A_MN ? tc::smem_desc_mn_sw128(as, kPanelBytes)
                                          : tc::smem_desc_sw128(as);
                const uint64_t bd0 = B_MN ? tc::smem_desc_mn_sw128(bs, kPanelBytes)
                                          : tc::smem_desc_sw128(bs);
                const auto wait_for = [&](uint64_t *bar, uint32_t parity) {
                    const bool ok = ptx::mbar_park(bar, parity, kWaitNs);
                    if (!ok) s_failed = 1;
                    tc::fence_after_sync();
                    return ok;
                };
                const auto commit = [](uint64_t *bar) {
                    if (PAIR) tc::commit_pair(bar);
                    else tc::commit(bar);
                };
                while (const Seg *sp = s_failed ? nullptr : listed(sq, true)) {
                    const Seg &sg = *sp;
                    const int k0 = sg.k0, k1 = sg.k1;
                    if constexpr (is_fp8(OP)) {
                        // An accumulator's halves are filled and given back by themselves;
                        // this issuer's has the tile's columns from 16 half.first on.
                        const Sides sides(OP == kFp8Narrow, sg.cols);
                        const Half half(OP == kFp8 && sg.turned, sg.cols, h);
                        const uint32_t idesc = tc::idesc_e4m3_f32(kLanes, half.steps * kStep);
                        const uint64_t bdh = bd0 + half.first * (kStep * kAtom / 16);
                        const bool some = half.steps > 0;
                        for (int kb = k0; kb < k1;) {
                            if (!wait_for(&full[st.at], st.parity)) break;
                            const uint32_t at = st.at * (uint32_t)(stage_bytes / 16);
                            if ((kb == k0 || sides.first(kb)) &&
                                !wait_for(&acc_free[acc.at][h], acc.parity ^ 1u))
                                break;
                            if (some) {
                                const uint32_t d = taddr + acc.at * kMaxCols + h * kHalfCols +
                                                   (OP == kFp8Narrow ? sides.col(kb) : 0);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc::mma_f8(d, ad0 + at + kk * kStepA, bdh + at + kk * kStepB,
                                               idesc, kk != 0);
                            }
                            ++kb;
                            if (kb == k1 || sides.first(kb)) {
                                commit(&acc_full[acc.at][h]);
                                acc.next();
                            }
                            commit(&empty[st.at]);
                            st.next();
                        }
                    } else {
                        const int n = (sg.cols + 15) / 16 * 16;
                        const uint32_t idesc = tc::idesc_bf16_f32(kLanes, n) | kMajor;
                        int left = KRAGGED ? plan.count[sg.g] - k0 * 64 : 64;  // rows of k
                        for (int kb = k0; kb < k1 && !s_failed;) {
                            const int from = kb, to = kRun < k1 - kb ? kb + kRun : k1;
                            const uint32_t d = taddr + acc.at * kMaxCols;
                            if (!wait_for(&full[st.at], st.parity)) break;
                            if (!wait_for(&acc_free[acc.at][0], acc.parity ^ 1u)) break;
                            for (; kb < to; ++kb, st.next()) {
                                if (kb != from && !wait_for(&full[st.at], st.parity)) break;
                                const uint32_t at = st.at * (uint32_t)(stage_bytes / 16);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    if (KRAGGED && kk != 0 && left <= 16 * kk) break;
                                    tc::mma_bf16_pair(d, ad0 + at + kk * kStepA,
                                                      bd0 + at + kk * kStepB, idesc,
                                                      kb != from || kk != 0);
                                }
                                if (KRAGGED) left -= 64;
                                commit(&empty[st.at]);
                            }
                            commit(&acc_full[acc.at][0]);
                            acc.next();
                        }
                    }
                    mbar_arrive(&seg_free[sq.at]);
                    sq.next();
                }
                commit(&drained);  // before tensor memory is freed
                ptx::mbar_park(&drained, 0, kWaitNs);
            }
        } else if (HELP && warp == kHelpWarp) {
            bool ok = true;
            Turn st(stages);          // (kWeightGrad)
            uint32_t parity = 0;
            Turn sc(kScaleSlots);     // (kFp8)
            while (ok) {
                const Seg *sp = listed(sq, true);
                if (__any_sync(0xffffffffu, sp == nullptr)) break;
                const Seg sg = *sp;
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_free[sq.at]);
                sq.next();
                if constexpr (is_fp8(OP)) {
                    // Products of the tokens' scales and the channels' of tiles that are not
                    // turned, four blocks of k (a run) at a time, for each column.
                    if (OP == kFp8 && sg.turned) continue;
                    const int KB = blocks, NB = (p.lanes + kScaleBlock - 1) / kScaleBlock;
                    const bool vec =
                        KB % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scale) % 16 == 0;
                    const int nb = OP == kFp8Narrow && plan.shape.thin ? sg.l / 2 : sg.l;
                    const float *sw = p.w_scale + ((size_t)sg.g * NB + nb) * KB;
                    const float *sx = p.x_scale + ((size_t)plan.start[sg.g] + sg.c0 + lane) * KB;
                    const int left = sg.cols - lane;  // tokens from this lane's first one on
                    for (int kb = sg.k0 & ~3; kb < sg.k1; kb += kScaleRun, sc.next()) {
                        float x[kFp8Cols / 32][kScaleRun], w[kScaleRun];
#pragma unroll
                        for (int j = 0; j < kFp8Cols / 32; ++j) {
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
                        for (int i = 0; i < kScaleRun; ++i)
                            w[i] = kb + i < KB ? __ldg(sw + kb + i) : 0.0f;
                        ok = __all_sync(0xffffffffu,
                                        ptx::mbar_park(&sc_free[sc.at], sc.parity ^ 1u, kWaitNs));
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        float *to = s_scale + sc.at * kScaleRun * kFp8Cols + lane;
#pragma unroll
                        for (int j = 0; j < kFp8Cols / 32; ++j)
#pragma unroll
                            for (int i = 0; i < kScaleRun; ++i)
                                to[i * kFp8Cols + 32 * j] = __fmul_rn(x[j][i], w[i]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_full[sc.at]);
                    }
                } else {
                    const int half = (sg.cols + 15) / 16 * 8, panels = 2 + (half + 63) / 64;
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int rows = rows_of(sg.g, kb);
                        if (rows == 64) continue;
                        ok = __all_sync(0xffffffffu,
                                        park_tiles(&tail[st.at], parity >> st.at & 1u));
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        parity ^= 1u << st.at;
                        // up to the end of the last step of 16 rows (B's panels follow A's)
                        const int chunks = ((rows + 15) / 16 * 16 - rows) * (kAtom / 16);
                        for (int i = lane; i < panels * chunks; i += 32) {
                            const int panel = i / chunks, c = i - panel * chunks;
                            uint8_t *at = a_of(st.at) + panel * kPanelBytes + rows * kAtom;
                            reinterpret_cast<uint4 *>(at)[c] = make_uint4(0, 0, 0, 0);
                        }
                        ptx::fence_proxy_async_smem();  // read next by the tensor cores
                        __syncwarp();
                        if (lane == 0) arrive_first(&full[st.at]);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // Each warp finishes 32 lanes by half of the tile's columns by itself.
        constexpr int kGrain = KRAGGED ? 4 : 1;  // (boxes of 64 columns)
        const int q = warp & 3, hf = warp >> 2, row = q * 32 + lane;
        Turn sq(kSegs), acc(kAccs), sc(kScaleSlots);
        const uint32_t mine = taddr + ((uint32_t)(q * 32) << 16);
        const uint32_t free0 = PAIR ? ptx::cluster_smem(&acc_free[0][0], 0) : 0;
        bool ok = true;
        const auto wait_for = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ptx::mbar_park(bar, parity, kWaitNs));
            if (!ok) s_failed = 1;
            return ok;
        };
        const auto release = [&] {  // the accumulator (8-bit: this half) has been read
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_pair(free0 + 16 * acc.at);
                else mbar_arrive(&acc_free[acc.at][hf]);
            }
            acc.next();
        };
        for (;;) {
            const Seg *const sp = listed(sq, false);
            if (__any_sync(0xffffffffu, sp == nullptr)) break;
            const Seg &sg = *sp;  // (stays there until the tile is stored)
            // this warp's steps of kStep columns of the tile, and the first one
            const auto steps_of = [&] {
                const int n = Half(OP == kFp8 && sg.turned, sg.cols, hf, kGrain).steps;
                if (OP == kFp8Narrow && plan.shape.thin && q >= 2) return 0;  // no lane
                if (OP != kFp8 || !sg.turned) return n;
                // channels that exist, if a token of the warp does
                const int chans = p.lanes - sg.l * kMaxCols - hf * kHalfCols;
                return q * 32 < sg.cols ? min(max((chans + kStep - 1) / kStep, 0), kSteps) : 0;
            };
            const auto first_of = [&] {
                return Half(OP == kFp8 && sg.turned, sg.cols, hf, kGrain).first * kStep;
            };
            // Sums to the columns from `to` on (16 a step).
            const auto keep = [&](uint32_t to, const auto &sum) {
                constexpr int S = sizeof sum / sizeof sum[0];
                const int steps = steps_of();
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    uint32_t v[kStep];
#pragma unroll
                    for (int j = 0; j < kStep; ++j) v[j] = __float_as_uint(sum[i][j]);
                    if (i < steps) tc::st_32x16(to + i * kStep, v);  // (no column more)
                }
                tc::wait_st();
            };
            const auto clear = [](auto &sum) {
#pragma unroll
                for (auto &step : sum)
#pragma unroll
                    for (float &v : step) v = 0.0f;
            };
            // What the sums (columns n0 + 16 i .. of this lane), kept in tensor memory, come
            // to.  (Held in registers here they do not leave enough for the rest.)
            const auto finish = [&](uint32_t from, bool none) {
                const int steps = steps_of(), n0 = first_of();
                const auto get = [&](int i, float (&v)[2][kStep]) {  // steps i and i + 1
                    uint32_t u[2][kStep];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < kStep; ++j) u[h][j] = 0;
                    if (!none) {
                        tc::ld_32x16(from + i * kStep, u[0]);
                        if (i + 1 < steps) tc::ld_32x16(from + (i + 1) * kStep, u[1]);
                        tc::wait_ld(u[0]);
                        tc::after_wait(u[1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < kStep; ++j) v[h][j] = __uint_as_float(u[h][j]);
                };
                // the lane's channel (not turned)
                const int chan = sg.l * (OP == kFp8Narrow && plan.shape.thin ? 64 : kLanes) +
                                 rank * kTileRows + row;
                const bool live = chan < p.lanes;
                uint16_t *const out16 = static_cast<uint16_t *>(p.out);
                // values 2 j and 2 j + 1
                const auto pack_bf16 = [](const float (&v)[kStep], int j) {
                    const __nv_bfloat162 o = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    return *reinterpret_cast<const uint32_t *>(&o);
                };
                // 16 neighbouring values of a row of `left` more, `left` a multiple of 8
                const bool whole32 = (KRAGGED ? p.cols : p.lanes) % 16 == 0 &&
                                     reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
                const auto store_row = [&](uint16_t *o, const float (&v)[kStep], int left) {
                    if (left <= 0) return;
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v, j);
                    if (whole32) {
                        store_256(o, w);
                    } else {
                        reinterpret_cast<uint4 *>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (left > 8)
                            reinterpret_cast<uint4 *>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                };
                // Where columns n of this lane go (n = 0: the tile's first), and how many are left.
                const size_t first = KRAGGED ? 0 : (size_t)plan.start[sg.g] + sg.c0;
                const int turned = OP == kFp8 && sg.turned, at0 = sg.l * kMaxCols;
                uint16_t *to16 = out16;
                size_t to = 0;
                int room = 0;
                if (turned) {  // a token's row
                    to16 += (first + row) * p.lanes + at0;
                    room = row < sg.cols ? p.lanes - at0 : 0;
                } else if (KRAGGED) {  // a row of the map's gradient
                    to = ((size_t)sg.g * p.lanes + chan) * p.cols + sg.c0;
                    room = live ? p.cols - sg.c0 : 0;
                } else {
                    to16 += (first + (lane & 1)) * p.lanes + (chan & ~1);
                    room = sg.cols - (lane & 1);
                }
                const bool words = p.lanes % 2 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
                // Columns n .. n + 15 (of the tile) of this lane.
                const auto store = [&](int n, const float (&v)[kStep]) {
                    const int left = room - n;
                    if (turned) {
                        store_row(to16 + n, v, left);
                    } else if constexpr (!KRAGGED) {
                        // Tokens as columns: two a word; neighbouring lanes exchange, so that the
                        // even lane stores both lanes' values of the first column and the odd
                        // lane those of the second.
                        const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
                        uint16_t *at = to16 + (size_t)n * p.lanes;
#pragma unroll
                        for (int j = 0; j < kStep / 2; ++j, at += 2 * (size_t)p.lanes) {
                            const uint32_t mine2 = pack_bf16(v, j);
                            const uint32_t both =
                                __byte_perm(mine2, __shfl_xor_sync(0xffffffffu, mine2, 1), pick);
                            if (words) {
                                if (live && 2 * j < left) *reinterpret_cast<uint32_t *>(at) = both;
                            } else if (2 * j < left) {  // rows may start off a word
                                if ((chan & ~1) < p.lanes) at[0] = (uint16_t)both;
                                if ((chan | 1) < p.lanes) at[1] = (uint16_t)(both >> 16);
                            }
                        }
                    } else if (!p.f32) {
                        store_row(out16 + to + n, v, left);
                    } else {
                        float *const o16 = static_cast<float *>(p.out) + to + n;
                        float4 old[kStep / 4];
#pragma unroll
                        for (int j = 0; j < kStep / 4; ++j)
                            old[j] = p.accumulate && 4 * j < left
                                         ? reinterpret_cast<const float4 *>(o16)[j]
                                         : make_float4(-0.0f, -0.0f, -0.0f, -0.0f);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (8 * h >= left) break;
                            float *o = o16 + 8 * h;
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                f[4 * j] = old[2 * h + j].x + v[8 * h + 4 * j];
                                f[4 * j + 1] = old[2 * h + j].y + v[8 * h + 4 * j + 1];
                                f[4 * j + 2] = old[2 * h + j].z + v[8 * h + 4 * j + 2];
                                f[4 * j + 3] = old[2 * h + j].w + v[8 * h + 4 * j + 3];
                            }
                            if (reinterpret_cast<uintptr_t>(p.out) % 32 == 0) {
                                uint32_t w[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[j]);
                                store_256(o, w);
                            } else {
                                float4 *o4 = reinterpret_cast<float4 *>(o);
                                o4[0] = make_float4(f[0], f[1], f[2], f[3]);
                                o4[1] = make_float4(f[4], f[5], f[6], f[7]);
                            }
                        }
                    }
                };
                // (adding nothing to what is there: left alone)
                if (KRAGGED && p.accumulate && none) return;
                int done = 0;  // steps
                if (KRAGGED && sg.whole) {
                    // Boxes of 32 rows by 128 bytes, through shared memory (128-byte swizzle),
                    // clipped at the map's last row by the tensor map; what is no whole box goes
                    // row by row.  (Added: in L2, once for every value, so the order of the CTAs
                    // changes nothing.  32 groups of 512 rows, 4096 x 2048, boxes and rows: bf16
                    // 203 and 214 us, fp32 287 and 340, added 442 and 649.)
                    uint8_t *box = smem + (kDynamic - 1024 - boxes) + warp * kBoxBytes;
                    const int y = sg.l * kLanes + rank * kTileRows + q * 32;
                    const int each = p.f32 ? 2 : 4;  // steps of a box
                    done = steps / each * each;
                    if (y < p.lanes)
#pragma unroll 1
                        for (int i = 0; i < done; i += each) {
                            if (lane == 0) ptx::bulk_wait_read<0>();  // (the box before)
                            __syncwarp();
#pragma unroll 1
                            for (int k = 0; k < each; k += 2) {
                                float v[2][kStep];
                                get(i + k, v);
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        uint4 w;
                                        int at = 4 * h + c;  // 16-byte chunk of the row
                                        if (p.f32) {
                                            w = make_uint4(__float_as_uint(v[h][4 * c]),
                                                           __float_as_uint(v[h][4 * c + 1]),
                                                           __float_as_uint(v[h][4 * c + 2]),
                                                           __float_as_uint(v[h][4 * c + 3]));
                                        } else {
                                            if (c >= 2) continue;
                                            at = 2 * (k + h) + c;
                                            w = make_uint4(pack_bf16(v[h], 4 * c),
                                                           pack_bf16(v[h], 4 * c + 1),
                                                           pack_bf16(v[h], 4 * c + 2),
                                                           pack_bf16(v[h], 4 * c + 3));
                                        }
                                        *reinterpret_cast<uint4 *>(box + lane * kAtom +
                                                                   ((at ^ (lane & 7)) << 4)) = w;
                                    }
                            }
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                const int x = sg.c0 + n0 + i * kStep;
                                if (p.accumulate) tc::tma_add_3d(&map_b8, x, y, sg.g, box);
                                else tc::tma_store_3d(&map_b8, x, y, sg.g, box);
                                ptx::bulk_commit();
                            }
                        }
                }
                if (sg.whole) {
#pragma unroll 1
                    for (int i = done; i < steps; i += 2) {
                        float v[2][kStep];
                        get(i, v);
                        store(n0 + i * kStep, v[0]);
                        if (i + 1 < steps) store(n0 + (i + 1) * kStep, v[1]);
                    }
                } else if (steps > 0) {
                    const int pair = blockIdx.x / kCtas;
                    // summed over `parts` pairs from p0 on; pair c keeps its part in slot 0
                    // unless it is p0
                    int p0 = sg.p0, parts = sg.parts, slot0 = 0;
                    if (!KRAGGED) {
                        const Parts pt(plan.cut(), sg.t, plan.blocks);
                        p0 = pt.c0;
                        parts = pt.count();
                        slot0 = pt.slot0;
                    }
                    auto part_of = [&](int c) {
                        const int slot = c == p0 ? slot0 : 0;
                        const size_t at = 2 * (kCtas * c + rank) + slot;
                        return p.part + at * p.nmax * kTileRows + row;
                    };
                    float *part = part_of(pair) + n0 * kTileRows;
#pragma unroll 1
                    for (int i = 0; i < steps; i += 2) {
                        float v[2][kStep];
                        get(i, v);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (i + h < steps)
#pragma unroll
                                for (int j = 0; j < kStep; ++j)
                                    __stcg(part + ((i + h) * kStep + j) * kTileRows, v[h][j]);
                    }
                    // the warp's parts, then lane 0's count, which releases them; and the other
                    // way round: what lane 0 finds counted (acquired), then the warp's reads
                    __syncwarp();
                    int last = 0;
                    if (lane == 0) {
                        int *m = &p.header->merged[hf][kCtas * p0 + rank][q];
                        last = count_up(m) == parts - 1;
                        if (last) *m = 0;  // for the next call
                    }
                    last = __shfl_sync(0xffffffffu, last, 0);
                    __syncwarp();
                    for (int i = 0; last && i < steps; ++i) {
                        const int n = n0 + i * kStep;
                        float v[kStep];
#pragma unroll
                        for (int j = 0; j < kStep; ++j) v[j] = 0.0f;
                        for (int c = p0; c < p0 + parts; ++c) {
                            const float *f = part_of(c) + (size_t)n * kTileRows;
#pragma unroll
                            for (int j = 0; j < kStep; ++j) v[j] += __ldcg(f + j * kTileRows);
                        }
                        store(n, v);
                    }
                }
            };
            if constexpr (is_fp8(OP)) {
                const auto scales = [&](int kb) {  // of block kb; a new run's once they are there
                    if (kb % kScaleRun == 0 || kb == sg.k0) wait_for(&sc_full[sc.at], sc.parity);
                    return s_scale + (sc.at * kScaleRun + kb % kScaleRun) * kFp8Cols;
                };
                const auto scales_read = [&](int kb) {
                    if (kb % kScaleRun == kScaleRun - 1 || kb + 1 == sg.k1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_free[sc.at]);
                        sc.next();
                    }
                };
                if (OP == kFp8 && sg.turned) {
                    // Four reads of 32 columns a block, the last of which is added when the
                    // accumulator's half has been given back.  (Reads in flight beside the
                    // additions gain nothing, or take registers that are not there: 197 to
                    // 294 us for 8192 x 4096 x 7168, by how; so 195 us.)
                    constexpr int kHeld = 32;
                    uint32_t u[kHeld];
                    float sum[kSteps][kStep];
                    clear(sum);
                    const auto add = [&](const uint32_t (&v)[kHeld], int at, float f) {
#pragma unroll
                        for (int j = 0; j < kHeld; j += 2) {
                            float *t = &sum[(at + j) / kStep][(at + j) % kStep];
                            const x2::f2 o = x2::fma(
                                x2::pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                x2::pack(f, f), x2::pack(t[0], t[1]));
                            x2::unpack(o, t[0], t[1]);
                        }
                    };
                    const int k0 = sg.k0, k1 = sg.k1;
                    // Scales of this lane's token, four blocks (a run) at a time, a run ahead.
                    const int KB = plan.blocks, NB = (p.lanes + kScaleBlock - 1) / kScaleBlock;
                    const bool there = row < sg.cols;
                    const bool vec =
                        KB % 4 == 0 && reinterpret_cast<uintptr_t>(p.x_scale) % 16 == 0;
                    const float *sx = p.x_scale + ((size_t)plan.start[sg.g] + sg.c0 + row) * KB;
                    const float *sw =
                        p.w_scale + ((size_t)sg.g * NB + min(2 * sg.l + hf, NB - 1)) * KB;
                    float4 x4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), f4 = x4;
                    const auto fetch = [&](int kb) {
                        if (!there) return;
                        if (vec) {
                            x4 = __ldg(reinterpret_cast<const float4 *>(sx + kb));
                        } else {
                            x4.x = __ldg(sx + kb);
                            if (kb + 1 < KB) x4.y = __ldg(sx + kb + 1);
                            if (kb + 2 < KB) x4.z = __ldg(sx + kb + 2);
                            if (kb + 3 < KB) x4.w = __ldg(sx + kb + 3);
                        }
                    };
                    fetch(k0 & ~3);
                    for (int kb = k0; kb < k1; ++kb) {
                        const int r = kb % kScaleRun;
                        if (r == 0 || kb == k0) {
                            const int b = kb - r;
                            f4.x = __fmul_rn(x4.x, __ldg(sw + b));
                            f4.y = __fmul_rn(x4.y, __ldg(sw + min(b + 1, KB - 1)));
                            f4.z = __fmul_rn(x4.z, __ldg(sw + min(b + 2, KB - 1)));
                            f4.w = __fmul_rn(x4.w, __ldg(sw + min(b + 3, KB - 1)));
                            if (b + kScaleRun < k1) fetch(b + kScaleRun);
                        }
                        const float f = r < 2 ? (r == 0 ? f4.x : f4.y) : (r == 2 ? f4.z : f4.w);
                        if (!wait_for(&acc_full[acc.at][hf], acc.parity)) break;
                        tc::fence_after_sync();
                        const uint32_t from = mine + acc.at * kMaxCols + hf * kHalfCols;
#pragma unroll
                        for (int i = 0; i < kHalfCols; i += kHeld) {
                            tc::ld_wait_32x32(from + i, u);
                            if (i + kHeld == kHalfCols && kb + 1 < k1) release();
                            add(u, i, f);
                        }
                    }
                    if (ok && sg.whole && p.lanes % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(p.out) % 32 == 0) {
                        release();
                        // Four lanes exchange 32-byte chunks, so that together they store 128
                        // bytes of one row after another.
                        const int t = lane & 3, c0 = sg.l * kMaxCols + hf * kHalfCols + t * kStep;
                        uint16_t *const o =
                            static_cast<uint16_t *>(p.out) +
                            ((size_t)plan.start[sg.g] + sg.c0 + (row & ~3)) * p.lanes + c0;
#pragma unroll
                        for (int i = 0; i < kSteps; i += 4) {
                            uint32_t w[4][8];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const __nv_bfloat162 two = __floats2bfloat162_rn(
                                        sum[i + c][2 * j], sum[i + c][2 * j + 1]);
                                    w[c][j] = *reinterpret_cast<const uint32_t *>(&two);
                                }
#pragma unroll
                            for (int b = 1; b < 4; b *= 2)
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    if (c & b) continue;
#pragma unroll
                                    for (int j = 0; j < 8; ++j) {
                                        const uint32_t give = t & b ? w[c][j] : w[c | b][j];
                                        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, b);
                                        if (t & b) w[c][j] = got;
                                        else w[c | b][j] = got;
                                    }
                                }
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c0 + i * kStep < p.lanes && (row & ~3) + c < sg.cols)
                                    store_256(o + (size_t)c * p.lanes + i * kStep, w[c]);
                        }
                    } else if (ok) {
                        const uint32_t at = mine + acc.at * kMaxCols + hf * kHalfCols;
                        keep(at, sum);
                        finish(at, false);
                        release();
                    }
                } else {
                    constexpr int kNarrow = kFp8Cols / 2 / kStep;  // steps, at most
                    const Sides sides(OP == kFp8Narrow, sg.cols);
                    const int steps = steps_of();
                    const int n0 = first_of(), k0 = sg.k0, k1 = sg.k1;
                    float sum[kNarrow][kStep];
                    clear(sum);
                    const auto add = [&](float (&t)[kStep], const uint32_t (&v)[kStep],
                                         const float *f) {
#pragma unroll
                        for (int j = 0; j < kStep; j += 4) {
                            const float4 f4 = *reinterpret_cast<const float4 *>(f + j);
                            t[j] = __fmaf_rn(__uint_as_float(v[j]), f4.x, t[j]);
                            t[j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), f4.y, t[j + 1]);
                            t[j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), f4.z, t[j + 2]);
                            t[j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), f4.w, t[j + 3]);
                        }
                    };
                    const uint32_t mine_half = mine + hf * kHalfCols;
                    for (int kb = k0; ok && kb < k1;) {
                        const int to = min(k1, sides.next(kb));
                        if (!wait_for(&acc_full[acc.at][hf], acc.parity)) break;
                        tc::fence_after_sync();
                        const uint32_t from = mine_half + acc.at * kMaxCols;
                        if (OP == kFp8Narrow && steps <= 1) {  // (four blocks) all at once
                            const float *f = scales(kb) - kb % 4 * kFp8Cols + n0;
                            uint32_t u[4][kStep];
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                tc::ld_32x16(from + r * (kHalfCols / 4), u[r]);
#pragma unroll
                            for (int r = 0; r < 4; ++r) tc::wait_ld(u[r]);
                            if (to < k1) release();
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (steps > 0 && r >= kb % 4 && r <= (to - 1) % 4)
                                    add(sum[0], u[r], f + r * kFp8Cols);
                            scales_read(to - 1);
                        } else {
                            for (int b = kb; ok && b < to; ++b) {
                                const float *f = scales(b) + n0;
                                const uint32_t at = from + sides.col(b);
                                uint32_t u[2][kStep];  // (the loads of the next step are in flight)
                                tc::ld_32x16(at, u[0]);
#pragma unroll
                                for (int i = 0; i < kNarrow; ++i) {
                                    if (i >= steps) break;
                                    tc::wait_ld(u[i & 1]);
                                    // (the last one once more: past it may be no column)
                                    const int next = min(i + 1, steps - 1);
                                    tc::ld_32x16(at + next * kStep, u[(i + 1) & 1]);
                                    add(sum[i], u[i & 1], f + i * kStep);
                                }
                                tc::wait_ld();  // the one that was not used
                                scales_read(b);
                            }
                            if (to < k1) release();
                        }
                        kb = to;
                    }
                    if (ok) {  // (kept where the last block was)
                        const uint32_t at = mine_half + acc.at * kMaxCols + sides.col(k1 - 1);
                        keep(at, sum);
                        finish(at, false);
                        release();
                    }
                }
            } else {
                const int steps = steps_of(), n0 = first_of(), k0 = sg.k0, k1 = sg.k1;
                if (k1 - k0 <= kRun) {  // all of k in one accumulator, or nothing
                    if (k0 < k1) wait_for(&acc_full[acc.at][0], acc.parity);
                    tc::fence_after_sync();
                } else {
                    float sum[kSteps][kStep];
                    clear(sum);
                    for (int kb = k0; kb < k1;) {
                        if (!wait_for(&acc_full[acc.at][0], acc.parity)) break;
                        tc::fence_after_sync();
                        const uint32_t from = mine + acc.at * kMaxCols + n0;
                        uint32_t u[2][kStep];  // (the loads of the next step are in flight)
                        tc::ld_32x16(from, u[0]);
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            if (i >= steps) break;
                            tc::wait_ld(u[i & 1]);
                            if (i + 1 < kSteps)
                                tc::ld_32x16(from + (i + 1) * kStep, u[(i + 1) & 1]);
#pragma unroll
                            for (int j = 0; j < kStep; ++j)
                                sum[i][j] = __fadd_rn(sum[i][j], __uint_as_float(u[i & 1][j]));
                        }
                        tc::wait_ld();  // the one that was not used
                        kb = kRun < k1 - kb ? kb + kRun : k1;
                        if (kb < k1) release();
                    }
                    if (ok) keep(mine + acc.at * kMaxCols + n0, sum);
                }
                if (ok) {
                    finish(mine + acc.at * kMaxCols + n0, k0 == k1);
                    if (k0 < k1) release();
                }
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_free[sq.at]);
            sq.next();
        }
    }

    if (KRAGGED && lane == 0) ptx::bulk_wait_all();  // output boxes on their way
    __syncwarp();
    if (warp == kMmaWarp && rank != 0)  // CTA 0's products read this CTA's memory too
        ptx::mbar_park(&drained, 0, kWaitNs);
    __syncwarp();
    tc::fence_before_sync();
    if (PAIR) ptx::cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    // the output may be an input that the next kernel reads before it waits for this
    // one: the CTA's stores (all of them are before the barrier) are visible first
    if (tid == 0) __threadfence();
    if (tid == 0 && s_failed) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_WAIT_TIMEOUT);
    if (warp == kMmaWarp) {
        if (PAIR) tc::tmem_dealloc_pair(taddr, kAccs * kMaxCols);
        else tc::tmem_dealloc(taddr, kAccs * kMaxCols);
    }
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
                   long long cols, int box_cols, int box_rows, bool bytes, bool f32 = false) {
    const long long ext[3] = {cols, rows, groups}, str[3] = {1, cols, rows * cols};
    const int box[3] = {box_cols, box_rows, 1};
    return make_map_nd(m, base, 3, ext, str, box, bytes, f32);
}

template <Op OP>
cudaError_t launch(const ProductParams &p, const CUtensorMap &a, const CUtensorMap &b,
                   const CUtensorMap &b8, int num_sms, cudaStream_t st) {
    constexpr int kCtas = ctas_of(OP);
    int grid = num_sms < kStreamMaxCtas ? num_sms : kStreamMaxCtas;
    grid -= grid % kCtas;
    if (grid < kCtas) return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> raised{0};
    const cudaError_t err = raise_smem_limit_once(product_kernel<OP>, (size_t)kDynamic, raised);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDynamic;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCtas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, product_kernel<OP>, a, b, b8, p);
}

}  // namespace product
}  // namespace moe
