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
// GB300 design (stream.cuh: weights are the A operand, tokens the columns):
// persistent pairs of CTAs, one CTA per SM.  A pair's tile is 256 channels
// (128 per CTA) by up to 256 tokens; each CTA widens its own weight rows and
// half of the token rows, and the pair's products (cta_group::2) read both
// halves, so a token row is widened once for 256 channels.  Whole waves of
// tiles go round robin; what is left over is cut by k.  In each CTA:
//   warps 0-3: epilogue (tensor-memory lane quadrants), 32 channels each;
//   warps 4-11: two groups widen a stage's 128 weight rows into tensor memory,
//     which the products read as their A operand;
//   warps 12-19: four groups widen the token rows into f16 tiles in shared
//     memory, half a k-block (64 codes) at a time;
//   warp 20: producer (TMA, 128-byte swizzle);
//   warp 21 of CTA 0: MMA issuer.
// Bounds.  8192 tokens x 4096 x 7168: 253 us, 1900 TFLOP/s (8-bit codes at the
// rate of a bf16 product), bound by the tensor cores.  One CTA a tile took 593
// us: it widens each token row twice as often.  16 tokens x 7168 x 4096: 15 us
// for 29 MB (4.4 us); bound by the widening of a unit (about 650 cycles) and
// the joining of cut tiles.  32 groups of up to 1024 rows, 4096 x 2048: 154 us,
// where 98 us of products would do (the tensor pipe is active 52 % of the time).  A
// tile of 256 columns has one accumulator, which is read between its products and the
// next tile's (two shorter ones gained 1 % at most), and a group of few rows waits for
// the widening of its weights; how the rest divides was not measured.  The ring is
// sized for the planes' places, not for what they hold: 32 planes with 4 to 32 rows
// each, 4096 x 2048, take 64 us in planes of 1024 places and 54 us in planes of 32.
#include "kernels.h"
#include "pair.cuh"
#include "ring.h"
#include "smem_limit_once.h"
#include "stream.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

#include "moe_a2a.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

using namespace stream;

constexpr int kWeightWarp0 = 4, kWeightGroups = 2;
constexpr int kTokenWarp0 = kWeightWarp0 + 4 * kWeightGroups, kTokenWarps = 8;
constexpr int kGroupWarps = 2, kGroups = kTokenWarps / kGroupWarps;
constexpr int kBatch = 4;                 // row blocks a token warp has in hand
constexpr int kProducerWarp = kTokenWarp0 + kTokenWarps, kMmaWarp = kProducerWarp + 1;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kPairRows = 2 * kTileRows;  // channels of a tile
constexpr int kMaxCols = 256;             // tokens of a tile
constexpr int kTmemCols = 512;            // accumulators, then widened weights
constexpr int kSlotCols = kBlockK / 2;    // a widened weight tile
constexpr int kMaxUnits = ring::kGemmMaxUnits;
constexpr int kWeightBytes = ring::kGemmWeightBytes;
constexpr int kMaxStages = ring::kGemmMaxStages;
static_assert(kWeightBytes == kTileRows * kBlockK && kAtom == ring::kGemmRowBytes, "a unit");
// Each widening warp takes every second unit (two groups of the halves a unit).
static_assert(kWeightGroups == ring::kTurns && kGroups == 2 * ring::kTurns, "every second unit");
constexpr int kRowGroup = 8;              // row tiles of a raster group
constexpr int kStepCols = 16;             // token columns an epilogue step takes
constexpr size_t kMaxDynamic = ring::kGemmDynamic;

// The tiles of a call: groups in turn, those with the widest tiles first; in a
// group, blocks of kRowGroup row tiles, token tile outer and row tile inner.
struct Tiles {
    const int *first;        // [G + 1] of the groups in this order
    const uint16_t *order;   // [G]
    const int *count;        // [G] token rows of a group
    int G, rtiles, nmax;
    __device__ int token_tiles(int c) const { return (c + nmax - 1) / nmax; }
    // token rows of a tile: evened out over the group's tiles, a multiple of 16
    __device__ int width(int c, int k) const {
        return (k == 1 ? c + 15 : (c + k - 1) / k + 15) / 16 * 16;
    }
    __device__ void of(int t, int &g, int &r, int &m0, int &rows) const {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= t) lo = mid; else hi = mid - 1;
        }
        g = order[lo];
        const int c = count[g], k = token_tiles(c), u = t - first[lo];
        if (k == 1) {
            m0 = 0;
            r = u;
            rows = c;
            return;
        }
        const int w = width(c, k), block = u / (kRowGroup * k);
        const int in = min(kRowGroup, rtiles - block * kRowGroup);
        const int v = u - block * kRowGroup * k;
        m0 = v / in;
        r = block * kRowGroup + v - m0 * in;
        m0 *= w;
        rows = min(w, c - m0);
    }
};

// The work of a pair in order: its parts of the cut tiles, which are the last
// ones, then a tile of each whole wave, to and fro, so that every pair gets
// its share of wide and narrow tiles.
struct Work {
    Segments segs;
    int wave, waves, pair, pairs, blocks;
    __device__ Work(const Cut &ct, int waves_, int blocks_, int pair_, int pairs_)
        : segs(ct, pair_, blocks_), wave(0), waves(waves_), pair(pair_), pairs(pairs_),
          blocks(blocks_) {}
    __device__ bool next(Segment &s) {
        if (segs.next(s)) {
            s.tile += waves * pairs;
            return true;
        }
        if (wave >= waves) return false;
        s.tile = wave * pairs + (wave & 1 ? pairs - 1 - pair : pair);
        s.k0 = 0;
        s.k1 = blocks;
        ++wave;
        return true;
    }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_int8_kernel(const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const GemmInt8Params p,
                     const ring::Gemm rings) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t raw_full[kMaxStages], raw_free[kMaxStages];
    // (full: CTA 0's, both CTAs arrive; free: either CTA's own)
    __shared__ uint64_t unit_full[kMaxUnits], unit_free[kMaxUnits];
    __shared__ uint64_t acc_full[2], acc_free[2], drained;
    __shared__ int s_first[kGemmInt8MaxGroups + 1], s_count[kGemmInt8MaxGroups];
    __shared__ uint16_t s_order[kGemmInt8MaxGroups];
    __shared__ int s_widths[kMaxCols / 16 + 1];
    __shared__ __align__(16) float s_sx[4][kMaxCols];  // the tile's token scales, a warp each
    __shared__ uint32_t s_taddr;
    __shared__ volatile int s_failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    const uint32_t base = ptx::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (base & 1023u)) & 1023u);
    const int half_bytes = rings.nmax / 2 * kAtom, raw_bytes = kWeightBytes + half_bytes;
    uint8_t *wide = smem + rings.stages * raw_bytes;  // raw_bytes: a multiple of 1024
    auto raw_w = [&](int s) { return smem + s * raw_bytes; };
    auto raw_x = [&](int s) { return smem + s * raw_bytes + kWeightBytes; };

    if (warp == kMmaWarp) tc::tmem_alloc_pair(&s_taddr, kTmemCols);
    if (tid < kMaxStages) {
        ptx::mbar_init(&raw_full[tid], 1);
        ptx::mbar_init(&raw_free[tid], 4 + 2 * kGroupWarps);
        if (tid < kMaxUnits) {
            ptx::mbar_init(&unit_full[tid], 2 * (4 + 2 * kGroupWarps));
            ptx::mbar_init(&unit_free[tid], 1);
        }
        if (tid < 2) {
            ptx::mbar_init(&acc_full[tid], 1);
            ptx::mbar_init(&acc_free[tid], 2 * 4);
        }
        if (tid == 0) {
            ptx::mbar_init(&drained, 1);
            s_failed = 0;
        }
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        tc::prefetch_map(&map_w);
        tc::prefetch_map(&map_x);
    }
    if (tid <= kMaxCols / 16) s_widths[tid] = 0;
    ptx::grid_dependency_wait();  // nothing of the caller's memory is touched before
    for (int g = tid; g < p.G; g += kThreads) {
        int c = p.M;
        if (p.counts != nullptr) c = min(max(__ldg(p.counts + g), 0), p.M);
        s_count[g] = c;
        if (p.G == 1) s_order[g] = 0;
    }
    tc::fence_before_sync();
    __syncthreads();
    // the pair's barriers are set up before either arrives on the other's
    ptx::cluster_arrive();
    const int rtiles = (p.N + kPairRows - 1) / kPairRows;
    const Tiles T{s_first, s_order, s_count, p.G, rtiles, rings.nmax};
    if (p.G > 1) {  // groups by the width of their tiles, stable
        const auto width = [&](int g) {
            const int c = s_count[g];
            return c > 0 ? T.width(c, T.token_tiles(c)) / 16 : 0;
        };
        for (int g = tid; g < p.G; g += kThreads) atomicAdd(&s_widths[width(g)], 1);
        __syncthreads();
        if (warp <= kMaxCols / 16) {
            const int mine = kMaxCols / 16 - warp;  // this warp's width
            int at = 0;
            for (int w = mine + 1; w <= kMaxCols / 16; ++w) at += s_widths[w];
            for (int g0 = 0; g0 < p.G; g0 += 32) {
                const bool hit = g0 + lane < p.G && width(g0 + lane) == mine;
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                if (hit) s_order[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(g0 + lane);
                at += __popc(m);
            }
        }
        __syncthreads();
    }
    if (warp == 0) {  // exclusive prefix of the groups' tiles
        int sum = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            const int n = g < p.G ? T.token_tiles(s_count[s_order[g]]) * rtiles : 0;
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
    int waves = tiles / pairs;
    const int rest = tiles - waves * pairs;
    if (waves > 0 && rest != 0 && rest * 4 < pairs) --waves;
    const int cut_tiles = tiles - waves * pairs;
    // (a merge costs about 4 units' time and 16 more for every 256 token columns)
    const Cut ct = rings.nmax <= 32 ? cut<true>(cut_tiles, blocks, pairs, 4 + rings.nmax / 16)
                                   : cut<false>(cut_tiles, blocks, pairs, 4 + rings.nmax / 16);
    const int nacc = 2 * rings.nmax <= kMaxCols ? 2 : 1;  // accumulators
    const uint32_t slots_at = taddr + kMaxCols;
    Work work(ct, waves, blocks, pair, pairs);
    Segment sg;
    ptx::cluster_wait();
    tc::fence_after_sync();

    // the widening warps' waits for a unit
    auto ready = [&](const Turn &st, const Turn &un) {
        return ring::widen_ready(
            [&] { return ptx::mbar_park(&unit_free[un.at], un.parity ^ 1u, kWaitNs); },
            [&] { return ptx::mbar_park(&raw_full[st.at], st.parity, kWaitNs); });
    };

    if (warp == kProducerWarp) {
        if (ptx::elect_one()) {
            Turn st(rings.stages);
            uint32_t issued = 0;  // stages in use
            while (!s_failed && work.next(sg)) {
                int g, r, m0, rows;
                T.of(sg.tile, g, r, m0, rows);
                const int half = (rows + 15) / 16 * 8;  // token rows of this CTA
                const int boxes = (half + rings.box - 1) / rings.box;
                const uint32_t bytes = kWeightBytes + boxes * rings.box * kAtom;
                const int w0 = r * kPairRows + rank * kTileRows, x0 = m0 + rank * half;
                for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                    const int s = (int)st.at;
                    if (!ptx::mbar_park(&raw_free[s], st.parity ^ 1u, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    issued |= 1u << s;
                    ptx::mbar_arrive_expect_tx(&raw_full[s], bytes);
                    tc::tma_load_3d(raw_w(s), &map_w, kb * kBlockK, w0, g, &raw_full[s]);
                    for (int b = 0; b < boxes; ++b)
                        tc::tma_load_3d(raw_x(s) + b * rings.box * kAtom, &map_x, kb * kBlockK,
                                        x0 + b * rings.box, g, &raw_full[s]);
                }
            }
            // copies still in flight land before shared memory goes away
            for (int i = 0; i < rings.stages; ++i, st.next()) {
                const uint32_t last = st.parity ^ 1u;
                if (issued >> st.at & 1u) ptx::mbar_park(&raw_full[st.at], last, kWaitNs);
            }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && ptx::elect_one()) {
            Turn un(rings.units), acc(nacc);
            const uint64_t bd0 = tc::smem_desc_sw128(ptx::smem_u32(wide));
            for (; !s_failed && work.next(sg); acc.next()) {
                int g, r, m0, rows;
                T.of(sg.tile, g, r, m0, rows);
                const uint32_t idesc = tc::idesc_f16_f32(kPairRows, (rows + 15) / 16 * 16);
                const uint32_t d = taddr + acc.at * rings.nmax;
                if (!ptx::mbar_park(&acc_free[acc.at], acc.parity ^ 1u, kWaitNs)) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                for (int kb = sg.k0; kb < sg.k1; ++kb, un.next()) {
                    const uint32_t a = slots_at + un.at * kSlotCols;
                    const uint64_t bd = bd0 + (uint64_t)(un.at * (half_bytes / 8));
                    if (!ptx::mbar_park(&unit_full[un.at], un.parity, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_f16_ta_pair(d, a + 8 * kk,
                                            bd + (kk >> 2) * (half_bytes / 16) + 2 * (kk & 3), idesc,
                                            kb != sg.k0 || kk != 0);
                    tc::commit_pair(&unit_free[un.at]);
                }
                tc::commit_pair(&acc_full[acc.at]);
            }
            tc::commit_pair(&drained);  // before tensor memory is freed
            ptx::mbar_park(&drained, 0, kWaitNs);
        }
    } else if (warp >= kWeightWarp0 && warp < kTokenWarp0) {
        // Thread l of a group of four warps owns weight row l of the CTA's half =
        // lane l; the groups take the units in turn.
        const int row = (tid - kWeightWarp0 * 32) & 127, group = (warp - kWeightWarp0) >> 2;
        Turn st(rings.stages), un(rings.units);
        bool ok = true;
        uint32_t n = 0;
        while (ok && !warp_flag(&s_failed) && work.next(sg)) {
            for (int kb = sg.k0; kb < sg.k1; ++kb, st.next(), un.next(), ++n) {
                if (n % kWeightGroups != (uint32_t)group) continue;
                ok = __all_sync(0xffffffffu, ready(st, un));
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                const uint8_t *src = raw_w(st.at) + row * kAtom;
                const uint32_t dst = slots_at + un.at * kSlotCols + ((uint32_t)(row & ~31) << 16);
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
                    mbar_arrive(&raw_free[st.at]);
                    ptx::mbar_arrive_pair(ptx::cluster_smem(&unit_full[un.at], 0));
                }
            }
        }
    } else if (warp >= kTokenWarp0 && warp < kTokenWarp0 + kTokenWarps) {
        // Groups of kGroupWarps warps take the halves in turn, so that one group's
        // loads, fence and arrival pass while the others compute.  The warps of a
        // group take blocks of 8 rows in turn, lane l the 16-code chunk l / 8 of row
        // l % 8: 8 consecutive lanes read (and write) 8 different 16-byte columns of
        // the swizzled rows, so no bank is hit twice.
        const int group = (warp - kTokenWarp0) / kGroupWarps, w = (warp - kTokenWarp0) % kGroupWarps;
        Turn st(rings.stages), un(rings.units);
        bool ok = true;
        uint32_t h = 0;
        while (ok && !warp_flag(&s_failed) && work.next(sg)) {
            int g, r, m0, rows;
            T.of(sg.tile, g, r, m0, rows);
            const int half = (rows + 15) / 16 * 8;
            for (int kb = sg.k0; kb < sg.k1 && ok; ++kb, st.next(), un.next()) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh, ++h) {
                    if (h % kGroups != (uint32_t)group) continue;
                    ok = __all_sync(0xffffffffu, ready(st, un));
                    if (!ok) {
                        s_failed = 1;
                        break;
                    }
                    const uint8_t *src = raw_x(st.at);
                    uint8_t *dst = wide + (2 * un.at + hh) * half_bytes;
                    const int c = lane >> 3, r8 = lane & 7, blocks8 = half >> 3;
                    // (row mod 8 is r8: the swizzle is the lane's own)
                    const uint8_t *from = src + r8 * kAtom + (((4 * hh + c) ^ r8) << 4);
                    uint8_t *to0 = dst + r8 * kAtom + (((2 * c) ^ r8) << 4);
                    uint8_t *to1 = dst + r8 * kAtom + (((2 * c + 1) ^ r8) << 4);
                    auto put = [&](int b, const uint4 &v) {
                        uint4 lo, hi;
                        int8_to_f16(v.x, lo.x, lo.y);
                        int8_to_f16(v.y, lo.z, lo.w);
                        int8_to_f16(v.z, hi.x, hi.y);
                        int8_to_f16(v.w, hi.z, hi.w);
                        *reinterpret_cast<uint4 *>(to0 + b * 8 * kAtom) = lo;
                        *reinterpret_cast<uint4 *>(to1 + b * 8 * kAtom) = hi;
                    };
                    auto get = [&](int b) {
                        return *reinterpret_cast<const uint4 *>(from + b * 8 * kAtom);
                    };
                    int b = w;
                    for (; b + (kBatch - 1) * kGroupWarps < blocks8; b += kBatch * kGroupWarps) {
                        uint4 v[kBatch];  // loads first
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) v[i] = get(b + i * kGroupWarps);
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) put(b + i * kGroupWarps, v[i]);
                    }
                    for (; b < blocks8; b += kGroupWarps) put(b, get(b));
                    ptx::fence_proxy_async_smem();  // read next by the tensor cores
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&raw_free[st.at]);
                        ptx::mbar_arrive_pair(ptx::cluster_smem(&unit_full[un.at], 0));
                    }
                }
            }
        }
    } else if (warp < 4) {
        // Each warp finishes 32 channels by itself.
        Turn acc(nacc);
        float *sx = s_sx[warp];
        for (; work.next(sg); acc.next()) {
            // what the tile needs is fetched while its products run
            int g, r, m0, rows;
            T.of(sg.tile, g, r, m0, rows);
            const int chan = r * kPairRows + rank * kTileRows + tid;
            const bool live = chan < p.N;
            const float sw = live ? __ldg(p.w_scale + (size_t)g * p.N + chan) : 0.0f;
            const float *xs = p.x_scale + (size_t)g * p.M + m0;
            __syncwarp();
            for (int i = lane; i < (rows + kStepCols - 1) / kStepCols * kStepCols; i += 32)
                sx[i] = i < rows ? __ldg(xs + i) : 0.0f;
            __syncwarp();
            const bool whole = sg.k0 == 0 && sg.k1 == blocks;
            Parts parts;
            if (!whole) parts = Parts(ct, sg.tile - waves * pairs, blocks);
            auto part_of = [&](int c) {
                return p.part + (size_t)(2 * (2 * c + rank) + parts.slot(c)) * p.nmax * kTileRows +
                       tid;
            };
            // the pair of channels that this lane stores; N even: both or neither exist
            uint16_t *out = p.out + ((size_t)g * p.M + m0) * p.N + (chan & ~1);
            const bool words = p.N % 2 == 0 && reinterpret_cast<uintptr_t>(p.out) % 4 == 0;
            // Columns n0 .. n0 + 15 of this lane's channel.  Two columns (tokens) a
            // word; neighbouring lanes (channels) exchange, so that the even lane
            // stores both channels of the first token and the odd lane both of the
            // second.
            const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
            auto store = [&](int n0, const float (&v)[kStepCols]) {
                uint16_t *at = out + (size_t)(n0 + (lane & 1)) * p.N;
                const int left = rows - n0 - (lane & 1);
#pragma unroll
                for (int i = 0; i < kStepCols; i += 2, at += 2 * (size_t)p.N) {
                    const float2 s2 = *reinterpret_cast<const float2 *>(&sx[n0 + i]);
                    const __nv_bfloat162 o =
                        __floats2bfloat162_rn(__fmul_rn(__fmul_rn(v[i], s2.x), sw),
                                              __fmul_rn(__fmul_rn(v[i + 1], s2.y), sw));
                    const uint32_t mine = *reinterpret_cast<const uint32_t *>(&o);
                    const uint32_t both =
                        __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
                    if (words) {
                        if (live && i < left) *reinterpret_cast<uint32_t *>(at) = both;
                    } else if (i < left) {  // odd N or address: rows start off a word
                        if ((chan & ~1) < p.N) at[0] = (uint16_t)both;
                        if ((chan | 1) < p.N) at[1] = (uint16_t)(both >> 16);
                    }
                }
            };
            bool ok = ptx::mbar_park(&acc_full[acc.at], acc.parity, kWaitNs) && !s_failed;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                s_failed = 1;
                break;
            }
            tc::fence_after_sync();
            const uint32_t from = taddr + acc.at * rings.nmax + ((uint32_t)(warp * 32) << 16);
            float *to = whole ? nullptr : part_of(pair);
            for (int n0 = 0; n0 < rows; n0 += kStepCols) {
                uint32_t u[kStepCols];
                float v[kStepCols];
                tc::ld_32x16(from + n0, u);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < kStepCols; ++i) v[i] = __uint_as_float(u[i]);
                if (whole) {
                    store(n0, v);
                } else {
#pragma unroll
                    for (int i = 0; i < kStepCols; ++i)
                        if (n0 + i < rows) __stcg(to + (n0 + i) * kTileRows, v[i]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_pair(ptx::cluster_smem(&acc_free[acc.at], 0));
            if (whole) continue;
            // the warp's parts, then lane 0's fence and count; and the other way round: what
            // lane 0 finds counted, its fence, then the warp's reads (a shuffle orders no memory)
            __syncwarp();
            __threadfence();
            int last = 0;
            if (lane == 0) {
                int *m = &p.header->merged[0][2 * parts.c0 + rank][warp];
                last = atomicAdd(m, 1) == parts.count() - 1;
                if (last) *m = 0;  // for the next call
                __threadfence();
            }
            if (!__shfl_sync(0xffffffffu, last, 0)) continue;
            __syncwarp();
            for (int n0 = 0; n0 < rows; n0 += kStepCols) {
                float v[kStepCols];
#pragma unroll
                for (int i = 0; i < kStepCols; ++i) v[i] = 0.0f;
                for (int c = parts.c0; c <= parts.c1; c += 2) {  // two parts in flight
                    const float *f = part_of(c) + (size_t)n0 * kTileRows;
                    const bool more = c < parts.c1;
                    const float *f2 = more ? part_of(c + 1) + (size_t)n0 * kTileRows : f;
                    float a[kStepCols], b[kStepCols];
#pragma unroll
                    for (int i = 0; i < kStepCols; ++i) {
                        const int at = n0 + i < rows ? i * kTileRows : 0;
                        a[i] = __ldcg(f + at);
                        b[i] = __ldcg(f2 + at);
                    }
#pragma unroll
                    for (int i = 0; i < kStepCols; ++i) {
                        v[i] += a[i];
                        if (more) v[i] += b[i];
                    }
                }
                store(n0, v);
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
    if (warp == kMmaWarp) tc::tmem_dealloc_pair(taddr, kTmemCols);
}

}  // namespace

int gemm_int8_nmax(int M) {
    int n = 16;  // a power of two: halves of whole TMA boxes
    while (n < M && n < kMaxCols) n *= 2;
    return n;
}

cudaError_t launch_gemm_int8(GemmInt8Params p, int num_sms, cudaStream_t st) {
    if (p.G < 1 || p.G > kGemmInt8MaxGroups || p.M < 1 || p.N < 1 || p.H < 16 || p.H % 16 != 0)
        return cudaErrorInvalidValue;
    int grid = num_sms < kStreamMaxCtas ? num_sms : kStreamMaxCtas;
    grid -= grid % 2;
    if (grid < 2) return cudaErrorInvalidValue;
    int nmax = gemm_int8_nmax(p.M);
    if (p.G == 1 && p.counts == nullptr) {
        // Narrower tiles while they still find an idle pair each: a narrow unit takes
        // 650 cycles and its tile's reading little, a 256-column one 1024 and 5000
        // (333 x 1000 x 1040: 11.3 us on 8 pairs, 9.3 us on 44).
        const long long rt = (p.N + kPairRows - 1) / kPairRows;
        while (nmax > 32 && (p.M + nmax / 2 - 1) / (nmax / 2) * rt <= grid / 2) nmax /= 2;
    }
    p.nmax = nmax;
    const ring::Gemm rings = ring::gemm(nmax);
    if (!ring::order_holds(rings.stages, rings.units)) return cudaErrorInvalidValue;
    const size_t smem = (size_t)ring::gemm_bytes(rings);
    CUtensorMap mx, mw;
    const long long H = p.H;
    const long long ext_x[3] = {H, p.M, p.G}, str_x[3] = {1, H, H * p.M};
    const long long ext_w[3] = {H, p.N, p.G}, str_w[3] = {1, H, H * p.N};
    const int box_x[3] = {kAtom, rings.box, 1}, box_w[3] = {kAtom, kTileRows, 1};
    if (!make_map_nd(&mx, p.xq, 3, ext_x, str_x, box_x, true) ||
        !make_map_nd(&mw, p.wq, 3, ext_w, str_w, box_w, true))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = raise_smem_limit_once(gemm_int8_kernel, kMaxDynamic, raised);
    if (err != cudaSuccess) return err;
    return launch_pdl(gemm_int8_kernel, dim3(grid), dim3(kThreads), smem, st, mx, mw, p, rings);
}

}  // namespace moe
