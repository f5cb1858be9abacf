// layer_small.cu -- a whole mixture-of-experts layer for a few tokens in one
// kernel: no receive planes, no intermediate launch.
//
// Operation, token t with experts e_k = topk_ids[t][k] and gates g_k:
//   h     = W13[e] x_t                       (rows 0..I-1 gate, I..2I-1 up),
//   a     = silu(h_gate * s13) * (h_up * s13),  silu(z) = z / (1 + e^-z),
//   y     = (W2[e] a) * s2,
//   out_t = bf16_rn( sum over k ascending of g_k * y_k  (+ residual_t) ),
// products accumulated in fp32 on the tensor cores, y and the sum in fp32;
// s13, s2 are the channels' scales of the 8-bit formats.  An expert named
// twice by a token counts once, with the sum of its gates.  Id -1 (and an
// id outside [-1, E), which raises the flag) is no expert.
//
// The tensor cores take the activations in bf16 beside the weights.  They are
// handed over as two of them, bf16_rn(a) and bf16_rn of what is left, which
// keeps 16 significant bits: with few tokens the second product on the same
// weight tile costs nothing beside reading the tile, and the output's own
// narrowing stays the only rounding that shows (1.4 times its error without).
//
// GB300 design: every weight row of the experts in use is read once, and
// nothing else is large, so the kernel is a stream of weight tiles at HBM's
// rate (stream.cuh: weights are the A operand, 128 channels a tile; the
// tokens are the columns).  One CTA per SM, launched cooperatively; two
// phases (W13, then W2) share one ring of shared-memory stages that runs on
// across them, so the first W2 tiles arrive while the last activations are
// still being made.  Every CTA builds the expert lists from the ids itself.
//   warps 0-3: epilogue (tensor-memory lane quadrants);
//   warp 4: weight producer (TMA, 128-byte swizzle);
//   warp 5: tensor-memory owner and MMA issuer;
//   warps 6-7: token rows into the stages, unit by unit in turn (16-byte
//     cp.async, swizzled alike);
//   warps 8-15, 8-bit formats: two groups of four in turn widen a stage's
//     weight rows to bf16 into tensor memory (exact), which the products read
//     as their A operand.
// Bounds.  8 tokens, hidden 7168, inter 2048, 64 experts, top-8, int8: 286-306
// us for 1.85 GB, 89-95 % of the copy rate; 64 tokens, hidden 2048, inter 1024,
// bf16: 142 us for 0.81 GB (118 us).  One token, hidden 2048, inter 768: 23 us
// for 75 MB (11 us); 5 us are the launch, the lists and the last exchange, and
// about 6 the way through the two phases (first weights, activations visible to
// all CTAs, outputs visible to all).
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

constexpr int kEpiThreads = 128;
constexpr int kCols = 8;        // token columns an epilogue step takes
constexpr int kProducerWarp = 4, kMmaWarp = 5, kLoaderWarp0 = 6;
// Loader warps that take the units in turn.  No more than a ring has stages: a warp
// knows of its last unit that all before the ring's length are free, and a wait by
// parity may be at most one phase ahead of that.
constexpr int kLoaders = 2;
static_assert(kLoaders <= ring::kLayerMinStages, "parity waits would run ahead");
constexpr int kConvertWarp0 = (kLoaderWarp0 + kLoaders + 3) / 4 * 4;  // warp mod 4: lane quadrant
constexpr int kHalfRows = 64;   // gate rows (and up rows) of a W13 tile
constexpr int kQuarter = 16;    // of them in a warp's 32 lanes: 16 gate rows, then 16 up rows
constexpr int kSlots = ring::kLayerSlots;  // widened weight tiles in tensor memory
constexpr int kSlotCols = kBlockK / 2;
constexpr int kAccCols = 2 * kLayerMaxTokens;  // of an accumulator: both terms' columns
constexpr int kMaxStages = ring::kLayerMaxStages;
constexpr size_t kMaxDynamic = ring::kLayerDynamic;

// The lists at the front of dynamic shared memory, for E experts and P pairs
// (token, k).
struct Lists {
    int16_t *kept;     // [P] expert of (t, k), -1 where dropped; 16-byte aligned, whole 16 bytes
    float *gate;       // [P] gate of (t, k)
    int *count;        // [E] kept pairs of an expert
    uint16_t *first;   // [E] first pair of an expert in use
    uint16_t *expert;  // [A] experts in use, ascending (A <= min(E, P))
    uint16_t *base;    // [A + 1] their first pairs
    uint16_t *token;   // [P] token of a pair
    int16_t *place;    // [P] pair of (t, k), -1 where dropped
    __device__ Lists(uint8_t *mem, int E, int P) {
        const int A = E < P ? E : P;
        kept = reinterpret_cast<int16_t *>(mem);
        gate = reinterpret_cast<float *>(kept + (P + 7) / 8 * 8);
        count = reinterpret_cast<int *>(gate + P);
        first = reinterpret_cast<uint16_t *>(count + E);
        expert = first + E;
        base = expert + A;
        token = base + A + 1;
        place = reinterpret_cast<int16_t *>(token + P);
    }
};

template <int FORMAT>
struct Shape {
    static constexpr bool kWiden = FORMAT != MOE_FORMAT_BF16;
    static constexpr int kThreads = (kWiden ? kConvertWarp0 + 8 : kLoaderWarp0 + kLoaders) * 32;
    static constexpr int kValue = kWiden ? 1 : 2;                     // bytes of a weight
    static constexpr int kA = kTileRows * kBlockK * kValue;           // weight bytes a stage
    static constexpr int kTmem = kWiden ? 512 : 256;                   // tensor-memory columns
};

template <int FORMAT>
__global__ void __launch_bounds__(Shape<FORMAT>::kThreads, 1)
    layer_small_kernel(const __grid_constant__ CUtensorMap map13,
                       const __grid_constant__ CUtensorMap map2, const LayerSmallParams p) {
    using S = Shape<FORMAT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar_a[kMaxStages], bar_b[kMaxStages], bar_free[kMaxStages];
    __shared__ uint64_t wide_full[kSlots], wide_free[kSlots];
    __shared__ uint64_t acc_full[2], acc_free[2], drained;
    __shared__ uint32_t s_taddr;
    __shared__ int s_used, s_most;
    __shared__ volatile int s_failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = p.T * p.K, cta = blockIdx.x, ctas = gridDim.x;

    const Lists L(smem_raw, p.E, P);
    const uint32_t after = ptx::smem_u32(smem_raw) + ring::layer_list_bytes(p.E, P);
    uint8_t *stage0 =
        smem_raw + ring::layer_list_bytes(p.E, P) + ((1024u - (after & 1023u)) & 1023u);
    if (warp == kMmaWarp) tc::tmem_alloc(&s_taddr, S::kTmem);
    if (tid < kMaxStages) {
        ptx::mbar_init(&bar_a[tid], 1);
        ptx::mbar_init(&bar_b[tid], 32);
        ptx::mbar_init(&bar_free[tid], 1);
        if (tid < kSlots) {
            ptx::mbar_init(&wide_full[tid], 4);
            ptx::mbar_init(&wide_free[tid], 1);
        }
        if (tid < 2) {
            ptx::mbar_init(&acc_full[tid], 1);
            ptx::mbar_init(&acc_free[tid], 4);
        }
        if (tid == 0) {
            ptx::mbar_init(&drained, 1);
            s_failed = 0;
        }
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        tc::prefetch_map(&map13);
        tc::prefetch_map(&map2);
    }
    for (int e = tid; e < p.E; e += S::kThreads) L.count[e] = 0;

    // ---- lists: experts in use, ascending, and the pairs of each, by token ----
    // Thread i takes (t, k) = (i >> kshift, i mod 2^kshift): a token's experts stand
    // in one warp.  The first pair of a token that names an expert is kept, with the
    // gates of all.
    const int kshift = p.kshift, slots = p.T << kshift;
    auto load = [&](int i, int &id, float &g) {
        const int k = i & ((1 << kshift) - 1);
        id = -1;
        g = 0.0f;
        if (i < slots && k < p.K) {
            id = __ldg(p.topk_ids + (i >> kshift) * p.K + k);
            g = __ldg(p.topk_w + (i >> kshift) * p.K + k);
        }
    };
    int id;
    float g;
    load(tid, id, g);
    __syncthreads();  // the counts are zero
    for (int i0 = warp * 32; i0 < slots; i0 += S::kThreads) {
        const int i = i0 + lane, t = i >> kshift, k = i & ((1 << kshift) - 1);
        const bool real = i < slots && k < p.K;
        const int pair = t * p.K + k;
        if (i0 >= S::kThreads) load(i, id, g);
        if (real) {
            if (id < -1 || id >= p.E) {
                if (cta == 0) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_BAD_EXPERT_ID);
                id = -1;
            }
        }
        // lanes of the same token and expert (a lane without one stands alone)
        const unsigned same =
            __match_any_sync(0xffffffffu, id >= 0 ? (t << 10 | id) : (int)(0x80000000u | lane));
        const bool keep = id >= 0 && (same & ((1u << lane) - 1u)) == 0;
        float sum = g;
        for (unsigned more = __reduce_or_sync(0xffffffffu, same & (same - 1u)); more != 0;
             more &= more - 1u) {  // repeats, by ascending lane
            const int src = __ffs(more) - 1;
            const float other = __shfl_sync(0xffffffffu, g, src);
            if (keep && src != lane && (same >> src & 1u)) sum = __fadd_rn(sum, other);
        }
        if (real) {
            L.kept[pair] = (int16_t)(keep ? id : -1);
            L.gate[pair] = sum;
        }
        if (keep) atomicAdd(&L.count[id], 1);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) {  // lane l: experts 32 l .. 32 l + 31
        uint32_t bits = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const unsigned m =
                __ballot_sync(0xffffffffu, e0 + lane < p.E && L.count[e0 + lane] > 0);
            if (lane == e0 >> 5) bits = m;
        }
        int used = __popc(bits);
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, used, o);
            if (lane >= o) used += v;
        }
        for (int a = used - __popc(bits); bits != 0; bits &= bits - 1)
            L.expert[a++] = (uint16_t)(32 * lane + __ffs(bits) - 1);
        used = __shfl_sync(0xffffffffu, used, 31);
        __syncwarp();
        int pairs = 0, most = 0;
        for (int a0 = 0; a0 < used; a0 += 32) {
            const int a = a0 + lane, e = a < used ? L.expert[a] : 0, c = a < used ? L.count[e] : 0;
            int s = c;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            if (a < used) {
                L.base[a] = (uint16_t)(pairs + s - c);
                L.first[e] = (uint16_t)(pairs + s - c);
            }
            most = max(most, c);
            pairs += __shfl_sync(0xffffffffu, s, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            L.base[used] = (uint16_t)pairs;
            s_used = used;
            s_most = most;
        }
    }
    __syncthreads();
    // where the pairs stand; the weight producer needs none of it and goes ahead
    if (warp != kProducerWarp) {
        const int me = tid < kProducerWarp * 32 ? tid : tid - 32;
        for (int i0 = me & ~31; i0 < slots; i0 += S::kThreads - 32) {
            const int i = i0 + lane, t = i >> kshift, k = i & ((1 << kshift) - 1);
            if (i >= slots || k >= p.K) continue;
            const int pair = t * p.K + k, id = L.kept[pair];
            int at = -1;
            if (id >= 0) {  // behind the expert's pairs of the tokens before
                at = L.first[id];
                const uint4 *kept8 = reinterpret_cast<const uint4 *>(L.kept);
                const uint32_t both = (uint32_t)id << 16 | (uint32_t)id;
                for (int j = 0; j <= pair; j += 8) {
                    const uint4 v = kept8[j >> 3];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t d = w[q] ^ both;
                        at += ((d & 0xffffu) == 0 && j + 2 * q < pair) +
                              (d < 0x10000u && j + 2 * q + 1 < pair);
                    }
                }
                L.token[at] = (uint16_t)t;
            }
            L.place[pair] = (int16_t)at;
        }
        asm volatile("bar.sync 2, %0;" ::"n"(S::kThreads - 32) : "memory");
    }

    const int A = s_used;
    const uint32_t taddr = s_taddr;
    // A stage holds a unit's weights and the token rows of the fullest expert, in
    // groups of 8, 64 columns at a time; in phase 1 the rows of the activations'
    // second term stand behind those of the first.  (Products read 16 rows at a
    // time: what they read past the rows only reaches columns that nobody reads.)
    const int b_half = ring::layer_half_bytes(s_most);
    const int stage_bytes = ring::layer_stage_bytes(S::kValue, s_most);
    const int stages = ring::layer_stages(p.ring_bytes, S::kValue, s_most);
    auto stage_a = [&](int s) { return stage0 + s * stage_bytes; };
    auto stage_b = [&](int s) { return stage0 + s * stage_bytes + S::kA; };
    // phase 0: tiles (expert, 64 gate + 64 up rows); phase 1: (128 rows of H, expert)
    const int tiles0 = (p.I + kHalfRows - 1) / kHalfRows, tiles1 = (p.H + kTileRows - 1) / kTileRows;
    const int blocks0 = (p.H + kBlockK - 1) / kBlockK, blocks1 = (p.I + kBlockK - 1) / kBlockK;
    // (merging parts takes about 2.5 us, a unit 0.7 us of bf16 weights, half of it of 8-bit)
    constexpr int kMerge = S::kWiden ? 7 : 4;
    const Cut cuts[2] = {cut<true>(A * tiles0, blocks0, ctas, kMerge),
                         cut<true>(A * tiles1, blocks1, ctas, kMerge)};
    auto tile_of = [&](int phase, int tile, int &a, int &r) {
        if (phase == 0) {
            a = tile / tiles0;
            r = tile - a * tiles0;
        } else {
            r = tile / A;
            a = tile - r * A;
        }
    };

    if (warp == kProducerWarp) {
        if (ptx::elect_one()) {
            Turn st(stages);
            uint32_t issued = 0;  // stages in use
            for (int phase = 0; phase < 2; ++phase) {
                Segments segs(cuts[phase], cta, phase ? blocks1 : blocks0);
                Segment sg;
                while (!s_failed && segs.next(sg)) {
                    int a, r;
                    tile_of(phase, sg.tile, a, r);
                    const int e = L.expert[a];
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int s = (int)st.at;
                        if (!ptx::mbar_park(&bar_free[s], st.parity ^ 1u, kWaitNs)) {
                            s_failed = 1;
                            break;
                        }
                        issued |= 1u << s;
                        ptx::mbar_arrive_expect_tx(&bar_a[s], (uint32_t)S::kA);
                        uint8_t *dst = stage_a(s);
                        constexpr int kHalves = S::kWiden ? 1 : 2;
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) {
                            const int x = kb * kBlockK + h * 64;
                            uint8_t *d = dst + h * kTileRows * kAtom;
                            if (phase == 0)
                                tc::tma_load_5d(d, &map13, x, 0, 0, r * (kHalfRows / kQuarter), e,
                                                &bar_a[s]);
                            else
                                tc::tma_load_3d(d, &map2, x, r * kTileRows, e, &bar_a[s]);
                        }
                    }
                }
            }
            // copies still in flight land before shared memory goes away
            for (int i = 0; i < stages; ++i, st.next()) {  // (parity: of the stage's last use)
                const uint32_t last = st.parity ^ 1u;
                if (issued >> st.at & 1u) ptx::mbar_park(&bar_a[st.at], last, kWaitNs);
            }
        }
    } else if (warp == kMmaWarp) {
        if (ptx::elect_one()) {
            uint32_t it = 0;
            Turn st(stages), wide(kSlots);
            const uint64_t ad0 = tc::smem_desc_sw128(ptx::smem_u32(stage0));
            const uint64_t half_a = kTileRows * kAtom / 16, half_b = b_half / 16;
            for (int phase = 0; phase < 2; ++phase) {
                Segments segs(cuts[phase], cta, phase ? blocks1 : blocks0);
                Segment sg;
                for (; !s_failed && segs.next(sg); ++it) {
                    int a, r;
                    tile_of(phase, sg.tile, a, r);
                    const int rows = L.base[a + 1] - L.base[a];
                    const int cols = phase ? (rows + 7) / 8 * 16 : (rows + 15) / 16 * 16;
                    const uint32_t idesc = tc::idesc_bf16_f32(kTileRows, cols);
                    const uint32_t b = it & 1u, d = taddr + b * kAccCols;
                    if (!ptx::mbar_park(&acc_free[b], ((it >> 1) & 1u) ^ 1u, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    tc::fence_after_sync();
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next(), wide.next()) {
                        const int s = (int)st.at;
                        bool ok = ptx::mbar_park(&bar_b[s], st.parity, kWaitNs);
                        if (S::kWiden)
                            ok = ok && ptx::mbar_park(&wide_full[wide.at], wide.parity,
                                                            kWaitNs);
                        else
                            ok = ok && ptx::mbar_park(&bar_a[s], st.parity, kWaitNs);
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        tc::fence_after_sync();
                        // token rows: written by cp.async (generic proxy), read next by
                        // the tensor cores (async proxy)
                        ptx::fence_proxy_async_smem();
                        const uint64_t ad = ad0 + (uint64_t)(s * (stage_bytes / 16));
                        const uint64_t bd = ad + S::kA / 16;
                        const uint32_t at = taddr + 2 * kAccCols + wide.at * kSlotCols;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {  // 16 k a step
                            const uint64_t bk = bd + (kk >> 2) * half_b + 2 * (kk & 3);
                            const bool acc = kb != sg.k0 || kk != 0;
                            const uint64_t ak = ad + (kk >> 2) * half_a + 2 * (kk & 3);
                            if constexpr (S::kWiden)
                                tc::mma_f16_ta(d, at + 8 * kk, bk, idesc, acc);
                            else
                                tc::mma_bf16(d, ak, bk, idesc, acc);
                        }
                        tc::commit(&bar_free[s]);
                        if (S::kWiden) tc::commit(&wide_free[wide.at]);
                    }
                    tc::commit(&acc_full[b]);
                }
            }
            tc::commit(&drained);  // before tensor memory is freed
            ptx::mbar_park(&drained, 0, kWaitNs);
        }
    } else if (warp >= kLoaderWarp0 && warp < kLoaderWarp0 + kLoaders) {
        // The warps take the units in turn.  Lane l copies 16-byte piece l % 16 (8
        // values) of the rows l / 16, l / 16 + 2, ... of a unit: half (piece / 8),
        // chunk piece % 8 stored at chunk ^ (row mod 8), the swizzle that TMA would
        // apply.
        const int piece = lane & 15, row0 = lane >> 4;
        Turn st(stages);
        uint32_t n = (uint32_t)(kLoaders - (warp - kLoaderWarp0));
        for (int phase = 0; phase < 2; ++phase) {
            const int width = phase ? p.I : p.H;
            Segments segs(cuts[phase], cta, phase ? blocks1 : blocks0);
            Segment sg;
            if (phase == 1) {
                // every activation is written before any is read
                bool ok = true;
                if (lane == 0) ok = wait_count(&p.header->done[0], A * tiles0 * 4, &s_failed);
                if (!__all_sync(0xffffffffu, ok)) s_failed = 1;
                __syncwarp();  // (a vote orders no memory)
            }
            while (!warp_flag(&s_failed) && segs.next(sg)) {
                int a, r;
                tile_of(phase, sg.tile, a, r);
                const int base = L.base[a], rows = L.base[a + 1] - base;
                const int second = (rows + 7) / 8 * 8 * kAtom;  // where the second term's rows begin
                const uint16_t *src = phase ? p.act + (size_t)base * 2 * p.I : p.x;
                for (int kb = sg.k0; kb < sg.k1; ++kb, st.next(), ++n) {
                    if (n % kLoaders != 0) continue;
                    const int s = (int)st.at;
                    if (!__all_sync(0xffffffffu, ptx::mbar_park(
                                                     &bar_free[s], st.parity ^ 1u, kWaitNs))) {
                        s_failed = 1;
                        break;
                    }
                    uint8_t *dst = stage_b(s) + (piece >> 3) * b_half;
                    const int col = kb * kBlockK + piece * 8;
                    for (int row = row0; row < rows; row += 2) {
                        const size_t at = (size_t)(phase ? 2 * row : L.token[base + row]) * width;
                        uint8_t *to = dst + row * kAtom + (((piece & 7) ^ (row & 7)) << 4);
                        if (col < width) {
                            ptx::cp_async16(to, src + at + col);
                            if (phase) ptx::cp_async16(to + second, src + at + width + col);
                        } else {  // past the end: zero, beside the weights' zero fill
                            ptx::cp_async16_zero(to, src);
                            if (phase) ptx::cp_async16_zero(to + second, src);
                        }
                    }
                    ptx::cp_async_mbar_arrive_noinc(&bar_b[s]);
                }
            }
        }
        ptx::cp_async_wait_all();  // copies land before shared memory goes away
    } else if (S::kWiden && warp >= kConvertWarp0) {
        // Thread l of a group owns weight row l of the tile = lane l; the groups
        // take the units in turn, so that one group's loads and waits pass while
        // the other computes.
        const int row = (tid - kConvertWarp0 * 32) & 127, group = (warp - kConvertWarp0) >> 2;
        long long units = 0;
        for (int phase = 0; phase < 2; ++phase)
            if (cta < cuts[phase].parts) units += cuts[phase].first(cta + 1) - cuts[phase].first(cta);
        Turn st(stages), wide(kSlots);
        for (uint32_t n = 0; n < (uint32_t)units; ++n, st.next(), wide.next()) {
            if ((n & 1u) != (uint32_t)group) continue;
            if (warp_flag(&s_failed)) break;
            const int s = (int)st.at, q = (int)wide.at;
            const bool ok = ring::widen_ready(
                [&] { return ptx::mbar_park(&wide_free[q], wide.parity ^ 1u, kWaitNs); },
                [&] { return ptx::mbar_park(&bar_a[s], st.parity, kWaitNs); });
            if (!__all_sync(0xffffffffu, ok)) {
                s_failed = 1;
                break;
            }
            tc::fence_after_sync();
            const uint8_t *src = stage_a(s) + row * kAtom;
            const uint32_t dst = taddr + 2 * kAccCols + q * kSlotCols +
                                 ((uint32_t)(row & ~31) << 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        src + (((4 * h + c) ^ (row & 7)) << 4));
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (FORMAT == MOE_FORMAT_FP8_E4M3)
                            e4m3_to_bf16(u[i], w[8 * c + 2 * i], w[8 * c + 2 * i + 1]);
                        else
                            int8_to_bf16(u[i], w[8 * c + 2 * i], w[8 * c + 2 * i + 1]);
                    }
                }
                tc::st_32x32(dst + 32 * h, w);
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&wide_full[q]);
        }
    } else if (warp < 4) {
        // Each warp finishes its 32 rows by itself: in phase 0 the lanes below 16
        // hold gate rows, the others the up rows of the same channels.
        uint32_t it = 0;
        bool ok = true;
        for (int phase = 0; phase < 2 && ok; ++phase) {
            const int blocks = phase ? blocks1 : blocks0;
            Segments segs(cuts[phase], cta, blocks);
            Segment sg;
            for (; segs.next(sg); ++it) {
                const uint32_t b = it & 1u;
                ok = __all_sync(0xffffffffu,
                                ptx::mbar_park(&acc_full[b], (it >> 1) & 1u, kWaitNs) &&
                                    !s_failed);
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                int a, r;
                tile_of(phase, sg.tile, a, r);
                const int e = L.expert[a], base = L.base[a], rows = L.base[a + 1] - base;
                const uint32_t acc = taddr + b * kAccCols + ((uint32_t)(warp * 32) << 16);
                const bool whole = sg.k0 == 0 && sg.k1 == blocks;
                const int second = (rows + 7) / 8 * 8;  // columns of the second term, phase 1
                auto take = [&](int n0, float (&v)[kCols]) {
                    uint32_t u[kCols], w[kCols];
                    tc::ld_32x8(acc + n0, u);
                    if (phase) tc::ld_32x8(acc + second + n0, w);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < kCols; ++i) {
                        v[i] = __uint_as_float(u[i]);
                        if (phase) v[i] += __uint_as_float(w[i]);
                    }
                };
                Parts parts;
                auto part_of = [&](int c) {
                    return p.part + ((size_t)(2 * c + parts.slot(c)) * p.nmax) * kTileRows + tid;
                };
                if (!whole) {
                    parts = Parts(cuts[phase], sg.tile, blocks);
                    float *to = part_of(cta);
                    for (int n0 = 0; n0 < rows; n0 += kCols) {
                        float v[kCols];
                        take(n0, v);
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            if (n0 + i < rows) __stcg(to + (n0 + i) * kTileRows, v[i]);
                    }
                    tc::fence_before_sync();
                    // the warp's parts, then lane 0's fence and count; and the other way
                    // round: what lane 0 finds counted, its fence, then the warp's reads
                    // (a shuffle orders no memory)
                    __syncwarp();
                    __threadfence();
                    int last = 0;
                    if (lane == 0) {
                        mbar_arrive(&acc_free[b]);
                        int *m = &p.header->merged[phase][parts.c0][warp];
                        last = atomicAdd(m, 1) == parts.count() - 1;
                        if (last) *m = 0;  // for the next call
                        __threadfence();
                    }
                    if (!__shfl_sync(0xffffffffu, last, 0)) continue;
                    __syncwarp();
                }
                // channel of this lane, whether it is stored, its scale
                int chan, limit;
                const float *scales;
                if (phase == 0) {
                    chan = r * kHalfRows + warp * kQuarter + (lane & (kQuarter - 1));
                    limit = p.I;
                    scales = p.w13_scale + (size_t)e * 2 * p.I + (lane < kQuarter ? 0 : p.I);
                } else {
                    chan = r * kTileRows + tid;
                    limit = p.H;
                    scales = p.w2_scale + (size_t)e * p.H;
                }
                float sc = S::kWiden && chan < limit ? __ldg(scales + chan) : 1.0f;
                if (FORMAT == MOE_FORMAT_INT8) sc *= kInt8Bf16;
                for (int n0 = 0; n0 < rows; n0 += kCols) {
                    float v[kCols];
                    if (whole) {
                        take(n0, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
                        for (int c = parts.c0; c <= parts.c1; ++c) {
                            const float *from = part_of(c);
#pragma unroll
                            for (int i = 0; i < kCols; ++i)
                                if (n0 + i < rows) v[i] += __ldcg(from + (n0 + i) * kTileRows);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kCols; ++i) {
                        if (n0 + i >= rows) break;  // (the warp alike)
                        const float z = v[i] * sc;
                        if (phase == 0) {
                            const float up = __shfl_down_sync(0xffffffffu, z, kQuarter);
                            const float f = z / (1.0f + expf(-z)) * up;
                            const __nv_bfloat16 hi = __float2bfloat16_rn(f);
                            const float fh = __bfloat162float(hi);
                            // (nothing is left of an infinity)
                            const __nv_bfloat16 lo =
                                __float2bfloat16_rn(isinf(fh) ? 0.0f : f - fh);
                            if (lane < kQuarter && chan < limit) {
                                uint16_t *to = p.act + (size_t)(base + n0 + i) * 2 * p.I + chan;
                                to[0] = *reinterpret_cast<const uint16_t *>(&hi);
                                to[p.I] = *reinterpret_cast<const uint16_t *>(&lo);
                            }
                        } else if (chan < limit) {
                            __stcg(p.y + (size_t)(base + n0 + i) * p.H + chan, z);
                        }
                    }
                }
                if (whole) tc::fence_before_sync();
                __syncwarp();
                __threadfence();
                if (lane == 0) {
                    if (whole) mbar_arrive(&acc_free[b]);
                    atomicAdd(&p.header->done[phase], 1);
                }
            }
        }
        // ---- gated sum over the token's experts, all CTAs ----
        if (ok && tid == 0 && !wait_count(&p.header->done[1], A * tiles1 * 4, &s_failed)) s_failed = 1;
        epi_sync();
        if (!s_failed) {
            const int H4 = p.H / 4;
            for (int i = cta * kEpiThreads + tid; i < p.T * H4; i += ctas * kEpiThreads) {
                const int t = i / H4, h = (i - t * H4) * 4;
                float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int k = 0; k < p.K; ++k) {
                    const int at = L.place[t * p.K + k];
                    if (at < 0) continue;
                    const float g = L.gate[t * p.K + k];
                    const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)at * p.H + h));
                    o[0] = fmaf(g, y.x, o[0]);
                    o[1] = fmaf(g, y.y, o[1]);
                    o[2] = fmaf(g, y.z, o[2]);
                    o[3] = fmaf(g, y.w, o[3]);
                }
                const size_t at = (size_t)t * p.H + h;
                if (p.residual != nullptr) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(p.residual + at);
                    o[0] += __uint_as_float(u.x << 16);
                    o[1] += __uint_as_float(u.x & 0xffff0000u);
                    o[2] += __uint_as_float(u.y << 16);
                    o[3] += __uint_as_float(u.y & 0xffff0000u);
                }
                __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]);
                __nv_bfloat162 hi = __floats2bfloat162_rn(o[2], o[3]);
                *reinterpret_cast<uint2 *>(p.out + at) =
                    make_uint2(*reinterpret_cast<uint32_t *>(&lo), *reinterpret_cast<uint32_t *>(&hi));
            }
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0) {
        if (s_failed) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_WAIT_TIMEOUT);
        // the last CTA to come through leaves the counters at zero
        __threadfence();
        if (atomicAdd(&p.header->left, 1) == ctas - 1) {
            p.header->done[0] = 0;
            p.header->done[1] = 0;
            p.header->left = 0;
        }
    }
    if (warp == kMmaWarp) tc::tmem_dealloc(taddr, S::kTmem);
}

template <int FORMAT>
cudaError_t launch_t(LayerSmallParams &p, int num_sms, cudaStream_t st) {
    using S = Shape<FORMAT>;
    CUtensorMap m13, m2;
    // W13: a box holds 4 times 16 gate rows and the up rows of the same channels;
    // W2: 128 rows.  What a box has past its expert's rows reads as zero.
    const long long H = p.H, I = p.I;
    const int width = S::kWiden ? kAtom : kAtom / 2;
    const long long ext13[5] = {H, kQuarter, 2, I / kQuarter, p.E};
    const long long str13[5] = {1, H, I * H, kQuarter * H, 2 * I * H};
    const int box13[5] = {width, kQuarter, 2, kHalfRows / kQuarter, 1};
    const long long ext2[3] = {I, H, p.E}, str2[3] = {1, I, H * I};
    const int box2[3] = {width, kTileRows, 1};
    if (!make_map_nd(&m13, p.w13, 5, ext13, str13, box13, S::kWiden) ||
        !make_map_nd(&m2, p.w2, 3, ext2, str2, box2, S::kWiden))
        return cudaErrorInvalidValue;
    const int P = p.T * p.K;
    p.ring_bytes = ring::layer_ring_bytes(p.E, P);
    if (!ring::layer_holds(S::kValue, ring::layer_stages(p.ring_bytes, S::kValue, p.T)))
        return cudaErrorInvalidValue;
    const size_t smem = (size_t)ring::layer_front_bytes(p.E, P) + (size_t)p.ring_bytes;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = raise_smem_limit_once(layer_small_kernel<FORMAT>, kMaxDynamic, raised);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms < kStreamMaxCtas ? num_sms : kStreamMaxCtas));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // the CTAs wait for one another: all of them run at once or none does
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, layer_small_kernel<FORMAT>, m13, m2,
                              (const LayerSmallParams &)p);
}

}  // namespace

cudaError_t launch_layer_small(LayerSmallParams p, int num_sms, cudaStream_t st) {
    if (p.T < 1 || p.T > kLayerMaxTokens || p.K < 1 || p.K > 32 || p.E < 1 || p.E > 1024 ||
        p.H % 16 != 0 || p.I % 16 != 0 || p.H < 16 || p.I < 16)
        return cudaErrorInvalidValue;
    p.nmax = (p.T + 15) / 16 * 16;
    p.kshift = 0;
    while (1 << p.kshift < p.K) ++p.kshift;
    if (p.format == MOE_FORMAT_BF16) return launch_t<MOE_FORMAT_BF16>(p, num_sms, st);
    if (p.format == MOE_FORMAT_FP8_E4M3) return launch_t<MOE_FORMAT_FP8_E4M3>(p, num_sms, st);
    return launch_t<MOE_FORMAT_INT8>(p, num_sms, st);
}

}  // namespace moe
