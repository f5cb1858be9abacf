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
//   warps 6-7: token rows into the stages (16-byte cp.async, swizzled alike);
//   warps 8-15, 8-bit formats: two groups of four in turn widen a stage's
//     weight rows to bf16 into tensor memory (exact), which the products read
//     as their A operand.
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

constexpr int kEpiThreads = 128;
constexpr int kProducerWarp = 4, kMmaWarp = 5, kLoaderWarp0 = 6, kConvertWarp0 = 8;
constexpr int kLoaderThreads = 64;
constexpr int kHalfRows = 64;   // gate rows (and up rows) of a W13 tile
constexpr int kSlots = 4;       // widened weight tiles in tensor memory
constexpr int kSlotCols = kBlockK / 2;
constexpr int kMaxStages = 16;
// dynamic shared memory: 227 KB a CTA less the static barriers and the exchange rows
constexpr size_t kMaxDynamic = (227 - 6) * 1024;

// Bytes of the lists at the front of dynamic shared memory.
__host__ __device__ inline int lists_bytes(int E, int P) {
    // experts in use and their first pairs; tokens, places, experts and gates of the pairs
    const int A = E < P ? E : P;
    return ((A * 2 + (A + 1) * 2 + P * 2 + P * 2 + P * 2) + P * 4 + 15 + 16) / 16 * 16;
}

struct Lists {
    float *gate;       // [P] gate of (t, k), set where kept
    uint16_t *expert;  // [A]
    uint16_t *base;    // [A + 1] first pair of an expert in use
    uint16_t *token;   // [P] token of a pair
    int16_t *place;    // [P] pair of (t, k), -1 where dropped (at first: its expert)
    int16_t *kept;     // [P] expert of (t, k), -1 where dropped
    __device__ Lists(uint8_t *mem, int E, int P) {
        const int A = E < P ? E : P;
        gate = reinterpret_cast<float *>(mem);
        expert = reinterpret_cast<uint16_t *>(gate + P);
        base = expert + A;
        token = base + A + 1;
        place = reinterpret_cast<int16_t *>(token + P);
        kept = place + P;
    }
};

template <int FORMAT>
struct Shape {
    static constexpr bool kWiden = FORMAT != MOE_FORMAT_BF16;
    static constexpr int kThreads = (kWiden ? 16 : 8) * 32;
    static constexpr int kA = kTileRows * kBlockK * (kWiden ? 1 : 2);  // weight bytes a stage
    static constexpr int kCols = kWiden ? 512 : 128;                   // tensor-memory columns
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
    __shared__ int s_used, s_most, s_last;
    __shared__ volatile int s_failed;
    __shared__ float s_up[16][kHalfRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = p.T * p.K, cta = blockIdx.x, ctas = gridDim.x;

    const Lists L(smem_raw, p.E, P);
    const uint32_t after = ptx::smem_u32(smem_raw) + lists_bytes(p.E, P);
    uint8_t *ring = smem_raw + lists_bytes(p.E, P) + ((1024u - (after & 1023u)) & 1023u);
    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar_a[s], 1);
            ptx::mbar_init(&bar_b[s], kLoaderThreads);
            ptx::mbar_init(&bar_free[s], 1);
        }
        for (int q = 0; q < kSlots; ++q) {
            ptx::mbar_init(&wide_full[q], 4);
            ptx::mbar_init(&wide_free[q], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_free[b], 4);
        }
        ptx::mbar_init(&drained, 1);
        ptx::fence_mbar_init();
        s_failed = 0;
    }
    if (warp == kMmaWarp) tc::tmem_alloc(&s_taddr, S::kCols);

    // ---- lists: experts in use, ascending, and the pairs of each, by token ----
    int *count = reinterpret_cast<int *>(ring);  // [E], before the ring is in use
    int *first = count + p.E;                    // [E] first pair of an expert
    for (int e = tid; e < p.E; e += S::kThreads) count[e] = 0;
    for (int i = tid; i < P; i += S::kThreads) {
        int id = __ldg(p.topk_ids + i);
        if (id < -1 || id >= p.E) {
            if (cta == 0) atomicOr(&p.header->flags, MOE_DEVICE_FLAG_BAD_EXPERT_ID);
            id = -1;
        }
        L.place[i] = (int16_t)id;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // the first pair of a token that names an expert is kept, with the gates of all
    for (int i = tid; i < P; i += S::kThreads) {
        const int t0 = i / p.K * p.K, id = L.place[i];
        bool keep = id >= 0;
        for (int j = t0; j < i && keep; ++j) keep = L.place[j] != id;
        L.kept[i] = (int16_t)(keep ? id : -1);
        if (!keep) continue;
        atomicAdd(&count[id], 1);
        float g = __ldg(p.topk_w + i);
        for (int j = i + 1; j < t0 + p.K; ++j)
            if (L.place[j] == id) g = __fadd_rn(g, __ldg(p.topk_w + j));
        L.gate[i] = g;
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefixes of the counts and of the experts in use
        int used = 0, pairs = 0, most = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane, c = e < p.E ? count[e] : 0;
            int s = c;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            const unsigned m = __ballot_sync(0xffffffffu, c > 0);
            most = max(most, c);
            if (c > 0) {
                const int a = used + __popc(m & ((1u << lane) - 1u));
                L.expert[a] = (uint16_t)e;
                L.base[a] = (uint16_t)(pairs + s - c);
                first[e] = pairs + s - c;
            }
            used += __popc(m);
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
    for (int i = tid; i < P; i += S::kThreads) {
        const int id = L.kept[i];
        int at = -1;
        if (id >= 0) {
            at = first[id];
            for (int j = 0; j < i; ++j) at += L.kept[j] == id;
            L.token[at] = (uint16_t)(i / p.K);
        }
        L.place[i] = (int16_t)at;
    }
    ptx::fence_proxy_async_smem();  // the ring's memory goes to TMA
    __syncthreads();

    const int A = s_used;
    const uint32_t taddr = s_taddr;
    // A stage holds a unit's weights and the token rows of the fullest expert, in
    // groups of 8, 64 columns at a time: two halves, and twice for the two terms
    // of the activations.  (Products read 16 rows at a time: what they read past
    // the rows only reaches columns that nobody reads.)
    const int b_rows = (s_most + 7) / 8 * 8, b_half = b_rows * kAtom;
    const int stage_bytes = S::kA + 4 * b_half;
    const int stages = min(kMaxStages, p.ring_bytes / stage_bytes);
    auto stage_a = [&](int s) { return ring + s * stage_bytes; };
    auto stage_b = [&](int s) { return ring + s * stage_bytes + S::kA; };
    // phase 0: tiles (expert, 64 gate + 64 up rows); phase 1: (128 rows of H, expert)
    const int tiles0 = (p.I + kHalfRows - 1) / kHalfRows, tiles1 = (p.H + kTileRows - 1) / kTileRows;
    const int blocks0 = (p.H + kBlockK - 1) / kBlockK, blocks1 = (p.I + kBlockK - 1) / kBlockK;
    const Cut cuts[2] = {cut((long long)A * tiles0 * blocks0, ctas),
                         cut((long long)A * tiles1 * blocks1, ctas)};
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
                    const void *map = phase ? (const void *)&map2 : (const void *)&map13;
                    const int row0 = phase ? e * p.H + r * kTileRows : e * 2 * p.I + r * kHalfRows;
                    const int row1 = phase ? row0 + kHalfRows : row0 + p.I;
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                        const int s = (int)st.at;
                        if (!ptx::mbar_wait_timed(&bar_free[s], st.parity ^ 1u, kWaitNs)) {
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
                            tc::tma_load_2d(d, map, x, row0, &bar_a[s]);
                            tc::tma_load_2d(d + kHalfRows * kAtom, map, x, row1, &bar_a[s]);
                        }
                    }
                }
            }
            // copies still in flight land before shared memory goes away
            for (int i = 0; i < stages; ++i, st.next()) {  // (parity: of the stage's last use)
                const uint32_t last = st.parity ^ 1u;
                if (issued >> st.at & 1u) ptx::mbar_wait_timed(&bar_a[st.at], last, kWaitNs);
            }
        }
    } else if (warp == kMmaWarp) {
        if (ptx::elect_one()) {
            uint32_t it = 0;
            Turn st(stages), wide(kSlots);
            for (int phase = 0; phase < 2; ++phase) {
                Segments segs(cuts[phase], cta, phase ? blocks1 : blocks0);
                Segment sg;
                for (; !s_failed && segs.next(sg); ++it) {
                    int a, r;
                    tile_of(phase, sg.tile, a, r);
                    const int cols = ((int)L.base[a + 1] - L.base[a] + 15) / 16 * 16;
                    const uint32_t idesc = tc::idesc_bf16_f32(kTileRows, cols);
                    const uint32_t b = it & 1u, d = taddr + b * kLayerMaxTokens;
                    if (!ptx::mbar_wait_timed(&acc_free[b], ((it >> 1) & 1u) ^ 1u, kWaitNs)) {
                        s_failed = 1;
                        break;
                    }
                    tc::fence_after_sync();
                    for (int kb = sg.k0; kb < sg.k1; ++kb, st.next(), wide.next()) {
                        const int s = (int)st.at;
                        bool ok = ptx::mbar_wait_timed(&bar_b[s], st.parity, kWaitNs);
                        if (S::kWiden)
                            ok = ok && ptx::mbar_wait_timed(&wide_full[wide.at], wide.parity,
                                                            kWaitNs);
                        else
                            ok = ok && ptx::mbar_wait_timed(&bar_a[s], st.parity, kWaitNs);
                        if (!ok) {
                            s_failed = 1;
                            break;
                        }
                        tc::fence_after_sync();
                        // token rows: written by cp.async (generic proxy), read next by
                        // the tensor cores (async proxy)
                        ptx::fence_proxy_async_smem();
                        const uint64_t ad = tc::smem_desc_sw128(ptx::smem_u32(stage_a(s)));
                        const uint64_t bd = tc::smem_desc_sw128(ptx::smem_u32(stage_b(s)));
                        const uint64_t half_a = kTileRows * kAtom / 16, half_b = b_half / 16;
                        const uint32_t at = taddr + 2 * kLayerMaxTokens + wide.at * kSlotCols;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {  // 16 k a step
                            const uint64_t bk = bd + (kk >> 2) * half_b + 2 * (kk & 3);
                            const bool acc = kb != sg.k0 || kk != 0;
                            const uint64_t ak = ad + (kk >> 2) * half_a + 2 * (kk & 3);
                            if constexpr (S::kWiden)
                                tc::mma_f16_ta(d, at + 8 * kk, bk, idesc, acc);
                            else
                                tc::mma_bf16(d, ak, bk, idesc, acc);
                            if (phase == 0) continue;
                            if constexpr (S::kWiden)  // the second term
                                tc::mma_f16_ta(d, at + 8 * kk, bk + 2 * half_b, idesc, true);
                            else
                                tc::mma_bf16(d, ak, bk + 2 * half_b, idesc, true);
                        }
                        tc::commit(&bar_free[s]);
                        if (S::kWiden) tc::commit(&wide_free[wide.at]);
                    }
                    tc::commit(&acc_full[b]);
                }
            }
            tc::commit(&drained);  // before tensor memory is freed
            ptx::mbar_wait_timed(&drained, 0, kWaitNs);
        }
    } else if (warp == kLoaderWarp0 || warp == kLoaderWarp0 + 1) {
        // Thread l copies 16-byte piece l % 16 (8 values) of the rows l / 16,
        // l / 16 + 4, ... of a unit: half (piece / 8), chunk piece % 8 stored at
        // chunk ^ (row mod 8), the swizzle that TMA would apply.
        const int l = tid - kLoaderWarp0 * 32, piece = l & 15, row0 = l >> 4;
        Turn st(stages);
        for (int phase = 0; phase < 2; ++phase) {
            const int width = phase ? p.I : p.H;
            Segments segs(cuts[phase], cta, phase ? blocks1 : blocks0);
            Segment sg;
            if (phase == 1) {
                // every activation is written before any is read
                bool ok = true;
                if (lane == 0) ok = wait_count(&p.header->done[0], A * tiles0, &s_failed);
                if (!__all_sync(0xffffffffu, ok)) s_failed = 1;
            }
            while (!warp_flag(&s_failed) && segs.next(sg)) {
                int a, r;
                tile_of(phase, sg.tile, a, r);
                const int base = L.base[a], rows = L.base[a + 1] - base;
                const uint16_t *src = phase ? p.act + (size_t)base * 2 * p.I : p.x;
                for (int kb = sg.k0; kb < sg.k1; ++kb, st.next()) {
                    const int s = (int)st.at;
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait_timed(
                                                     &bar_free[s], st.parity ^ 1u, kWaitNs))) {
                        s_failed = 1;
                        break;
                    }
                    uint8_t *dst = stage_b(s) + (piece >> 3) * b_half;
                    const int col = kb * kBlockK + piece * 8;
                    for (int row = row0; row < rows; row += 4) {
                        const size_t at = (size_t)(phase ? 2 * row : L.token[base + row]) * width;
                        uint8_t *to = dst + row * kAtom + (((piece & 7) ^ (row & 7)) << 4);
                        if (col < width) {
                            ptx::cp_async16(to, src + at + col);
                            if (phase) ptx::cp_async16(to + 2 * b_half, src + at + width + col);
                        } else {  // past the end: zero, beside the weights' zero fill
                            ptx::cp_async16_zero(to, src);
                            if (phase) ptx::cp_async16_zero(to + 2 * b_half, src);
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
            const bool ok = ptx::mbar_wait_timed(&bar_a[s], st.parity, kWaitNs) &&
                            ptx::mbar_wait_timed(&wide_free[q], wide.parity ^ 1u, kWaitNs);
            if (!__all_sync(0xffffffffu, ok)) {
                s_failed = 1;
                break;
            }
            tc::fence_after_sync();
            const uint8_t *src = stage_a(s) + row * kAtom;
            const uint32_t dst = taddr + 2 * kLayerMaxTokens + q * kSlotCols +
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
                uint32_t it = 0;
        bool ok = true;
        for (int phase = 0; phase < 2 && ok; ++phase) {
            const int blocks = phase ? blocks1 : blocks0;
            Segments segs(cuts[phase], cta, blocks);
            Segment sg;
            for (; segs.next(sg); ++it) {
                const uint32_t b = it & 1u;
                ok = ptx::mbar_wait_timed(&acc_full[b], (it >> 1) & 1u, kWaitNs);
                ok = !epi_any(!ok || s_failed);  // (all four warps leave together)
                if (!ok) {
                    s_failed = 1;
                    break;
                }
                tc::fence_after_sync();
                int a, r;
                tile_of(phase, sg.tile, a, r);
                const int e = L.expert[a], base = L.base[a], rows = L.base[a + 1] - base;
                const uint32_t acc = taddr + b * kLayerMaxTokens + ((uint32_t)(tid & ~31) << 16);
                const bool whole = sg.k0 == 0 && sg.k1 == blocks;
                const Parts parts(cuts[phase], sg.tile, blocks);
                auto part_of = [&](int c) {
                    return p.part + ((size_t)(2 * c + parts.slot(c)) * p.nmax) * kTileRows + tid;
                };
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
                        int *m = &p.header->merged[phase][parts.c0];
                        s_last = atomicAdd(m, 1) == parts.count() - 1;
                        if (s_last) *m = 0;  // for the next call
                    }
                    epi_sync();
                    if (!s_last) continue;
                    __threadfence();
                }
                // channel of this thread: its row, whether it is stored, its scale
                int chan, limit;
                const float *scales;
                if (phase == 0) {
                    chan = r * kHalfRows + (tid & (kHalfRows - 1));
                    limit = p.I;
                    scales = p.w13_scale + (size_t)e * 2 * p.I + (tid < kHalfRows ? 0 : p.I);
                } else {
                    chan = r * kTileRows + tid;
                    limit = p.H;
                    scales = p.w2_scale + (size_t)e * p.H;
                }
                float sc = S::kWiden && chan < limit ? __ldg(scales + chan) : 1.0f;
                if (FORMAT == MOE_FORMAT_INT8) sc *= kInt8Bf16;
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
                    for (int i = 0; i < 16; ++i) v[i] *= sc;
                    if (phase == 0) {
                        if (tid >= kHalfRows) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) s_up[i][tid - kHalfRows] = v[i];
                        }
                        epi_sync();
                        if (tid < kHalfRows && chan < limit) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (n0 + i < rows) {
                                    const float z = v[i] / (1.0f + expf(-v[i])) * s_up[i][tid];
                                    const __nv_bfloat16 hi = __float2bfloat16_rn(z);
                                    const float zh = __bfloat162float(hi);
                                    // (nothing is left of an infinity)
                                    const __nv_bfloat16 lo = __float2bfloat16_rn(
                                        isinf(zh) ? 0.0f : z - zh);
                                    uint16_t *to = p.act + (size_t)(base + n0 + i) * 2 * p.I + chan;
                                    to[0] = *reinterpret_cast<const uint16_t *>(&hi);
                                    to[p.I] = *reinterpret_cast<const uint16_t *>(&lo);
                                }
                        }
                        epi_sync();
                    } else if (chan < limit) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < rows)
                                __stcg(p.y + (size_t)(base + n0 + i) * p.H + chan, v[i]);
                    }
                }
                if (whole) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[b]);
                }
                __threadfence();
                epi_sync();
                if (tid == 0) atomicAdd(&p.header->done[phase], 1);
            }
        }
        // ---- gated sum over the token's experts, all CTAs ----
        if (ok && tid == 0 && !wait_count(&p.header->done[1], A * tiles1, &s_failed)) s_failed = 1;
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
    if (warp == kMmaWarp) tc::tmem_dealloc(taddr, S::kCols);
}

template <int FORMAT>
cudaError_t launch_t(LayerSmallParams &p, int num_sms, cudaStream_t st) {
    using S = Shape<FORMAT>;
    CUtensorMap m13, m2;
    if (!make_map(&m13, p.w13, (long long)p.E * 2 * p.I, p.H, kHalfRows, S::kWiden) ||
        !make_map(&m2, p.w2, (long long)p.E * p.H, p.I, kHalfRows, S::kWiden))
        return cudaErrorInvalidValue;
    // 1 KB aligns the ring and 1 KB stands behind it (reads of 16 rows where there are 8)
    const int front = lists_bytes(p.E, p.T * p.K) + 2048;
    p.ring_bytes = (int)kMaxDynamic - front;
    // the lists are built where the ring will be
    if (2 * p.E * (int)sizeof(int) > p.ring_bytes) return cudaErrorInvalidValue;
    const size_t smem = (size_t)front + (size_t)p.ring_bytes;
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
    if (p.format == MOE_FORMAT_BF16) return launch_t<MOE_FORMAT_BF16>(p, num_sms, st);
    if (p.format == MOE_FORMAT_FP8_E4M3) return launch_t<MOE_FORMAT_FP8_E4M3>(p, num_sms, st);
    return launch_t<MOE_FORMAT_INT8>(p, num_sms, st);
}

}  // namespace moe
