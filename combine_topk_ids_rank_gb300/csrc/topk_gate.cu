// topk_gate.cu -- the router gate: logits of the experts -> the top-k expert
// ids and weights in the form that dispatch takes.
//
// Operation, per token with logits l_e, e < E, and S = {e : l_e > -inf} (an
// expert whose logit is -inf or NaN is closed to the token):
//   ids[0..K) = the K experts of S with the largest logits, descending, equal
//               logits by ascending expert id; -1 past |S|,
//   softmax:  s_e = exp(l_e - m) / sum_{f in S} exp(l_f - m), m = max over S,
//   sigmoid:  s_e = 1 / (1 + exp(-l_e)), 0 where exp(-l_e) leaves binary64,
//   w[k] = scale * s_{ids[k]} (/ sum of the K selected s if renormalised; 0
//          where ids[k] = -1).
// Both scores grow with the logit, so the logits themselves are compared,
// as order-preserving 32-bit integers; the weights are fp32 throughout.
//
// GB300 design: one warp per token, the row in registers (VPL consecutive
// experts a lane, 16-byte loads), the selection in integers.  K rounds of a
// warp-wide maximum (redux.sync) over the lanes' heads; ties between lanes go
// to the lowest lane, which holds the lowest ids.
// At most 256 experts and top-8, the usual gate: key and id share one word, so a
// lane sorts its values once (a network of 2-instruction exchanges) and a round
// only shifts the winner's list.  Otherwise fp32 keys fill the word; the winner
// lane clears the first value equal to the maximum and looks for its next.
// 32768 tokens x 256 logits, top-8: bf16 10.4 us (its 18.9 MB would take 2.8 us;
// scalar loads and unsorted keys took 29 us, one token a warp 13.5 us), fp32 15.4 us
// from memory, 14.3 us from L2 (its 35.7 MB would take 5.3 us; unsorted whole keys
// took 27.7 us).  fp32 logits that were bf16 before take 19.6 us: a token whose last
// selected logit equals the next one is selected twice, and they have many such.
// The bf16 kernel issues 241 instructions a token, 13 thousand cycles of a scheduler,
// in 62 % of its slots.  The rest is latency: the rounds of a token are one chain of
// dependent reductions, and a warp's tokens go through it one after another.
#include "kernels.h"
#include "layer.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Of a CTA; with 256 the waves are coarser: 9.7 us for 16384 x 256 fp32 logits,
// 8.5 with 128.
constexpr int kThreads = 128;

// The one-launch dispatches read ids and weights, their inputs, before they wait
// for the kernels in front of them.  So this kernel does not let dependents
// start early, and its stores are visible to the device before a CTA is gone.
__device__ __forceinline__ void publish() { __threadfence(); }

// Order-preserving key of a logit; 0 for NaN and -inf.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __float_as_uint(__fadd_rn(l, 0.0f));  // -0 becomes +0: equal logits
    const uint32_t k = u ^ (((int32_t)u >> 31) | 0x80000000u);
    return l > -INFINITY ? k : 0u;
}

__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The lane's VPL logits, experts lane * VPL + j; -inf past E.
template <int VPL, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const TopkGateParams &p, long long t, int lane,
                                         float (&l)[VPL]) {
    const int e0 = lane * VPL;
    if (VEC && e0 + VPL <= p.E) {
        if (BF16) {
            const uint16_t *row = static_cast<const uint16_t *>(p.logits) + t * p.row_stride + e0;
            uint32_t w[(VPL + 1) / 2];
            if constexpr (VPL >= 8) {
#pragma unroll
                for (int j = 0; j < VPL / 8; ++j) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row) + j);
                    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
                }
            } else if constexpr (VPL == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row));
                w[0] = v.x, w[1] = v.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t *>(row));
            }
#pragma unroll
            for (int j = 0; j < VPL / 2; ++j) {
                l[2 * j] = __uint_as_float(w[j] << 16);
                l[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float *row = static_cast<const float *>(p.logits) + t * p.row_stride + e0;
            if constexpr (VPL >= 4) {
#pragma unroll
                for (int j = 0; j < VPL / 4; ++j) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(row) + j);
                    l[4 * j] = v.x, l[4 * j + 1] = v.y, l[4 * j + 2] = v.z, l[4 * j + 3] = v.w;
                }
            } else {
                const float2 v = __ldg(reinterpret_cast<const float2 *>(row));
                l[0] = v.x, l[1] = v.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = e0 + j;
            const long long at = t * p.row_stride + e;
            if (e >= p.E)
                l[j] = -INFINITY;
            else if (BF16)
                l[j] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]);
            else
                l[j] = static_cast<const float *>(p.logits)[at];
        }
    }
}

// The logit of a bf16 key (any low half).
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)) & 0xffff0000u);
}

// exp(v - top), 1 where they are equal (also for +inf, whose difference is NaN)
__device__ __forceinline__ float exp_from(float v, float top) {
    return v == top ? 1.0f : expf(v - top);
}

// 1 / (1 + exp(-v)), times exp(-shift) for v < 0.  A renormalised token whose
// largest logit is negative takes that logit for the shift: its scores are fractions
// of one another, and may all be below what fp32 holds (from -87 down).  What
// binary64 does not hold either counts as 0: exp(-v) past its largest number, exp(709.78).
__device__ __forceinline__ float sigmoid_from(float v, float shift) {
    if (v >= 0.0f) return 1.0f / (1.0f + expf(-v));
    return v < -709.7827f ? 0.0f : expf(v - shift) / (1.0f + expf(v));
}

// Sorts descending.
template <int VPL>
__device__ __forceinline__ void sort_down(uint32_t (&k)[VPL]) {
    auto exchange = [&](int a, int b) {
        const uint32_t hi = max(k[a], k[b]), lo = min(k[a], k[b]);
        k[a] = hi;
        k[b] = lo;
    };
    if constexpr (VPL == 2) {
        exchange(0, 1);
    } else if constexpr (VPL == 4) {
        exchange(0, 1), exchange(2, 3), exchange(0, 2), exchange(1, 3), exchange(1, 2);
    } else {  // Batcher's odd-even merge network for eight, 19 exchanges
        exchange(0, 1), exchange(2, 3), exchange(4, 5), exchange(6, 7);
        exchange(0, 2), exchange(1, 3), exchange(4, 6), exchange(5, 7);
        exchange(1, 2), exchange(5, 6);
        exchange(0, 4), exchange(1, 5), exchange(2, 6), exchange(3, 7);
        exchange(2, 4), exchange(3, 5);
        exchange(1, 2), exchange(3, 4), exchange(5, 6);
    }
}

// The K largest of a warp's whole keys: lane at + k gets the k-th and its id.
template <int VPL>
__device__ __forceinline__ void select_whole(uint32_t (&key)[VPL], int K, int lane, int at,
                                             uint32_t &sel_key, int &sel_id) {
    for (int k = 0; k < K; ++k) {
        uint32_t best = key[0];
#pragma unroll
        for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
        const uint32_t m = __reduce_max_sync(kFull, best);
        if (m == 0) break;
        const int src = __ffs(__ballot_sync(kFull, best == m)) - 1;
        int first = 0;  // the first value equal to the maximum, in the winner lane
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j) first = key[j] == m ? j : first;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane == src && first == j) key[j] = 0;
        const int id = src * VPL + __shfl_sync(kFull, first, src);
        if (lane == at + k) {
            sel_key = m;
            sel_id = id;
        }
    }
}

// N words, from an address that is a multiple of their size (16 bytes at most).
template <int N>
__device__ __forceinline__ void load_words(const void *from, uint32_t (&w)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
            const uint4 v = __ldg(static_cast<const uint4 *>(from) + j);
            w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = __ldg(static_cast<const uint2 *>(from));
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = __ldg(static_cast<const uint32_t *>(from));
    }
}

template <int VPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) topk_gate_kernel(const TopkGateParams p) {
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    for (long long t = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
         t < p.tokens; t += warps) {
        float l[VPL];
        load_row<VPL, BF16, VEC>(p, t, lane, l);
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            key[j] = key_of(l[j]);
            if (BF16 && key[j] != 0)  // the low half is free: lower ids are larger
                key[j] = (key[j] & 0xffff0000u) | (uint32_t)(0xffff - lane * VPL - j);
        }
        float total = 0.0f;  // softmax over the whole row, where it is asked for
        if (!p.sigmoid && !p.renormalize) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < VPL; ++j) m = fmaxf(m, l[j]);  // (drops NaN)
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] != 0) total += l[j] == m ? 1.0f : expf(l[j] - m);
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        }
        uint32_t sel_key = 0;  // lane k holds selection k
        int sel_id = -1;
        constexpr bool kSorted = BF16 && VPL <= 8;
        if constexpr (kSorted) sort_down<VPL>(key);
        if constexpr (BF16) {  // keys are unique
            for (int k = 0; k < p.K; ++k) {
                uint32_t best = key[0];
                if constexpr (!kSorted) {
#pragma unroll
                    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
                }
                const uint32_t m = __reduce_max_sync(kFull, best);
                if (m == 0) break;
                if constexpr (kSorted) {
                    if (best == m) {
#pragma unroll
                        for (int j = 0; j + 1 < VPL; ++j) key[j] = key[j + 1];
                        key[VPL - 1] = 0;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) key[j] = key[j] == m ? 0u : key[j];
                }
                if (lane == k) {
                    sel_key = m | 0xffffu;
                    sel_id = (int)(0xffffu - (m & 0xffffu));
                }
            }
        } else {
            select_whole<VPL>(key, p.K, lane, 0, sel_key, sel_id);
        }
        // (a bf16 key's low half is the sign's: 0 under a positive key, all ones
        // under the complement of a negative one)
        if (BF16 && sel_key >= 0x80000000u) sel_key &= 0xffff0000u;
        float s = 0.0f;
        const float v = logit_of(sel_key), l0 = __shfl_sync(kFull, v, 0);
        if (sel_id >= 0)
            s = p.sigmoid ? sigmoid_from(v, p.renormalize ? fminf(l0, 0.0f) : 0.0f)
                          : exp_from(v, l0);
        float sum = total;
        if (p.renormalize) {
            sum = s;
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        }
        if ((p.renormalize || !p.sigmoid) && s != 0.0f) s = s / sum;
        if (lane < p.K) {
            p.topk_ids[t * p.K + lane] = sel_id;
            p.topk_w[t * p.K + lane] = sel_id >= 0 ? s * p.scale : 0.0f;  // (any scale)
        }
    }
    publish();
}

// At most 256 experts and top-8: NT tokens a warp, whose selections (eight lanes
// a token) are weighted together.  Keys and ids share a word: 16 + 16 bits for
// bf16; for fp32 the key's upper 24 bits and the id, which may put logits that
// agree to 2^-15 in the wrong order.  So the selected logits are read again
// (their weights need them) and compared; a token that has two of them in the
// wrong order, or the last of them no further than 2^-15 from the next one, is
// selected anew on whole keys.
constexpr int kTokens = 4;
// Tokens an SM, up to which a warp takes one: 8 tokens of 256 fp32 logits take
// 2.3 us with one a warp and 3.4 us with four, 2048 3.2 and 4.7 us, 4864 (32 an
// SM) 4.2 and 4.8 us, 9728 7.1 and 6.2 us; bf16 2.0 and 2.8, 2.5 and 3.4, 3.3
// and 3.4, 5.7 and 4.3 us.
constexpr long long kSpread = 32;
template <int VPL, bool BF16, int NT, bool VEC>
__global__ void __launch_bounds__(kThreads) topk_gate_packed_kernel(const TopkGateParams p) {
    static_assert(VPL == 2 || VPL == 4 || VPL == 8, "values a lane");
    constexpr int kWords = BF16 ? VPL / 2 : VPL;       // of a lane's part of a row
    constexpr uint32_t kIdMask = BF16 ? 0xffffu : 0xffu;  // id bits of a packed key
    constexpr int kLooks = BF16 ? 8 : 9;               // rounds that look at the heads
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, e0 = lane * VPL;
    const long long stride = (long long)gridDim.x * (kThreads / 32) * NT;
    // low halves of the bf16 keys, two a word: lower ids are larger
    uint32_t tag[(VPL + 1) / 2];
#pragma unroll
    for (int j = 0; j < VPL / 2; ++j)
        tag[j] = (uint32_t)(0xffff - e0 - 2 * j) | ((uint32_t)(0xffff - e0 - 2 * j - 1) << 16);
    for (long long t0 = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * NT;
         t0 < p.tokens; t0 += stride) {
        uint32_t w[NT][kWords];
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            const long long t = t0 + q < p.tokens ? t0 + q : p.tokens - 1;
            if constexpr (BF16) {
                const uint16_t *row =
                    static_cast<const uint16_t *>(p.logits) + t * p.row_stride + e0;
                if (VEC && e0 + VPL <= p.E) {
                    load_words<kWords>(row, w[q]);
                } else {
#pragma unroll
                    for (int j = 0; j < VPL / 2; ++j) {
                        const uint32_t lo = e0 + 2 * j < p.E ? row[2 * j] : 0xff80u;  // -inf past E
                        const uint32_t hi = e0 + 2 * j + 1 < p.E ? row[2 * j + 1] : 0xff80u;
                        w[q][j] = lo | hi << 16;
                    }
                }
            } else {
                const uint32_t *row =
                    static_cast<const uint32_t *>(p.logits) + t * p.row_stride + e0;
                if (VEC && e0 + VPL <= p.E) {
                    load_words<kWords>(row, w[q]);
                } else {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) w[q][j] = e0 + j < p.E ? row[j] : 0xff800000u;
                }
            }
        }
        uint32_t sel = 0;  // lane 8 q + k: selection k of token q (0: none)
        bool unsure = false;
        float total = 0.0f;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            uint32_t key[VPL];
            float sum = 0.0f;
            const bool whole_row = !p.sigmoid && !p.renormalize;  // softmax over it
            if constexpr (BF16) {
#pragma unroll
                for (int j = 0; j < VPL / 2; ++j) {
                    // order-preserving 16-bit keys of both halves; 0 for NaN and -inf
                    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&w[q][j]);
                    const uint32_t open = __hgt2_mask(x, __float2bfloat162_rn(-INFINITY));
                    x = __hadd2(x, __float2bfloat162_rn(0.0f));  // -0 becomes +0: equal logits
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(&x);
                    uint32_t sign;  // all ones over a negative half (prmt's sign mode)
                    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(sign) : "r"(u));
                    const uint32_t k = (u ^ (sign | 0x80008000u)) & open;
                    key[2 * j] = __byte_perm(k, tag[j], 0x1054);
                    key[2 * j + 1] = __byte_perm(k, tag[j], 0x3276);
                }
                if (whole_row) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) m = max(m, key[j]);
                    const float top = value_of(__reduce_max_sync(kFull, m));
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (key[j] > kIdMask) sum += exp_from(value_of(key[j]), top);
                }
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j) key[j] = key_of(__uint_as_float(w[q][j]));
                if (whole_row) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) m = max(m, key[j]);
                    const float top = logit_of(__reduce_max_sync(kFull, m));
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (key[j] != 0) sum += exp_from(__uint_as_float(w[q][j]), top);
                }
                // (an open expert's key is 0x00800000 at least; a closed one's
                // packed key is its id bits alone)
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    key[j] = (key[j] & ~kIdMask) | (kIdMask - (uint32_t)(e0 + j));
            }
            if (whole_row) {
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                if (lane >> 3 == q) total = sum;
            }
            sort_down<VPL>(key);
#pragma unroll
            for (int k = 0; k < kLooks; ++k) {
                if (k > p.K || (BF16 && k == p.K)) break;
                const uint32_t m = __reduce_max_sync(kFull, key[0]);
                if (k == p.K) {  // the one that comes after the selected ones
                    if (lane == 8 * q + k - 1) unsure = m > kIdMask && (m ^ sel) <= kIdMask;
                    break;
                }
                if (key[0] == m) {
                    // (what is further down than the looks left is not looked at)
#pragma unroll
                    for (int j = 0; j < VPL - 1; ++j)
                        if (j < kLooks - 1 - k) key[j] = key[j + 1];
                    if (VPL - 1 < kLooks - k) key[VPL - 1] = 0;
                }
                if (lane == 8 * q + k) sel = m;
            }
        }
        const int q = lane >> 3, k = lane & 7;
        bool some = sel > kIdMask;
        int id = some ? (int)(kIdMask - (sel & kIdMask)) : -1;
        float v;
        if constexpr (BF16) {
            v = value_of(sel);
        } else {
            const long long t = t0 + q < p.tokens ? t0 + q : p.tokens - 1;
            v = some ? static_cast<const float *>(p.logits)[t * p.row_stride + id] : 0.0f;
            const float after = __shfl_down_sync(kFull, v, 1);
            const uint32_t sel_after = __shfl_down_sync(kFull, sel, 1);
            if (k + 1 < p.K && sel_after > kIdMask && v < after) unsure = true;
            const unsigned again = __ballot_sync(kFull, unsure);
            if (again != 0) {
                for (int r = 0; r < NT; ++r) {
                    if ((again >> (8 * r) & 0xffu) == 0) continue;
                    float l[VPL];
                    uint32_t key[VPL], whole = 0;
                    const long long tr = t0 + r < p.tokens ? t0 + r : p.tokens - 1;
                    load_row<VPL, false, VEC>(p, tr, lane, l);
#pragma unroll
                    for (int j = 0; j < VPL; ++j) key[j] = key_of(l[j]);
                    int found = -1;
                    select_whole<VPL>(key, p.K, lane, 8 * r, whole, found);
                    if (q == r && found >= 0) {  // (as many as there were)
                        id = found;
                        v = logit_of(whole);
                    }
                }
            }
        }
        const float top = __shfl_sync(kFull, v, lane & 24);
        float s = 0.0f;
        if (some)
            s = p.sigmoid ? sigmoid_from(v, p.renormalize ? fminf(top, 0.0f) : 0.0f)
                          : exp_from(v, top);
        if (p.renormalize) {
            total = s;
            for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        }
        if ((p.renormalize || !p.sigmoid) && s != 0.0f) s = s / total;
        if (q < NT && k < p.K && t0 + q < p.tokens) {
            p.topk_ids[(t0 + q) * p.K + k] = id;
            p.topk_w[(t0 + q) * p.K + k] = id >= 0 ? s * p.scale : 0.0f;  // (any scale)
        }
    }
    publish();
}

template <int VPL, bool BF16>
cudaError_t launch_packed(const TopkGateParams &p, bool aligned, int num_sms, cudaStream_t st) {
    const int per = p.tokens > kSpread * num_sms ? kTokens : 1;  // tokens a warp
    const long long want = (p.tokens + per * (kThreads / 32) - 1) / (per * (kThreads / 32));
    const dim3 grid((unsigned)(want < num_sms * 16LL ? want : num_sms * 16LL));
    auto kern = per == 1 ? (aligned ? topk_gate_packed_kernel<VPL, BF16, 1, true>
                                    : topk_gate_packed_kernel<VPL, BF16, 1, false>)
                         : (aligned ? topk_gate_packed_kernel<VPL, BF16, kTokens, true>
                                    : topk_gate_packed_kernel<VPL, BF16, kTokens, false>);
    return launch_pdl(kern, grid, dim3(kThreads), 0, st, p);
}

template <int VPL>
cudaError_t launch_t(const TopkGateParams &p, int num_sms, cudaStream_t st) {
    const long long want = (p.tokens + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(want < num_sms * 16LL ? want : num_sms * 16LL);
    // whole vectors a lane, where every row starts on one
    const uintptr_t vec = VPL * (p.bf16 ? 2 : 4) < 16 ? VPL * (p.bf16 ? 2 : 4) : 16;
    const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % vec == 0 &&
                         (uintptr_t)(p.row_stride * (p.bf16 ? 2 : 4)) % vec == 0;
    if constexpr (VPL <= 8) {
        if (p.K <= 8)
            return p.bf16 ? launch_packed<VPL, true>(p, aligned, num_sms, st)
                          : launch_packed<VPL, false>(p, aligned, num_sms, st);
    }
    auto kern = p.bf16 ? (aligned ? topk_gate_kernel<VPL, true, true>
                                  : topk_gate_kernel<VPL, true, false>)
                       : (aligned ? topk_gate_kernel<VPL, false, true>
                                  : topk_gate_kernel<VPL, false, false>);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), 0, st, p);
}

}  // namespace

cudaError_t launch_topk_gate(const TopkGateParams &p, int num_sms, cudaStream_t st) {
    if (p.E < 1 || p.E > kGateMaxExperts || p.K < 1 || p.K > 32) return cudaErrorInvalidValue;
    if (p.E <= 64) return launch_t<2>(p, num_sms, st);
    if (p.E <= 128) return launch_t<4>(p, num_sms, st);
    if (p.E <= 256) return launch_t<8>(p, num_sms, st);
    if (p.E <= 512) return launch_t<16>(p, num_sms, st);
    return launch_t<32>(p, num_sms, st);
}

}  // namespace moe
