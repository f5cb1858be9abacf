// topk_gate.cu -- the router gate: logits of the experts -> the top-k expert
// ids and weights in the form that dispatch takes.
//
// Operation, per token with logits l_e, e < E, and S = {e : l_e > -inf} (an
// expert whose logit is -inf or NaN is closed to the token):
//   ids[0..K) = the K experts of S with the largest logits, descending, equal
//               logits by ascending expert id; -1 past |S|,
//   softmax:  s_e = exp(l_e - m) / sum_{f in S} exp(l_f - m), m = max over S,
//   sigmoid:  s_e = 1 / (1 + exp(-l_e)),
//   w[k] = scale * s_{ids[k]} (/ sum of the K selected s if renormalised; 0
//          where ids[k] = -1).
// Both scores grow with the logit, so the logits themselves are compared,
// as order-preserving 32-bit integers; the weights are fp32 throughout.
//
// GB300 design: one warp per token, the row in registers (VPL values a
// lane), K rounds of a warp-wide integer maximum (redux.sync) over the
// lanes' own maxima; the winner lane drops its value and looks again.
#include "layer.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;

// Order-preserving key of a logit; 0 for NaN and -inf.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __float_as_uint(__fadd_rn(l, 0.0f));  // -0 becomes +0: equal logits
    const uint32_t k = u ^ (((int32_t)u >> 31) | 0x80000000u);
    return l > -INFINITY ? k : 0u;
}

__device__ __forceinline__ float logit_of(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

template <bool BF16>
__device__ __forceinline__ float load(const void *p, long long i) {
    if (BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(kThreads) topk_gate_kernel(const TopkGateParams p) {
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    for (long long t = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
         t < p.tokens; t += warps) {
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = j * 32 + lane;
            key[j] = e < p.E ? key_of(load<BF16>(p.logits, t * p.row_stride + e)) : 0u;
        }
        float total = 0.0f;  // softmax over the whole row, where it is asked for
        if (!p.sigmoid && !p.renormalize) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) m = max(m, key[j]);
            const float lm = logit_of(__reduce_max_sync(kFull, m));
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const float l = logit_of(key[j]);
                if (key[j] != 0) total += l == lm ? 1.0f : expf(l - lm);
            }
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        }
        uint32_t sel_key = 0;  // lane k holds selection k
        int sel_id = -1;
        for (int k = 0; k < p.K; ++k) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] > best) {
                    best = key[j];
                    at = j;
                }
            const uint32_t m = __reduce_max_sync(kFull, best);
            if (m == 0) break;
            const int id = best == m ? at * 32 + lane : INT32_MAX;
            const int win = __reduce_min_sync(kFull, id);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (j * 32 + lane == win) key[j] = 0;
            if (lane == k) {
                sel_key = m;
                sel_id = win;
            }
        }
        float s = 0.0f;
        const float l0 = logit_of(__shfl_sync(kFull, sel_key, 0));
        if (sel_id >= 0) {
            const float l = logit_of(sel_key);
            // (equal to the maximum: also for +inf, whose difference is NaN)
            s = p.sigmoid ? 1.0f / (1.0f + expf(-l)) : (l == l0 ? 1.0f : expf(l - l0));
        }
        float sum = total;
        if (p.renormalize) {
            sum = s;
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        }
        if ((p.renormalize || !p.sigmoid) && s != 0.0f) s = s / sum;
        if (lane < p.K) {
            p.topk_ids[t * p.K + lane] = sel_id;
            p.topk_w[t * p.K + lane] = s * p.scale;
        }
    }
}

template <int VPL>
cudaError_t launch_t(const TopkGateParams &p, int num_sms, cudaStream_t st) {
    const long long want = (p.tokens + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(want < num_sms * 8LL ? want : num_sms * 8LL);
    if (p.bf16)
        topk_gate_kernel<VPL, true><<<grid, kThreads, 0, st>>>(p);
    else
        topk_gate_kernel<VPL, false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
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
