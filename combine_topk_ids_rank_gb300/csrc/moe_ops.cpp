// moe_ops.cpp -- C entry points of the operators around dispatch and combine
// (include/moe_a2a.h): argument checks on the host, then one launch.
#include "layer.h"

#include "moe_a2a.h"

#include <cuda_runtime.h>

namespace {

using namespace moe;

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A CUDA call failed: clear the runtime's last error, so that the caller's
// next CUDA call does not report it again.
int cuda_failed() {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
}

bool sm_count(int *sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// A launcher's result as a status; nothing is thrown through the C entries.
template <typename Launch>
int launched(Launch &&launch) {
    try {
        return launch() == cudaSuccess ? MOE_OK : cuda_failed();
    } catch (...) {
        return cuda_failed();
    }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t part_bytes(int nmax) {
    return (size_t)kStreamMaxCtas * 2 * (size_t)nmax * 128 * sizeof(float);
}

bool layer_shape_ok(int T, int K, int E, int H, int I) {
    return T >= 0 && T <= kLayerMaxTokens && K >= 1 && K <= MOE_MAX_TOP_K && E >= 1 && E <= 1024 &&
           H >= 16 && H <= MOE_MAX_HIDDEN && H % 16 == 0 && I >= 16 && I <= MOE_MAX_HIDDEN &&
           I % 16 == 0;
}

struct LayerScratch {
    size_t act, y, part, total;
    LayerScratch(int T, int K, int H, int I) {
        const size_t pairs = (size_t)T * K;
        act = kStreamHeaderBytes;
        y = act + up256(pairs * I * 4);
        part = y + up256(pairs * H * 4);
        total = part + part_bytes((T + 15) / 16 * 16);
    }
};

}  // namespace

extern "C" {

int moe_topk_gate(const void *d_logits, int32_t bf16, int64_t tokens, int64_t row_stride,
                  int32_t num_experts, int32_t top_k, int32_t scoring, int32_t renormalize,
                  float scale, int32_t *d_topk_ids, float *d_topk_w, void *stream) {
    if (tokens < 0 || num_experts < 1 || num_experts > kGateMaxExperts || top_k < 1 ||
        top_k > MOE_MAX_TOP_K || top_k > num_experts || row_stride < num_experts ||
        (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID))
        return MOE_ERR_INVALID_ARG;
    if (tokens == 0) return MOE_OK;
    if (d_logits == nullptr || d_topk_ids == nullptr || d_topk_w == nullptr ||
        !aligned(d_logits, bf16 ? 2 : 4) || !aligned(d_topk_ids, 4) || !aligned(d_topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    TopkGateParams p;
    p.logits = d_logits;
    p.topk_ids = d_topk_ids;
    p.topk_w = d_topk_w;
    p.tokens = tokens;
    p.row_stride = row_stride;
    p.E = num_experts;
    p.K = top_k;
    p.bf16 = bf16 != 0;
    p.sigmoid = scoring == MOE_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    return launched([&] { return launch_topk_gate(p, sms, static_cast<cudaStream_t>(stream)); });
}

int moe_quantize_rows_int8(const void *d_x, int32_t bf16, int32_t groups, int32_t rows,
                           int32_t hidden, int64_t row_stride, const int32_t *d_counts,
                           int8_t *d_q, float *d_scale, void *stream) {
    const int vec = bf16 ? 8 : 4;  // elements of a 16-byte load
    if (groups < 0 || rows < 0 || hidden < 8 || hidden > MOE_MAX_HIDDEN || hidden % 8 != 0 ||
        row_stride < hidden || row_stride % vec != 0)
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    if (d_x == nullptr || d_q == nullptr || d_scale == nullptr || !aligned(d_x, 16) ||
        !aligned(d_q, 16) || !aligned(d_scale, 4) || !aligned(d_counts, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    QuantInt8Params p;
    p.x = d_x;
    p.q = d_q;
    p.scale = d_scale;
    p.counts = d_counts;
    p.row_stride = row_stride;
    p.groups = groups;
    p.rows = rows;
    p.H = hidden;
    p.bf16 = bf16 != 0;
    return launched([&] { return launch_quantize_rows_int8(p, sms, static_cast<cudaStream_t>(stream)); });
}

size_t moe_gemm_int8_scratch_bytes(int32_t rows) {
    if (rows < 1) return 0;
    return kStreamHeaderBytes + part_bytes(gemm_int8_nmax(rows));
}

int moe_gemm_int8(const int8_t *d_xq, const float *d_x_scale, const int8_t *d_wq,
                  const float *d_w_scale, const int32_t *d_counts, int32_t groups, int32_t rows,
                  int32_t N, int32_t hidden, void *d_out, void *d_scratch, size_t scratch_bytes,
                  void *stream) {
    if (groups < 0 || groups > kGemmInt8MaxGroups || rows < 0 || N < 1 || hidden < 16 ||
        hidden % 16 != 0 || hidden > kGemmInt8MaxExtent ||
        (int64_t)groups * rows > kGemmInt8MaxExtent || (int64_t)groups * N > kGemmInt8MaxExtent)
        return MOE_ERR_INVALID_ARG;
    if (groups == 0 || rows == 0) return MOE_OK;
    // tiles are counted in 32 bits
    const int64_t tiles = (int64_t)groups * ((N + 127) / 128) *
                          ((rows + gemm_int8_nmax(rows) - 1) / gemm_int8_nmax(rows));
    if (tiles > INT32_MAX / 2) return MOE_ERR_INVALID_ARG;
    if (d_xq == nullptr || d_x_scale == nullptr || d_wq == nullptr || d_w_scale == nullptr ||
        d_out == nullptr || d_scratch == nullptr || !aligned(d_xq, 16) || !aligned(d_wq, 16) ||
        !aligned(d_x_scale, 4) || !aligned(d_w_scale, 4) || !aligned(d_counts, 4) ||
        !aligned(d_out, 2) || !aligned(d_scratch, 256))
        return MOE_ERR_INVALID_ARG;
    if (scratch_bytes < moe_gemm_int8_scratch_bytes(rows)) return MOE_ERR_CAPACITY;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    GemmInt8Params p;
    p.xq = d_xq;
    p.x_scale = d_x_scale;
    p.wq = d_wq;
    p.w_scale = d_w_scale;
    p.counts = d_counts;
    p.out = static_cast<uint16_t *>(d_out);
    p.header = static_cast<StreamHeader *>(d_scratch);
    p.part = reinterpret_cast<float *>(static_cast<char *>(d_scratch) + kStreamHeaderBytes);
    p.G = groups;
    p.M = rows;
    p.N = N;
    p.H = hidden;
    p.nmax = 0;
    return launched([&] { return launch_gemm_int8(p, sms, static_cast<cudaStream_t>(stream)); });
}

size_t moe_layer_small_scratch_bytes(int32_t tokens, int32_t top_k, int32_t hidden,
                                     int32_t inter) {
    if (tokens < 1 || !layer_shape_ok(tokens, top_k, 1, hidden, inter)) return 0;
    return LayerScratch(tokens, top_k, hidden, inter).total;
}

int moe_layer_small(const void *d_x, const int32_t *d_topk_ids, const float *d_topk_w,
                    const void *d_w13, const float *d_w13_scale, const void *d_w2,
                    const float *d_w2_scale, const void *d_residual, int32_t tokens,
                    int32_t top_k, int32_t num_experts, int32_t hidden, int32_t inter,
                    int32_t format, void *d_out, void *d_scratch, size_t scratch_bytes,
                    void *stream) {
    if (!layer_shape_ok(tokens, top_k, num_experts, hidden, inter) ||
        (format != MOE_FORMAT_BF16 && format != MOE_FORMAT_FP8_E4M3 && format != MOE_FORMAT_INT8))
        return MOE_ERR_INVALID_ARG;
    if (tokens == 0) return MOE_OK;
    const bool scaled = format != MOE_FORMAT_BF16;
    if (d_x == nullptr || d_topk_ids == nullptr || d_topk_w == nullptr || d_w13 == nullptr ||
        d_w2 == nullptr || d_out == nullptr || d_scratch == nullptr ||
        (scaled && (d_w13_scale == nullptr || d_w2_scale == nullptr)) || !aligned(d_x, 16) ||
        !aligned(d_topk_ids, 4) || !aligned(d_topk_w, 4) || !aligned(d_w13, 16) ||
        !aligned(d_w2, 16) || !aligned(d_w13_scale, 4) || !aligned(d_w2_scale, 4) ||
        !aligned(d_residual, 8) || !aligned(d_out, 8) || !aligned(d_scratch, 256))
        return MOE_ERR_INVALID_ARG;
    const LayerScratch s(tokens, top_k, hidden, inter);
    if (scratch_bytes < s.total) return MOE_ERR_CAPACITY;
    int sms = 0;
    if (!sm_count(&sms)) return cuda_failed();
    char *mem = static_cast<char *>(d_scratch);
    LayerSmallParams p;
    p.x = static_cast<const uint16_t *>(d_x);
    p.topk_ids = d_topk_ids;
    p.topk_w = d_topk_w;
    p.w13 = d_w13;
    p.w2 = d_w2;
    p.w13_scale = d_w13_scale;
    p.w2_scale = d_w2_scale;
    p.residual = static_cast<const uint16_t *>(d_residual);
    p.out = static_cast<uint16_t *>(d_out);
    p.header = reinterpret_cast<StreamHeader *>(mem);
    p.act = reinterpret_cast<uint16_t *>(mem + s.act);
    p.y = reinterpret_cast<float *>(mem + s.y);
    p.part = reinterpret_cast<float *>(mem + s.part);
    p.T = tokens;
    p.K = top_k;
    p.E = num_experts;
    p.H = hidden;
    p.I = inter;
    p.format = format;
    p.nmax = p.ring_bytes = p.kshift = 0;
    return launched([&] { return launch_layer_small(p, sms, static_cast<cudaStream_t>(stream)); });
}

int moe_scratch_init(void *d_scratch, size_t scratch_bytes, void *stream) {
    if (d_scratch == nullptr || !aligned(d_scratch, 256)) return MOE_ERR_INVALID_ARG;
    if (scratch_bytes < kStreamHeaderBytes) return MOE_ERR_CAPACITY;
    return cudaMemsetAsync(d_scratch, 0, kStreamHeaderBytes, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MOE_OK
               : cuda_failed();
}

int moe_scratch_get_error(void *d_scratch, void *stream, uint32_t *flags) {
    if (d_scratch == nullptr || !aligned(d_scratch, 256)) return MOE_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t f = 0;
    if (cudaMemcpyAsync(&f, &static_cast<StreamHeader *>(d_scratch)->flags, sizeof f,
                        cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return cuda_failed();
    // (a call that gave up may have left its counters behind as well)
    if (f != 0 && (cudaMemsetAsync(d_scratch, 0, kStreamHeaderBytes, st) != cudaSuccess ||
                   cudaStreamSynchronize(st) != cudaSuccess))
        return cuda_failed();
    if (flags != nullptr) *flags = f;
    if (f & MOE_DEVICE_FLAG_WAIT_TIMEOUT) return MOE_ERR_DEVICE_TIMEOUT;
    return f & MOE_DEVICE_FLAG_BAD_EXPERT_ID ? MOE_ERR_ROUTING : MOE_OK;
}

}  // extern "C"
