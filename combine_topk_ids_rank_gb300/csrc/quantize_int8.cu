// quantize_int8.cu -- activation rows to 8-bit integer codes with one scale
// per row, the token operand of the 8-bit integer product.
//
// Operation, per row x[0..H) (bf16 or fp32):
//   amax = max_h |x_h|,  scale = max(RN32(amax / 127), 2^-126), 1 if amax = 0,
//   q_h  = the integer nearest to RN32(x_h / scale), ties to even: |q_h| <= 127.
// A row that holds a NaN or an infinity has scale NaN and zero codes, so
// whatever is computed from it is NaN.  With counts, rows j >= counts[g] of
// plane g are neither read nor written.
//
// The quotients come from one reciprocal per row and remainder steps (fp8.cuh
// explains them): two steps, which give the correctly rounded x / scale, for
// fp32 rows; for bf16 rows one step, which leaves the same nearest integer for
// every pair of a bf16 maximum and a bf16 value (there are 128 x 128 pairs of
// significands and nine binades in which a code is not zero; the tests go
// through all of them).  The rounding to an integer adds and keeps 1.5 * 2^23,
// whose neighbours are one apart.
//
// Memory bound: each element is read once and its code written once.  One
// CTA a row, the row in registers, 16 bytes a thread and load, the next row's
// loads in flight (without them 198 us).  32768 bf16 rows of 7168 take 108 us,
// 6.5 TB/s; with two remainder steps and a quarter of the threads idle in the
// last vector 127 us.  As fp32 rows they take 180 us, 6.5 TB/s.  With counts a CTA
// steps over the rows that are not in use: 32 planes of 1024 x 7168 bf16 take 114 us
// full, 50 us a third full (35 at the copy rate) and 18 us with 16 rows each.
#include "fp8.cuh"
#include "kernels.h"
#include "layer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxWarps = 8;

__device__ __forceinline__ fp8::RowScale int8_scale(float amax) {
    fp8::RowScale r;
    r.s = amax > 0.0f ? fmaxf(__fdiv_rn(amax, 127.0f), 0x1p-126f) : 1.0f;
    r.m = r.s < 0x1p-100f ? 0x1p100f : (r.s > 0x1p100f ? 0x1p-100f : 1.0f);
    r.sd = __fmul_rn(r.s, r.m);
    r.y = __frcp_rn(r.sd);
    return r;
}

// The low byte of each word: the nearest integers to a / s and b / s.
template <bool SCALED, bool BF16>
__device__ __forceinline__ void code2(float a, float b, const fp8::RowScale &r, uint32_t &ca,
                                      uint32_t &cb) {
    x2::f2 xs = x2::pack(a, b);
    if (SCALED) xs = x2::mul(xs, x2::pack(r.m, r.m));
    const x2::f2 y = x2::pack(r.y, r.y), nsd = x2::pack(-r.sd, -r.sd);
    x2::f2 q = x2::mul(xs, y);
    q = x2::fma(x2::fma(q, nsd, xs), y, q);
    if (!BF16) q = x2::fma(x2::fma(q, nsd, xs), y, q);
    q = x2::add(q, x2::pack(12582912.0f, 12582912.0f));
    float fa, fb;
    x2::unpack(q, fa, fb);
    ca = __float_as_uint(fa);
    cb = __float_as_uint(fb);
}

template <bool SCALED, bool BF16>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const fp8::RowScale &r) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        code2<SCALED, BF16>(v[2 * i], v[2 * i + 1], r, c[2 * i], c[2 * i + 1]);
    uint2 o;
    o.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    return o;
}

// Eight elements of a row as loaded: one 16-byte vector of bf16, two of fp32.
template <bool BF16>
struct Vec8 {
    uint4 v[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const uint4 *row, int i) {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) v[k] = __ldcs(row + i * (BF16 ? 1 : 2) + k);
    }
    // bits of the largest |x| (NaN above infinity above every number)
    __device__ __forceinline__ uint32_t most() const {
        if (BF16) {  // two 16-bit lanes at a time
            const uint32_t k = 0x7fff7fffu;
            const uint32_t a = __vmaxu2(__vmaxu2(v[0].x & k, v[0].y & k),
                                        __vmaxu2(v[0].z & k, v[0].w & k));
            return max(a << 16, a & 0xffff0000u);
        } else {
            const uint32_t k = 0x7fffffffu;
            const uint32_t a = max(max(v[0].x & k, v[0].y & k), max(v[0].z & k, v[0].w & k));
            const uint4 w = v[BF16 ? 0 : 1];
            return max(a, max(max(w.x & k, w.y & k), max(w.z & k, w.w & k)));
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        if (BF16) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint4 b = v[BF16 ? 0 : 1];
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        }
    }
};

// One CTA a row; thread i takes the 8-element vectors i, i + threads, ...  The
// next row's loads are in flight while this row is reduced and stored.
template <int VPT, bool BF16>
__global__ void __launch_bounds__(kMaxWarps * 32) quantize_int8_kernel(const QuantInt8Params p) {
    __shared__ uint32_t red[2][kMaxWarps];
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x, nt = blockDim.x, H8 = p.H / 8;
    const long long total = (long long)p.groups * p.rows;
    // the first row from r on that is in use (the whole CTA alike)
    auto used = [&](long long r) {
        if (p.counts == nullptr) return r;
        for (; r < total; r += gridDim.x) {
            const long long g = r / p.rows;
            if (r - g * p.rows < __ldg(p.counts + g)) break;
        }
        return r;
    };
    auto load = [&](Vec8<BF16> (&x)[VPT], long long r) {
        const uint4 *row = reinterpret_cast<const uint4 *>(
            static_cast<const char *>(p.x) + r * p.row_stride * (BF16 ? 2 : 4));
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (tid + j * nt < H8) x[j].load(row, tid + j * nt);
    };
    Vec8<BF16> next[VPT];
    long long r = used(blockIdx.x);
    if (r < total) load(next, r);
    for (int turn = 0; r < total; turn ^= 1) {
        Vec8<BF16> x[VPT];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (tid + j * nt < H8) {
                x[j] = next[j];
                m = max(m, x[j].most());
            }
        const long long after = used(r + gridDim.x);
        if (after < total) load(next, after);
        m = __reduce_max_sync(kFull, m);
        if ((tid & 31) == 0) red[turn][tid >> 5] = m;
        __syncthreads();
        for (int w = 0; w < nt / 32; ++w) m = max(m, red[turn][w]);
        const bool finite = m < 0x7f800000u;
        const fp8::RowScale s = int8_scale(finite ? __uint_as_float(m) : 0.0f);
        uint2 *q = reinterpret_cast<uint2 *>(p.q + r * p.H);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = tid + j * nt;
            if (v < H8) {
                float f[8];
                x[j].values(f);
                uint2 o = make_uint2(0, 0);
                if (finite) o = s.m == 1.0f ? codes8<false, BF16>(f, s) : codes8<true, BF16>(f, s);
                q[v] = o;
            }
        }
        if (tid == 0) p.scale[r] = finite ? s.s : __uint_as_float(0x7fc00000u);
        r = after;
    }
}

template <int VPT>
cudaError_t launch_t(const QuantInt8Params &p, int threads, int num_sms, cudaStream_t st) {
    const long long total = (long long)p.groups * p.rows;
    const long long most = (long long)num_sms * 16;
    const unsigned grid = (unsigned)(total < most ? total : most);
    return launch_pdl(p.bf16 ? quantize_int8_kernel<VPT, true> : quantize_int8_kernel<VPT, false>,
                      dim3(grid), dim3(threads), 0, st, p);
}

}  // namespace

cudaError_t launch_quantize_rows_int8(const QuantInt8Params &p, int num_sms, cudaStream_t st) {
    if (p.H % 8 != 0 || p.H < 8 || p.H > 16384) return cudaErrorInvalidValue;
    const int H8 = p.H / 8;
    // as many vectors a thread as 256 threads need, then as few threads as those need
    int vpt = (H8 + kMaxWarps * 32 - 1) / (kMaxWarps * 32);
    vpt = vpt <= 2 ? vpt : (vpt <= 4 ? 4 : 8);
    const int threads = ((H8 + vpt - 1) / vpt + 31) / 32 * 32;
    if (vpt == 1) return launch_t<1>(p, threads, num_sms, st);
    if (vpt == 2) return launch_t<2>(p, threads, num_sms, st);
    if (vpt == 4) return launch_t<4>(p, threads, num_sms, st);
    return launch_t<8>(p, threads, num_sms, st);
}

}  // namespace moe
