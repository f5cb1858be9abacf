// stream.cuh -- what the two persistent products that stream weights through
// the tensor cores share (layer_small.cu, gemm_int8.cu; the split and the merge
// also expert_product.cuh): the even split of
// the k-blocks of all output tiles over the CTAs, the widening of 8-bit
// weight rows into tensor memory, and waits on counters in global memory.
//
// Orientation.  The weights are the A operand: 128 output channels a tile
// are the 128 tensor-memory lanes, and the tokens are the columns (N), as
// few as the group has (a multiple of 16).  So a tile costs what its weight
// bytes cost, whatever the number of tokens.
//
// Split.  Tiles x k-blocks ("units") form one line that is cut into equal
// ranges, one per CTA, wherever the cuts fall.  A tile cut between CTAs is
// summed by the CTA that finishes its part last, over the parts in ascending
// k: the order of the additions does not depend on timing.
#pragma once

#include <cstdint>

#include "layer.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace stream {

constexpr int kTileRows = 128;   // output channels of a tile
constexpr int kBlockK = 128;     // k extent of a unit
constexpr int kAtom = 128;       // bytes of a shared-memory row (128-byte swizzle)
constexpr uint64_t kWaitNs = 500ull * 1000 * 1000;  // 0.5 s of wall time per wait

// Units cut into `parts` ranges at multiples of `grain` units: the first
// `more` parts have q + 1 grains, the others q >= 1.
struct Cut {
    int parts, grain, q, more;
    __device__ Cut(int grains, int parts_, int grain_) : parts(parts_), grain(grain_) {
        q = parts ? grains / parts : 0;
        more = parts ? grains - q * parts : 0;
    }
    __device__ int first(int c) const { return (c * q + min(c, more)) * grain; }
    // the part that holds unit u
    __device__ int of(int u) const {
        const int g = u / grain, big = more * (q + 1);
        return g < big ? g / (q + 1) : more + (g - big) / q;
    }
};

// `tiles` of `blocks` units over the CTAs: cut anywhere, or between tiles only.
// Cutting inside tiles evens out the CTAs' work but adds the parts' way
// through memory, about `merge` units' time.  SHARED: the memory's rate is the
// bound, and a CTA alone can do 1.5 times its even share of the work in the
// same time, so some CTAs may idle before whole tiles cost anything.
template <bool SHARED>
__device__ __forceinline__ Cut cut(int tiles, int blocks, int ctas, int merge) {
    const int total = tiles * blocks, rounds = (tiles + ctas - 1) / ctas;
    const int even = (total + ctas - 1) / ctas;
    const int whole = max(SHARED ? rounds * blocks * 2 / 3 : rounds * blocks, even);
    if (whole <= even + merge || total < ctas) return Cut(tiles, min(tiles, ctas), blocks);
    return Cut(total, ctas, 1);
}

// A run of units of one tile: k-blocks [k0, k1) of tile `tile`.
struct Segment {
    int tile, k0, k1;
};

// The segments of CTA c in ascending order; `blocks` k-blocks a tile.
struct Segments {
    int u, end, blocks;
    __device__ Segments(const Cut &ct, int c, int blocks_) : u(0), end(0), blocks(blocks_) {
        if (c < ct.parts) {
            u = ct.first(c);
            end = ct.first(c + 1);
        }
    }
    __device__ bool next(Segment &s) {
        if (u >= end) return false;
        s.tile = u / blocks;
        s.k0 = u - s.tile * blocks;
        s.k1 = min(s.k0 + end - u, blocks);
        u += s.k1 - s.k0;
        return true;
    }
};

// Parts of tile t: CTAs [c0, c1]; the part of CTA c is kept in slot 0 if it
// begins that CTA's range, else in slot 1.
struct Parts {
    int c0, c1, slot0;
    Parts() = default;
    __device__ Parts(const Cut &ct, int tile, int blocks) {
        const int a = tile * blocks;
        c0 = ct.of(a);
        c1 = ct.of(a + blocks - 1);
        slot0 = ct.first(c0) == a ? 0 : 1;
    }
    __device__ int slot(int c) const { return c == c0 ? slot0 : 0; }
    __device__ int count() const { return c1 - c0 + 1; }
};

__device__ __forceinline__ int ld_acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Position in a ring of `size` barriers that a role walks through: the index
// and the parity of the phase that the role's next use of it completes.
struct Turn {
    uint32_t at, parity, size;
    __device__ explicit Turn(uint32_t size_) : at(0), parity(0), size(size_) {}
    __device__ void next() {
        if (++at == size) {
            at = 0;
            parity ^= 1u;
        }
    }
};

// Wait until *p reaches `want` (it only grows meanwhile); false on timeout or
// when another role of this CTA has failed.
__device__ __forceinline__ bool wait_count(const int *p, int want, volatile int *failed) {
    if (ld_acquire(p) >= want) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (ld_acquire(p) >= want) return true;
        if (*failed || ptx::globaltimer_ns() - t0 > kWaitNs) return false;
    }
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(
                     ptx::smem_u32(bar))
                 : "memory");
}

// Barrier 1 of the 128 epilogue threads.
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// A flag in shared memory, read alike by all lanes of a warp.
__device__ __forceinline__ bool warp_flag(const volatile int *f) {
    return __any_sync(0xffffffffu, *f != 0);
}

// ---- four 8-bit codes -> four 16-bit values (two words, ascending) -----------

// int8 -> bf16, exact up to the power of two kInt8Bf16: a 16-bit lane that
// holds the integer u = code + 128, read as bf16, is u * 2^-133 for all of
// 0..255 (bf16's subnormals run on into its smallest normals), so one fused
// multiply-add by 2^127 gives code * 2^-6.
constexpr float kInt8Bf16 = 64.0f;  // what the sums are multiplied by in turn
__device__ __forceinline__ void int8_to_bf16(uint32_t v, uint32_t &a, uint32_t &b) {
    const uint32_t u = v ^ 0x80808080u;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(a) : "r"(__byte_perm(u, 0, 0x4140)), "r"(0x7f007f00u), "r"(0xc000c000u));  // - 2
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(b) : "r"(__byte_perm(u, 0, 0x4342)), "r"(0x7f007f00u), "r"(0xc000c000u));
}

// int8 -> f16, exact: code + 128 rides on 1024 (0x6400, one unit apart).
__device__ __forceinline__ void int8_to_f16(uint32_t v, uint32_t &a, uint32_t &b) {
    const uint32_t u = v ^ 0x80808080u;
    const uint32_t ua = __byte_perm(u, 0x64646464u, 0x5140), ub = __byte_perm(u, 0x64646464u, 0x7362);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(ua), "r"(0x64806480u));  // 1152
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(ub), "r"(0x64806480u));
}

// e4m3 -> bf16, exact, through f16 and fp32 (NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two_codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c, l, h;\n\t.reg .b32 p;\n\t.reg .f32 x, y;\n\t"
        "cvt.u16.u32 c, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, c;\n\t"
        "mov.b32 {l, h}, p;\n\t"
        "cvt.f32.f16 x, l;\n\t"
        "cvt.f32.f16 y, h;\n\t"
        "cvt.rn.bf16x2.f32 %0, y, x;\n\t}"
        : "=r"(r)
        : "r"(two_codes));
    return r;
}
__device__ __forceinline__ void e4m3_to_bf16(uint32_t v, uint32_t &a, uint32_t &b) {
    a = e4m3_pair(v);
    b = e4m3_pair(v >> 16);
}

}  // namespace stream
}  // namespace moe
