// ring.h -- the rings of the persistent products (gemm_int8.cu): what they
// hold, and the order in which a widening warp waits on them.  Plain C++, so
// that the host can go through the rule (tests/test_moe_rings.py).
// Internal to libmoe_a2a.so.
//
// A stage holds a unit's 8-bit rows as TMA brought them, a place what they
// were widened to; unit n uses stage n mod S and place n mod U.  The widening
// warps form groups that take the units in turn, so the unit that used a stage
// before (n - S) may be another group's.
//
// A wait on a barrier's parity tells "this phase is over" from "this phase is
// running", but not from "the phase before is running": it is only good once
// the phase before is known to be over.  Loads of different units land in any
// order.  So a warp waits for the place first.  Place n mod U is free when unit
// n - U was multiplied; the products run in order, so all units up to n - U
// have landed, and with S >= U unit n - S is among them: the stage's phase is
// now the one of unit n.  (For the place's own wait the phase before is that of
// unit n - 2U: multiplied, since the warp's last unit, n - 2, waited for n - 2 - U.)
#pragma once

#ifdef __CUDACC__
#define MOE_RING_FN __host__ __device__ __forceinline__
#else
#define MOE_RING_FN inline
#endif

namespace moe {
namespace ring {

constexpr int kTurns = 2;  // groups of widening warps that take the units in turn

// True when unit n's rows are there and its place is free; `place` and `stage`
// wait with a time limit and return false when it runs out.
template <typename Place, typename Stage>
MOE_RING_FN bool widen_ready(const Place &place, const Stage &stage) {
    return place() && stage();
}

// What widen_ready needs of S stages and U places.
MOE_RING_FN constexpr bool order_holds(int stages, int places) {
    return places >= kTurns && stages >= places;
}

// ---- 8-bit product ------------------------------------------------------------

constexpr int kGemmRowBytes = 128;              // codes of a row in a unit
constexpr int kGemmWeightBytes = 128 * kGemmRowBytes;
constexpr int kGemmMaxStages = 12, kGemmMaxUnits = 4;
// dynamic shared memory: 227 KB a CTA less the static tables
constexpr int kGemmDynamic = (227 - 15) * 1024;

struct Gemm {
    int nmax;      // tokens of a tile, at most
    int box;       // rows of a token TMA box
    int stages;    // raw stages: 128 weight rows + nmax / 2 token rows of 128 codes
    int units;     // widened units: a weight tile in tensor memory, and nmax / 2 token
                   // rows of 128 f16, as two tiles of 64, in shared memory
};

// The rings of tiles of at most `nmax` tokens (16 .. 256, a power of two).
inline Gemm gemm(int nmax) {
    Gemm r;
    const int half = nmax / 2 * kGemmRowBytes;
    r.nmax = nmax;
    r.box = nmax / 2 < 32 ? nmax / 2 : 32;
    r.units = nmax > 128 ? 3 : kGemmMaxUnits;
    r.stages = (kGemmDynamic - 1024 - 2 * r.units * half) / (kGemmWeightBytes + half);
    if (r.stages > kGemmMaxStages) r.stages = kGemmMaxStages;
    return r;
}

// Dynamic shared memory that they take (1 KB aligns them).
inline int gemm_bytes(const Gemm &r) {
    const int half = r.nmax / 2 * kGemmRowBytes;
    return 1024 + r.stages * (kGemmWeightBytes + half) + 2 * r.units * half;
}

}  // namespace ring
}  // namespace moe
