// ring.h -- the rings of the persistent products (gemm_int8.cu, layer_small.cu):
// what they hold, and the order in which a widening warp waits on them.  Plain
// C++, so that the host can go through the rule (tests/test_moe_rings.py).
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

// ---- layer for a few tokens -----------------------------------------------------

constexpr int kLayerSlots = 4;        // places: widened weight tiles in tensor memory
constexpr int kLayerMaxStages = 16;
constexpr int kLayerMinStages = 2;
// dynamic shared memory: 227 KB a CTA less the static barriers
constexpr int kLayerDynamic = (227 - 2) * 1024;

// Bytes of the lists of E experts and P pairs (token, k), in front of the stages.
MOE_RING_FN constexpr int layer_list_bytes(int E, int P) {
    const int P8 = (P + 7) / 8 * 8;
    return (P8 * 2 + P * 4 + E * 4 + E * 2 + (E < P ? E : P) * 4 + 2 + P * 4 + 15) / 16 * 16;
}

// Bytes in front of the stages and behind them: 1 KB aligns the ring and 1 KB
// stands behind it (reads of 16 rows where there are 8).
MOE_RING_FN constexpr int layer_front_bytes(int E, int P) { return layer_list_bytes(E, P) + 2048; }
MOE_RING_FN constexpr int layer_ring_bytes(int E, int P) {
    return kLayerDynamic - layer_front_bytes(E, P);
}

// Token rows of a stage, twice: the halves of 64 columns in phase 0, the two
// terms of the activations in phase 1.
MOE_RING_FN constexpr int layer_half_bytes(int rows) { return (rows + 7) / 8 * 8 * 2 * 128; }

// Stages of 128 weight rows (128 columns of `value_bytes` each) and the token rows of
// an expert of `rows` pairs.
MOE_RING_FN constexpr int layer_stage_bytes(int value_bytes, int rows) {
    return 128 * 128 * value_bytes + 2 * layer_half_bytes(rows);
}
MOE_RING_FN constexpr int layer_stages(int ring_bytes, int value_bytes, int rows) {
    const int n = ring_bytes / layer_stage_bytes(value_bytes, rows);
    return n < kLayerMaxStages ? n : kLayerMaxStages;
}

// Whether a ring of `stages` serves: 8-bit weights (value_bytes 1) are widened.
MOE_RING_FN constexpr bool layer_holds(int value_bytes, int stages) {
    return stages >= kLayerMinStages && (value_bytes != 1 || order_holds(stages, kLayerSlots));
}

}  // namespace ring
}  // namespace moe
