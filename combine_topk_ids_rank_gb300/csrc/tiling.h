// tiling.h -- how the experts' products (expert_product.cuh) divide their groups
// into tiles.  Plain C++, so that the host can go through the rules
// (tests/test_moe_tiling.py).  Internal to libmoe_a2a.so.
#pragma once

#include <climits>

#ifdef __CUDACC__
#define MOE_TILING_FN __host__ __device__ __forceinline__
#else
#define MOE_TILING_FN inline
#endif

namespace moe {
namespace product {

enum Op { kFp8, kFp8Narrow, kForward, kInputGrad, kWeightGrad };
constexpr bool is_fp8(Op op) { return op == kFp8 || op == kFp8Narrow; }
constexpr int ctas_of(Op op) { return is_fp8(op) ? 1 : 2; }

constexpr int kTileLanes = 128;  // of a CTA
constexpr int kTileCols = 256;   // at most

// Columns of the `k` tiles of `cols` columns: evened out, a multiple of 16.
MOE_TILING_FN int width_of(int cols, int k) {
    return k <= 1 ? (cols + 15) / 16 * 16 : ((cols + k - 1) / k + 15) / 16 * 16;
}

// How groups are divided into tiles.
template <Op OP>
struct Shape {
    static constexpr int kLanes = ctas_of(OP) * kTileLanes;
    int turn_from;  // tokens that make a group's tiles turned
    int shift;      // columns of a tile that is not, at most: 1 << shift
    int even;       // tiles of a group are evened out (else: full ones and what is left)
    int thin;       // kFp8Narrow: a tile has 64 lanes only, so that few are cut

    MOE_TILING_FN bool turned(int c) const { return OP == kFp8 && c >= turn_from; }
    // Tiles along the channels, and along `c` tokens (or the maps' columns).
    MOE_TILING_FN int ltiles(int c, int lanes) const {
        const int l = turned(c) ? kTileCols : (OP == kFp8Narrow && thin ? 64 : kLanes);
        return (lanes + l - 1) / l;
    }
    MOE_TILING_FN int mtiles(int c) const {
        return turned(c) ? (c + kTileLanes - 1) / kTileLanes : (c + (1 << shift) - 1) >> shift;
    }
    // Columns of a tile, and the tokens (or columns) from one tile to the next.
    MOE_TILING_FN int width(int c) const {
        if (turned(c)) return kTileCols;
        return even ? width_of(c, mtiles(c)) : (c < 1 << shift ? c : 1 << shift);
    }
    MOE_TILING_FN int stride(int c) const { return turned(c) ? kTileLanes : width(c); }
    MOE_TILING_FN int tiles(int c, int lanes) const { return mtiles(c) * ltiles(c, lanes); }
};

// Tiles of all groups: as `shape` has them, and along the tokens with 128, 64 and 32 columns.
template <Op OP>
MOE_TILING_FN void add_tiles(int (&sums)[4], const Shape<OP> &shape, int c, int wide, int lanes) {
    sums[0] += shape.tiles(wide, lanes);
    for (int i = 1; i < 4; ++i) sums[i] += (c + (128 >> (i - 1)) - 1) >> (8 - i);
}

// Offsets that descend may repeat rows, and so count more tiles than 32 bits hold (others
// stay below the host's limit): whether `groups` groups of `rows` rows could.
template <Op OP>
MOE_TILING_FN bool could_repeat_too_many(const Shape<OP> &shape, int groups, int rows, int lanes) {
    return OP != kWeightGrad && (long long)groups * shape.tiles(rows, lanes) >= 1 << 29;
}

// The tiles of a call from those sums, over `pairs` pairs of CTAs (CTAs); narrower ones
// where they are few.  `repeats`: could_repeat_too_many, and the offsets do descend; then
// the sums may have wrapped, none is looked at, and there is no work at all.
template <Op OP>
MOE_TILING_FN int settle(Shape<OP> &shape, const int (&sums)[4], bool repeats, int pairs,
                         int lanes) {
    if (repeats) return 0;
    int tiles = sums[0];
    // Few tiles: narrower ones while each still finds an idle pair (333 x 1000 x 1040 in
    // 8 bits: 12 turned tiles of nine blocks, or 56 of 48 columns).
    if (OP != kWeightGrad && tiles * 2 <= pairs) {
        const int l = (lanes + Shape<OP>::kLanes - 1) / Shape<OP>::kLanes;
        for (int i = 1; i < 4; ++i)
            if (sums[i] * l <= pairs) {
                shape.turn_from = INT_MAX;
                shape.shift = 8 - i;
                tiles = sums[i] * l;
            }
    }
    // 8-bit, fewer tiles than half the SMs: of 64 lanes instead of cut ones (one SM can
    // take more than its share of the memory's rate, and no part goes through memory;
    // 16 x 7168 x 4096: 13.0 us, 14.3 with 128 lanes)
    if (OP == kFp8Narrow && tiles * 2 <= pairs) {
        shape.thin = 1;
        tiles = sums[8 - shape.shift] * ((lanes + 63) / 64);
    }
    return tiles;
}

}  // namespace product
}  // namespace moe
