"""How the experts' products divide their groups into tiles, on the host: csrc/tiling.h
against the same counts in Python's integers, offsets that descend among them."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include "tiling.h"
using namespace moe::product;
// out: tiles, columns of a tile (a power of two), turned tiles, thin tiles
template <Op OP>
void plan(int groups, int rows, const int *offsets, int lanes, int pairs, int *out) {
    Shape<OP> s;
    s.turn_from = OP == kFp8 && lanes % 8 == 0 ? 33 : INT_MAX;
    s.shift = is_fp8(OP) ? 7 : 8;
    s.even = 1;
    s.thin = 0;
    int sums[4] = {0, 0, 0, 0};
    bool down = false;
    for (int g = 0; g < groups; ++g) {
        const int a = offsets[g] < 0 ? 0 : offsets[g] > rows ? rows : offsets[g];
        int b = offsets[g + 1] < a ? a : offsets[g + 1];
        if (b > rows) b = rows;
        down = down || offsets[g + 1] < offsets[g];
        add_tiles(sums, s, b - a, b - a, lanes);
    }
    const bool repeats = could_repeat_too_many(s, groups, rows, lanes) && down;
    out[0] = settle(s, sums, repeats, pairs, lanes);
    out[1] = 1 << s.shift;
    out[2] = s.turn_from != INT_MAX;
    out[3] = s.thin;
}
extern "C" void plan_of(int op, int groups, int rows, const int *offsets, int lanes, int pairs,
                        int *out) {
    if (op == 0) plan<kFp8>(groups, rows, offsets, lanes, pairs, out);
    if (op == 1) plan<kFp8Narrow>(groups, rows, offsets, lanes, pairs, out);
    if (op == 2) plan<kForward>(groups, rows, offsets, lanes, pairs, out);
    if (op == 3) plan<kInputGrad>(groups, rows, offsets, lanes, pairs, out);
}
"""

FP8, NARROW, FORWARD, INPUT_GRAD = range(4)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("tiling")
    src, so = str(d / "tiling.cpp"), str(d / "tiling.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    # (sums that wrap do so as the device's)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "combine_topk_ids_rank_gb300", "csrc"), src,
                    "-o", so], check=True)
    return ctypes.CDLL(so)


def run(lib, op, rows, offsets, lanes):
    pairs = 152 if op in (FP8, NARROW) else 76
    out = (ctypes.c_int * 4)()
    lib.plan_of(op, len(offsets) - 1, rows, (ctypes.c_int * len(offsets))(*offsets), lanes, pairs,
                out)
    return pairs, tuple(out)


def up(a, b):
    return -(-a // b)


def counted(op, rows, offsets, lanes, cols, turned, thin):
    """Tiles of all groups of such a shape, without a limit."""
    total = 0
    for a, b in zip(offsets, offsets[1:]):
        a = min(max(a, 0), rows)
        c = min(max(b, a), rows) - a
        if turned and c >= 33:
            total += up(c, 128) * up(lanes, 256)
        else:
            total += up(c, cols) * up(lanes, 64 if thin else 128 if op in (FP8, NARROW) else 256)
    return total


def check(lib, op, rows, offsets, lanes):
    """The shape that is chosen has the tiles that are counted, few of them if it is a
    narrow one; none at all where repeated rows could count more than 32 bits."""
    G = len(offsets) - 1
    widest = 128 if op in (FP8, NARROW) else 256
    most = counted(op, rows, [0, rows], lanes, widest, op == FP8 and lanes % 8 == 0, 0)
    pairs, (tiles, cols, turned, thin) = run(lib, op, rows, offsets, lanes)
    if G * most >= 1 << 29 and any(b < a for a, b in zip(offsets, offsets[1:])):
        assert tiles == 0
        return
    assert tiles == counted(op, rows, offsets, lanes, cols, turned, thin)
    assert 0 <= tiles < 1 << 30
    if cols < widest or thin:
        assert tiles <= pairs


# every other group has all rows
def alternating(groups, rows):
    return [rows if g % 2 else 0 for g in range(groups + 1)]


@pytest.mark.parametrize("op,rows,offsets,lanes", [
    # tiles of 32 columns that wrap to -2^31, to 0 and to 12 (two of the sums do)
    (FORWARD, 1 << 27, alternating(1024, 1 << 27), 1),
    (FORWARD, 1 << 28, alternating(1024, 1 << 28), 8),
    (FORWARD, (1 << 28) + 1, [0] + [1 << 28, 0] * 500 + [(1 << 28) + 1, 0] * 12, 8),
    (INPUT_GRAD, (1 << 28) + 1, [0] + [1 << 28, 0] * 500 + [(1 << 28) + 1, 0] * 12, 8),
    # wide maps: the product with the tiles along the channels wraps
    (FORWARD, (1 << 24) + 32, [0] + [(1 << 24) + 32, 0] * 2 + [1 << 24, 0] * 510, 4096),
    # 8-bit rows of few tokens on average: tiles of 64 channels
    (NARROW, 48000, alternating(1024, 48000), 200000),
    (NARROW, 48000, alternating(1024, 48000), 180000),
    (FP8, 1 << 22, alternating(1024, 1 << 22), 4096),
])
def test_descending_offsets_that_count_too_many_tiles_give_none(lib, op, rows, offsets, lanes):
    assert run(lib, op, rows, offsets, lanes)[1][0] == 0
    check(lib, op, rows, offsets, lanes)


@pytest.mark.parametrize("op", [FP8, NARROW, FORWARD, INPUT_GRAD])
def test_tiles_of_the_chosen_shape(lib, op):
    rng = random.Random(op)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    for i in range(3000):
        G = min(1024, log(1, 1100))
        rows, lanes = log(1, 1 << 29), log(1, 1 << 20)
        # (what the entry points take)
        if G * lanes >= 2 ** 31 - 2 ** 24 or up(lanes, 128) * (rows // 128 + G) >= 2 ** 30:
            continue
        offsets = sorted(rng.randrange(rows + 1) for _ in range(G + 1))
        if rng.random() < 0.3:          # a few rows only
            offsets = [o % min(rows + 1, 40) for o in offsets]
        if i % 3 == 0:
            rng.shuffle(offsets)
        elif i % 3 == 1:
            offsets.sort()
        check(lib, op, rows, offsets, lanes)
