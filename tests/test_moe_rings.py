"""The rings of the persistent products on the host: csrc/ring.h (what the rings
hold and the order of a widening warp's waits) against a model of one CTA in
which loads land in any order, walked through exhaustively.

The model knows of a barrier what hardware tells a parity wait: whether the
number of completed phases is even or odd.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include "ring.h"
extern "C" {
// which wait comes first, 0 the place, 1 the stage; -1 if one is left out
int first_wait() {
    int n = 0, at[2] = {-1, -1};
    const bool ok = moe::ring::widen_ready([&] { at[0] = n++; return true; },
                                           [&] { at[1] = n++; return true; });
    return ok && at[0] >= 0 && at[1] >= 0 ? (at[0] < at[1] ? 0 : 1) : -1;
}
// whether a wait that ran out of time is taken for success
int ready_despite(int place, int stage) {
    return moe::ring::widen_ready([&] { return place != 0; }, [&] { return stage != 0; });
}
int turns() { return moe::ring::kTurns; }
int order_holds(int s, int u) { return moe::ring::order_holds(s, u); }
void gemm_ring(int nmax, int *out) {
    const auto r = moe::ring::gemm(nmax);
    out[0] = r.nmax, out[1] = r.box, out[2] = r.stages, out[3] = r.units;
    out[4] = moe::ring::gemm_bytes(r);
}
int layer_stages(int E, int P, int value_bytes, int rows) {
    return moe::ring::layer_stages(moe::ring::layer_ring_bytes(E, P), value_bytes, rows);
}
int layer_bytes(int E, int P, int value_bytes, int rows) {
    return moe::ring::layer_front_bytes(E, P) +
           layer_stages(E, P, value_bytes, rows) * moe::ring::layer_stage_bytes(value_bytes, rows);
}
int layer_holds(int value_bytes, int stages) {
    return moe::ring::layer_holds(value_bytes, stages);
}
int layer_slots() { return moe::ring::kLayerSlots; }
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("ring")
    src, lib = str(d / "ring.cpp"), str(d / "ring.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "combine_topk_ids_rank_gb300", "csrc"), src,
                    "-o", lib], check=True)
    return ctypes.CDLL(lib)


def reads_unlanded_unit(S, U, place_first, freed_by_products=False, turns=2):
    """Whether some order of events lets a widening group of unit n pass both of its
    waits before unit n has landed.  `turns` groups take the units in turn; products
    run in unit order; a stage is free again once its unit was widened (or, with
    freed_by_products, multiplied)."""
    N = 2 * S + 2 * U + 2
    # (units issued, landed set, waits each group has passed for its unit, each group's
    #  unit, widened set, units multiplied)
    start = (0, frozenset(), (0,) * turns, tuple(range(turns)), frozenset(), 0)
    seen, todo = {start}, [start]

    def phase_over(completed, j):       # what a parity wait for phase j sees
        return (completed ^ j) & 1 == 1

    while todo:
        issued, landed, passed, unit, wide, mul = todo.pop()
        nxt = []
        freed = mul if freed_by_products else None
        if issued < N and (issued < S or (issued - S < freed if freed_by_products
                                          else issued - S in wide)):
            nxt.append((issued + 1, landed, passed, unit, wide, mul))
        for n in range(issued):
            if n not in landed:
                nxt.append((issued, landed | {n}, passed, unit, wide, mul))
        if mul in wide:
            nxt.append((issued, landed, passed, unit, wide, mul + 1))
        for g in range(turns):
            n = unit[g]
            if n >= N:
                continue
            if passed[g] == 2:          # reads the stage now
                if n not in landed:
                    return True
                p, u = list(passed), list(unit)
                p[g], u[g] = 0, n + turns
                nxt.append((issued, landed, tuple(p), tuple(u), wide | {n}, mul))
                continue
            if (passed[g] == 0) == place_first:
                done = len([i for i in range(n % U, mul, U)])
                ok = phase_over(done, n // U - 1)
            else:
                done = len([i for i in landed if i % S == n % S])
                ok = phase_over(done, n // S)
            if ok:
                p = list(passed)
                p[g] += 1
                nxt.append((issued, landed, tuple(p), unit, wide, mul))
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


def test_the_model_finds_the_stage_that_was_waited_for_too_early():
    # two groups, an odd ring: the stage's last unit is the other group's
    assert reads_unlanded_unit(3, 3, place_first=False)
    assert not reads_unlanded_unit(3, 3, place_first=True)
    # and an even one, where it is the group's own
    assert not reads_unlanded_unit(4, 4, place_first=False)


def test_fewer_stages_than_places_are_refused(ring):
    assert reads_unlanded_unit(3, 4, place_first=True)
    assert not ring.order_holds(3, 4) and not ring.order_holds(2, 1)
    assert ring.order_holds(3, 3) and ring.order_holds(6, 4)


def test_a_wait_that_runs_out_is_no_success(ring):
    assert ring.ready_despite(1, 1)
    for place, stage in ((0, 0), (0, 1), (1, 0)):
        assert not ring.ready_despite(place, stage)


@pytest.mark.parametrize("nmax", [16, 32, 64, 128, 256])
def test_product_rings(ring, nmax):
    out = (ctypes.c_int * 5)()
    ring.gemm_ring(nmax, out)
    n, box, stages, units, nbytes = out
    assert n == nmax and (nmax // 2) % box == 0 and box <= 32
    assert ring.order_holds(stages, units)
    # shared memory of a CTA: 227 KB, 15 of them for the static tables
    assert nbytes <= (227 - 15) * 1024
    raw = (128 + nmax // 2) * 128
    assert stages == 12 or nbytes + raw > (227 - 15) * 1024
    # tensor memory: 256 columns of sums beside 64 a widened weight tile
    assert 256 + 64 * units <= 512


def test_product_waits(ring):
    out = (ctypes.c_int * 5)()
    shapes = set()
    for nmax in (16, 32, 64, 128, 256):
        ring.gemm_ring(nmax, out)
        shapes.add((min(out[2], 7), out[3]))            # (longer rings only have more slack)
    assert (3, 3) in shapes
    first = ring.first_wait()
    assert first in (0, 1)
    for S, U in sorted(shapes):
        assert not reads_unlanded_unit(S, U, place_first=first == 0, turns=ring.turns()), (S, U)


def layer_sizes():
    """Experts, top-k and tokens up to their limits; the fullest expert takes 1 .. all tokens."""
    for E in (1, 2, 31, 64, 300, 1024):
        for K in (1, 2, 8, 32):
            for T in (1, 7, 8, 33, 41, 48, 56, 64):
                for rows in range(1, T + 1):
                    yield E, K, T, rows


def test_layer_rings(ring):
    stages = set()
    for E, K, T, rows in layer_sizes():
        for size in (1, 2):
            n = ring.layer_stages(E, T * K, size, rows)
            assert ring.layer_holds(size, n), (E, K, T, rows, size)
            assert ring.layer_bytes(E, T * K, size, rows) <= (227 - 2) * 1024
            if size == 1:
                stages.add(n)
    assert {4, 5, 7} <= stages                          # odd rings are met
    assert not ring.layer_holds(1, 3) and ring.layer_holds(2, 3)
    assert not ring.layer_holds(2, 1)


def test_layer_waits(ring):
    U = ring.layer_slots()
    assert reads_unlanded_unit(5, U, place_first=False, freed_by_products=True)
    first = ring.first_wait()
    for S in {min(ring.layer_stages(E, T * K, 1, rows), 7) for E, K, T, rows in layer_sizes()}:
        assert not reads_unlanded_unit(S, U, place_first=first == 0, freed_by_products=True,
                                       turns=ring.turns()), S
