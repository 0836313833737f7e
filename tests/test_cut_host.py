"""The cut of the experts' rows into tiles, replayed on the host from the
kernels' own header (compiled here with the host compiler): a stage of the
ring holds the columns of the widest tile, so no tile may be wider, whatever
the capacity takes from which expert."""
import ctypes as C
import os
import random
import subprocess

import numpy as np
import pytest

from combine_ep_get_layout_gb300 import build

SHIM = """
#include "ep_cut.h"
extern "C" int widest(int cap, int most_rows, int max_cols, const int32_t *offset, const int32_t *count, int experts,
                      int lanes) {
  const ep::RowLimits l{cap, most_rows, max_cols};
  int most = 0;
  for (int i = 0; i < lanes; ++i) {
    const int n = ep::widest_tile(l, offset, count, experts, i, lanes);
    most = n > most ? n : most;
  }
  return most;
}
extern "C" int any_call(int cap, int most_rows, int max_cols) {
  return ep::most_cols_of(ep::RowLimits{cap, most_rows, max_cols});
}
// The tiles of one expert: (first row, rows, columns) each; their number.
extern "C" int tiles(int cap, int most_rows, int max_cols, int first, int count, int32_t *out) {
  const ep::RowLimits l{cap, most_rows, max_cols};
  const int rows = ep::rows_within(l, first, count), n = ep::tiles_of(l, rows);
  for (int i = 0; i < n; ++i) {
    int from;
    const int here = ep::tile_rows(l, rows, i, &from);
    out[3 * i] = first + from;
    out[3 * i + 1] = here;
    out[3 * i + 2] = ep::ceil_over(here, ep::kColumnStep) * ep::kColumnStep;
  }
  return n;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    folder = tmp_path_factory.mktemp("cut")
    src, lib = os.path.join(folder, "cut.cpp"), os.path.join(folder, "cut.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    return C.CDLL(lib)


def ints(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(C.c_void_p)


def check(cut, counts, offset, cap, most_rows, max_cols):
    """Every tile fits a stage; the tiles are the rows below the capacity, each once."""
    counts, pc = ints(counts)
    offset, po = ints(offset)
    # a call of so few rows does not look at its counts (Walker::most_cols)
    wide = cut.widest(cap, most_rows, max_cols, po, pc, len(counts), 32)
    assert wide <= cut.any_call(cap, most_rows, max_cols)
    out = np.zeros(3 * 4096, np.int32)
    for e in range(len(counts)):
        n = cut.tiles(cap, most_rows, max_cols, int(offset[e]), int(counts[e]), out.ctypes.data_as(C.c_void_p))
        at = int(offset[e])
        for first, rows, cols in out[:3 * n].reshape(n, 3).tolist():
            assert first == at and rows > 0 and rows <= cols <= max_cols and cols % 32 == 0
            assert cols <= wide, (counts.tolist(), cap, e, cols, wide)
            at += rows
        want = max(0, min(int(counts[e]), most_rows, cap - int(offset[e]))) if 0 <= offset[e] < cap else 0
        assert at - int(offset[e]) == want


def test_a_cut_expert_may_have_wider_tiles(cut):
    """Four experts of 300 rows: two tiles of 160 each; the last one cut to
    180 is a single tile of 192.  260 rows cut to 256: 160 and 256."""
    check(cut, [300] * 4, [0, 300, 600, 900], 1080, 1200, 256)
    check(cut, [260, 260], [0, 260], 516, 520, 256)
    check(cut, [384] * 64, [384 * e for e in range(64)], 384 * 63 + 240, 4096, 256)


@pytest.mark.parametrize("seed", range(8))
def test_no_tile_is_wider_than_a_stage(cut, seed):
    r = random.Random(seed)
    for _ in range(400):
        experts = r.choice([1, 2, 3, 8, 33, 64])
        mean = r.choice([1, 20, 65, 130, 200, 300, 390, 700])
        counts = [max(0, int(r.gauss(mean, r.choice([0, mean ** 0.5, mean])))) for _ in range(experts)]
        align = r.choice([1, 1, 8, 128])
        offset, at = [], 0
        for n in counts:
            offset.append(at)
            at += (n + align - 1) // align * align
        cap = r.choice([at, max(1, at - r.randint(0, 2 * mean)), r.randint(1, max(1, at)), at + 5])
        most_rows = min(cap, r.choice([max(counts + [1]), sum(counts) + 1, max(1, mean)]))
        check(cut, counts, offset, cap, most_rows, r.choice(range(32, 257, 32)))


def test_offsets_that_are_none(cut):
    """Offsets and counts that no layout has reach no row outside the capacity."""
    check(cut, [10, 2 ** 31 - 1, 70, -5, 8], [-3, 5, 2 ** 31 - 1, 4, 90], 90, 90, 64)
