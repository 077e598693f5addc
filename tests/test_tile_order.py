"""The order in which the gated product's tiles go to the XCDs (CPU): every tile
once, groups whole on one XCD, and an even share for each of the 8 XCDs wherever
the rows in use lie in the buffer.  csrc/tile_order.h is compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_dispatch_layout_02_amd", "csrc")

SOURCE = """
#include "tile_order.h"
extern "C" int64_t blocks(int slots, int cols) { return ep::TileOrder(slots, cols).blocks(); }
extern "C" void tiles(int slots, int cols, int32_t *slot, int32_t *col) {
    const ep::TileOrder o(slots, cols);
    for (int64_t b = 0; b < o.blocks(); ++b) {
        int s, c;
        const bool live = o.tile((uint32_t)b, &s, &c);
        slot[b] = live ? s : -1;
        col[b] = live ? c : -1;
    }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    out = tmp_path_factory.mktemp("order")
    src, lib = str(out / "order.cpp"), str(out / "order.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib],
                   check=True, env={k: v for k, v in os.environ.items() if k != "LD_PRELOAD"})
    c = ctypes.CDLL(lib)
    c.blocks.restype = ctypes.c_int64

    def tiles(slots, cols):
        n = c.blocks(slots, cols)
        s, k = np.empty(n, np.int32), np.empty(n, np.int32)
        c.tiles(slots, cols, s.ctypes.data_as(ctypes.c_void_p), k.ctypes.data_as(ctypes.c_void_p))
        return s, k
    return tiles


@pytest.mark.parametrize("slots", [1, 7, 8, 9, 64, 130, 288, 2080])
@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 16, 17, 56])
def test_every_tile_once(order, slots, cols):
    s, c = order(slots, cols)
    live = s >= 0
    assert (s[live].astype(np.int64) * cols + c[live]).size == slots * cols
    assert np.unique(s[live].astype(np.int64) * cols + c[live]).size == slots * cols
    # blocks without a tile: less than a quarter more columns, and what fills up the last turn
    assert s.size <= (slots + 7) // 8 * 8 * cols * 5 // 4 + 8 * 32 and s.size % 8 == 0


def _per_xcd(s, lo, hi):
    """Tiles of the row tiles [lo, hi) on each XCD."""
    at = np.flatnonzero((s >= lo) & (s < hi))
    return np.bincount(at % 8, minlength=8)


# (row tiles of the buffer, columns, row tiles in use): a whole buffer, one of 8 ranks' experts as a slice of a
# dispatch of 262144 rows, a buffer half filled, a quarter, some rows in the middle
@pytest.mark.parametrize("slots,cols,lo,hi", [(288, 16, 0, 288), (2080, 16, 512, 800), (2080, 16, 0, 288),
                                              (288, 16, 0, 144), (288, 16, 0, 72), (288, 16, 100, 140),
                                              (2080, 8, 1000, 1280), (1100, 3, 300, 600), (288, 5, 64, 192)])
def test_xcds_share_the_rows_in_use(order, slots, cols, lo, hi):
    s, _ = order(slots, cols)
    n = _per_xcd(s, lo, hi)
    assert n.sum() == (hi - lo) * cols
    assert n.max() - n.min() <= 2 * 8 * 4, n     # a group at either end
    # and at any time: no XCD is further ahead in launch order than a turn of groups
    at = np.flatnonzero((s >= lo) & (s < hi)) // 8
    assert at.max() - at.min() + 1 <= n.max() + 2 * 8 * 4


def test_a_group_stays_on_one_xcd(order):
    s, c = order(288, 16)
    b = np.arange(s.size)
    for row in range(0, 288, 8):
        for col in range(0, 16, 4):
            mine = b[(s // 8 == row // 8) & (c // 4 == col // 4)]
            assert np.unique(mine % 8).size == 1 and mine.max() - mine.min() == 8 * 31
