"""The order in which the gated product's tiles go to the XCDs (CPU): every tile
once, an even share for each of the 8 XCDs however much larger the buffer and
the launch are than the tiles in use, and neighbours that share operands on one
XCD.  csrc/tile_order.h is compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_dispatch_layout_02_amd", "csrc")

SOURCE = """
#include "tile_order.h"
extern "C" int64_t blocks(int most, int cols) { return ep::TileOrder::blocks(most, cols); }
extern "C" void tiles(int rows, int cols, int64_t n, int32_t *row, int32_t *col) {
    const ep::TileOrder o{rows, cols};
    for (int64_t b = 0; b < n; ++b) {
        int r, c;
        const bool live = o.tile((uint32_t)b, &r, &c);
        row[b] = live ? r : -1;
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

    def tiles(rows, cols, most):
        """Row tile and column (-1: none) of every block of a launch for `most` row tiles, of which `rows` have rows."""
        n = c.blocks(most, cols)
        r, k = np.empty(n, np.int32), np.empty(n, np.int32)
        c.tiles(rows, cols, ctypes.c_int64(n), r.ctypes.data_as(ctypes.c_void_p), k.ctypes.data_as(ctypes.c_void_p))
        return r, k
    return tiles


@pytest.mark.parametrize("rows", [0, 1, 7, 8, 9, 64, 130, 281])
@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 7, 8, 9, 13, 16, 17, 56])
def test_every_tile_once(order, rows, cols):
    for most in (max(rows, 1), rows + 40, 8 * rows + 32):
        r, c = order(rows, cols, most)
        live = r >= 0
        assert ((c[live] >= 0) & (c[live] < cols) & (r[live] < rows)).all()
        at = r[live].astype(np.int64) * cols + c[live]
        assert at.size == rows * cols and np.unique(at).size == rows * cols


# row tiles in use, columns, row tiles of the launch: a whole buffer of 32 experts, one of 8 ranks' experts as a
# slice of 262144 rows, buffers that are half and a quarter full, small and odd ones
@pytest.mark.parametrize("rows,cols,most", [(272, 16, 288), (272, 16, 2080), (144, 16, 288), (72, 16, 288),
                                            (40, 16, 2080), (280, 8, 2080), (300, 3, 1100), (77, 5, 288), (9, 16, 64)])
def test_xcds_share_the_tiles(order, rows, cols, most):
    r, _ = order(rows, cols, most)
    live = np.flatnonzero(r >= 0)
    n = np.bincount(live % 8, minlength=8)
    assert n.sum() == rows * cols
    # the rows up to a whole number of 8 are in the last share
    assert n.max() == -(-rows // 8) * cols and n.max() - n.min() <= 7 * cols
    assert live.max() < 8 * n.max()                  # nothing is behind blocks without a tile


def test_neighbours_share_an_xcd(order):
    """8 row tiles by 4 columns follow each other on one XCD."""
    r, c = order(64, 16, 64)
    b = np.arange(r.size)
    for row in range(0, 64, 8):
        for col in range(0, 16, 4):
            mine = b[(r // 8 == row // 8) & (c // 4 == col // 4)]
            assert np.unique(mine % 8).size == 1 and mine.max() - mine.min() == 8 * 31
