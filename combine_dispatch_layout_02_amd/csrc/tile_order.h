// tile_order.h -- which tile a block of the gated product's tile kernel takes.
// Integer arithmetic only, for the host and the device.
#pragma once

#include <stdint.h>

namespace ep {

// Consecutive blocks go to the 8 XCDs in turn, and each XCD takes an eighth of
// the tiles, 8 row tiles by 4 columns together, which share their operands in
// its L2.  The row tiles are those that have rows, counted on the device: an
// eighth of all that the buffer could hold would leave most XCDs without work
// where the rows in use are a part of it (a slice of the experts, masked pairs,
// capacity to spare).  32 experts, K = 7168, 4096 weight rows, us, against that:
//   32768 rows 1896 (1932); the same as a slice of 262144 rows 2110 to 2170
//   (11100), the rest for the blocks past the tiles, which count them and end;
//   16384 rows in a buffer of 32768 1091 (1712), in one of their own 1074 (1072)
// Ragged segments gain too, as numbers without a tile spread unevenly: 5600 rows
// 441 (490).  Whole groups of 32 tiles to the XCDs in turn took 1911 for the
// first and 2137 for the second, but up to 30 % more where there are few groups.
struct TileOrder {
    int rows, cols;   // row tiles with rows, columns
    // The row tile and column of a block; false for blocks past the tiles.
    constexpr bool tile(uint32_t block, int *row, int *col) const {
        const uint32_t share = (uint32_t)((rows + 7) / 8) * cols, at = block / 8, per = 8 * cols;
        if (at >= share) return false;
        const uint32_t tile = block % 8 * share + at, in = tile % per, group = in / 32;
        const uint32_t left = cols - 4 * group, wide = left < 4 ? left : 4;
        *row = (int)(tile / per * 8 + (in - 32 * group) / wide);
        *col = (int)(4 * group + (in - 32 * group) % wide);
        return *row < rows;
    }
    // Blocks to launch for at most this many row tiles.
    static constexpr int64_t blocks(int most, int cols) { return (int64_t)((most + 7) / 8) * 8 * cols; }
};

}  // namespace ep
