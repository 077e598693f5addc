// tile_order.h -- which tile a block of the gated product's tile kernel takes.
// Integer arithmetic only, for the host and the device.
#pragma once

#include <stdint.h>

namespace ep {

// Consecutive blocks go to the 8 XCDs in turn.  A group of 8 row tiles by up to
// 4 columns is taken whole by one XCD, so that its tiles share their operands in
// the XCD's L2; the groups go to the XCDs in turn, so that wherever the rows in
// use lie in the buffer (a slice of the experts, a part-filled block) every XCD
// has its share of them.  32768 rows, 32 experts, K = 7168, 4096 weight rows: 1911
// us (all columns of 2 row tiles together, measured on another form, 6 % more;
// an eighth of the tile numbers to each XCD 1945).  The same rows as a slice of a
// buffer of 262144: 2137 us, most of the difference for blocks without a tile
// (an eighth to each XCD: 10940, as nine tenths of the rows were on one XCD).
struct TileOrder {
    int slots, cols;   // row tiles, columns
    int bands, wide;   // groups side by side over the columns, columns of one (the last may have fewer)
    constexpr TileOrder(int slots_, int cols_)
        : slots(slots_), cols(cols_), bands((cols_ + 3) / 4), wide((cols_ + bands - 1) / bands) {}
    // blocks to launch: whole groups, the same number for every XCD
    constexpr int64_t blocks() const { return ((int64_t)((slots + 7) / 8) * bands + 7) / 8 * 8 * (8 * wide); }
    // The row tile and column of a block; false for those that fill up a group or a turn.
    constexpr bool tile(uint32_t block, int *slot, int *col) const {
        const uint32_t size = 8 * wide, turn = block / 8, in = turn % size;
        const uint32_t group = turn / size * 8 + block % 8;
        *slot = (int)(group / bands * 8 + in / wide);
        *col = (int)(group % bands * wide + in % wide);
        return *slot < slots && *col < cols;
    }
};

}  // namespace ep
