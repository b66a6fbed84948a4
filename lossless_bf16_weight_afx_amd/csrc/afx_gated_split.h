// afx_gated_split.h -- how the slabs of the gated block's matrices are cut into
// ranges, one per workgroup (afx_gated_gemm.hip). constexpr, no HIP: the same
// functions run in the kernels and in a host program that checks them.
//
// A wave takes 16 rows of a matrix. A tile is the rows of the `waves` waves of
// a workgroup; it has tile_slabs slabs of 256 columns, and slab s of all
// tiles' belongs to tile s / tile_slabs. Range w of R takes slabs [T w / R, T
// (w + 1) / R) of all T (rounded down), so that ranges differ by at most one
// slab.
#pragma once

#include <cstdint>

namespace afx {

constexpr uint32_t kGatedWaveRows = 16;
constexpr uint32_t kSlabCols = 256;  // columns restored per step

struct GatedSplit {
    uint32_t waves;      // that take rows, of a workgroup
    uint32_t tiles, tile_slabs, ranges;
    uint32_t most;       // most ranges that share a tile
    uint32_t row_tiles;  // 16-row tiles of a matrix
};

constexpr uint32_t range_begin(const GatedSplit &s, uint32_t w) {
    return (uint32_t)((uint64_t)s.tiles * s.tile_slabs * w / s.ranges);
}

// The range that slab i lies in: the largest w with T w / R < i + 1.
constexpr uint32_t range_of(const GatedSplit &s, uint32_t i) {
    const uint64_t total = (uint64_t)s.tiles * s.tile_slabs;
    return (uint32_t)((((uint64_t)i + 1) * s.ranges + total - 1) / total - 1);
}

// s's slabs in at most `resident` ranges, none empty.
constexpr GatedSplit with_ranges(GatedSplit s, uint32_t resident) {
    const uint64_t total = (uint64_t)s.tiles * s.tile_slabs;
    s.ranges = (uint32_t)(total < resident ? total : resident);
    // a tile's slabs reach over at most this many ranges of total / ranges or more
    const uint32_t least = (uint32_t)(total / s.ranges);
    s.most = (s.tile_slabs - 1) / least + 2;
    if (s.most > s.tile_slabs) s.most = s.tile_slabs;
    return s;
}

// Both for the tiles of one matrix. A small matrix is given to fewer
// waves of each workgroup, so that there are slabs for all workgroups. rows <
// 2^21 and cols < 2^22 keep the slab count below 2^32.
constexpr GatedSplit split_slabs(uint64_t rows, uint64_t cols, uint32_t resident, uint32_t waves) {
    GatedSplit s{};
    s.tile_slabs = (uint32_t)((cols + kSlabCols - 1) / kSlabCols);
    s.row_tiles = (uint32_t)((rows + kGatedWaveRows - 1) / kGatedWaveRows);
    for (s.waves = waves;; s.waves /= 2) {
        s.tiles = (s.row_tiles + s.waves - 1) / s.waves;
        if (s.waves == 1 || (uint64_t)s.tiles * s.tile_slabs >= resident) break;
    }
    return with_ranges(s, resident);
}

// Where the sums of one wave's rows from one range go: tile, the range's place
// in it, the wave.
constexpr uint64_t part_place(const GatedSplit &s, uint32_t tile, uint32_t place, uint32_t wave) {
    return ((uint64_t)tile * s.most + place) * s.waves + wave;
}
constexpr uint64_t part_places(const GatedSplit &s) { return (uint64_t)s.tiles * s.most * s.waves; }

}  // namespace afx
