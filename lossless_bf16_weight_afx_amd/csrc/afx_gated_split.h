// afx_gated_split.h -- how the slabs of the gated block's tiles are cut into
// ranges (afx_gated_gemm.hip). constexpr, no HIP: the same functions run in
// the kernels and in a host program that checks them.
//
// Tiles of kGatedTileRows weight rows (of both matrices) have tile_slabs
// slabs of 256 columns each; slab s belongs to tile s / tile_slabs. Range w
// of R takes slabs [T w / R, T (w + 1) / R) of all T (rounded down), so that
// ranges differ by at most one slab.
#pragma once

#include <cstdint>

namespace afx {

constexpr uint32_t kGatedTileRows = 32;
constexpr uint32_t kSlabCols = 256;  // columns restored per step

struct GatedSplit {
    uint32_t tiles, tile_slabs, ranges;
    uint32_t most;  // most ranges that share a tile
};

constexpr uint32_t range_begin(const GatedSplit &s, uint32_t w) {
    return (uint32_t)((uint64_t)s.tiles * s.tile_slabs * w / s.ranges);
}

// The range that slab i lies in: the largest w with T w / R < i + 1.
constexpr uint32_t range_of(const GatedSplit &s, uint32_t i) {
    const uint64_t total = (uint64_t)s.tiles * s.tile_slabs;
    return (uint32_t)((((uint64_t)i + 1) * s.ranges + total - 1) / total - 1);
}

// At most `resident` ranges, none empty. rows < 2^21 and cols < 2^22 keep the
// slab count below 2^30.
constexpr GatedSplit split_slabs(uint64_t rows, uint64_t cols, uint32_t resident) {
    GatedSplit s{};
    s.tiles = (uint32_t)((rows + kGatedTileRows - 1) / kGatedTileRows);
    s.tile_slabs = (uint32_t)((cols + kSlabCols - 1) / kSlabCols);
    const uint64_t total = (uint64_t)s.tiles * s.tile_slabs;
    s.ranges = (uint32_t)(total < resident ? total : resident);
    // a tile's slabs reach over at most this many ranges of total / ranges or more
    const uint32_t least = (uint32_t)(total / s.ranges);
    s.most = (s.tile_slabs - 1) / least + 2;
    if (s.most > s.tile_slabs) s.most = s.tile_slabs;
    return s;
}

}  // namespace afx
