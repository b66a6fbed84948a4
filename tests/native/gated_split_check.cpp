// gated_split_check.cpp -- on the CPU, the gated block's division of its
// slabs into ranges (afx_gated_split.h): the ranges take every slab once, in
// order, none is empty, they differ by at most one slab, range_of finds the
// range of every slab, and no tile is shared by more ranges than `most`, the
// number of places it has in the workspace. Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_gated_split.py; prints "gated
// split ok" and exits 0, else exits 1.
#include <cstdint>
#include <cstdio>
#include <random>

#include "afx_gated_split.h"

using namespace afx;

namespace {

int g_fail = 0;
#define CHECK(cond, ...)                                         \
    do {                                                         \
        if (!(cond)) {                                           \
            if (g_fail++ < 20) {                                 \
                std::fprintf(stderr, "gated split: " __VA_ARGS__); \
                std::fputc('\n', stderr);                        \
            }                                                    \
        }                                                        \
    } while (0)

void check(uint64_t rows, uint64_t cols, uint32_t resident, uint32_t waves) {
    const GatedSplit s = split_slabs(rows, cols, resident, waves);
    const uint64_t total = (uint64_t)s.tiles * s.tile_slabs;
    CHECK((uint64_t)s.tiles * s.waves * kGatedWaveRows >= rows && (uint64_t)s.tile_slabs * kSlabCols >= cols &&
              (uint64_t)s.row_tiles * kGatedWaveRows >= rows && (s.row_tiles - 1) * (uint64_t)kGatedWaveRows < rows,
          "%llu x %llu not covered", (unsigned long long)rows, (unsigned long long)cols);
    CHECK(s.waves >= 1 && s.waves <= waves && (s.waves == waves || total < 2ull * resident + s.tile_slabs),
          "%u waves for %llu slabs", s.waves, (unsigned long long)total);
    CHECK(s.ranges >= 1 && s.ranges <= resident, "%u ranges", s.ranges);
    CHECK(range_begin(s, 0) == 0 && range_begin(s, s.ranges) == total, "ends");
    const uint32_t least = (uint32_t)(total / s.ranges);
    for (uint32_t w = 0; w < s.ranges; ++w) {
        const uint32_t b = range_begin(s, w), e = range_begin(s, w + 1);
        CHECK(e > b && e - b >= least && e - b <= least + 1, "range %u of %llu x %llu: %u slabs", w,
              (unsigned long long)rows, (unsigned long long)cols, e - b);
        for (uint32_t i = b; i < e; i += (e - b > 64 ? 7 : 1)) {
            CHECK(range_of(s, i) == w, "slab %u is in range %u, not %u", i, w, range_of(s, i));
            const uint32_t tile = i / s.tile_slabs, place = w - range_of(s, tile * s.tile_slabs);
            CHECK(place < s.most, "tile %u: place %u of %u", tile, place, s.most);
            CHECK(part_place(s, tile, place, s.waves - 1) < part_places(s), "place past the workspace");
        }
    }
}

}  // namespace

int main() {
    for (uint64_t rows : {1, 5, 16, 17, 31, 33, 64, 100, 1024, 5461, 17408})
        for (uint64_t cols : {32, 224, 256, 288, 512, 2048, 5120, 17408})
            for (uint32_t resident : {1, 2, 7, 128, 384})
                for (uint32_t waves : {1, 4, 16}) check(rows, cols, resident, waves);
    check((1u << 21) - 1, 256, 128, 16);
    check(1024, (1u << 22) - 32, 384, 4);
    std::mt19937_64 rng(3);
    for (int i = 0; i < 400; ++i) check(1 + rng() % 40000, 32 * (1 + rng() % 300), 1 + rng() % 500, 1u << rng() % 5);
    if (g_fail) return 1;
    std::puts("gated split ok");
    return 0;
}
