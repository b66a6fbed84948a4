// segment_check.cpp -- on the CPU, the row segments that the gated block's and
// the transposed product's kernels decode (afx_index.h: seg_refs, seg_end,
// seg_staged): on streams of random code lengths, for every segment of small
// and odd matrices, the lanes' groups start where the stream has them, and the
// words staged reach to the segment's end, also where it is the tensor's last
// one and crosses into the last chunk; and on corrupt streams their count stays
// within the slice. The tiles, segments and clamps are
// composed here as the kernels compose them. Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_segments.py; prints "segments ok"
// and exits 0, else exits 1.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "afx_index.h"

using namespace afx;

namespace {

int g_fail = 0;
#define CHECK(cond, ...)                                      \
    do {                                                      \
        if (!(cond)) {                                        \
            if (g_fail++ < 20) {                              \
                std::fprintf(stderr, "segments: " __VA_ARGS__); \
                std::fputc('\n', stderr);                     \
            }                                                 \
        }                                                     \
    } while (0)

// Where every element's code starts, and the sections a blob records of it.
struct Stream {
    std::vector<uint64_t> at, chunk_base;
    std::vector<uint16_t> gap;
    uint64_t bits() const { return at.back(); }
};
Stream stream(uint64_t n, uint32_t kind, std::mt19937_64 &rng) {
    Stream s;
    s.at.resize(n + 1);
    uint64_t p = 0;
    for (uint64_t i = 0; i < n; ++i) {
        s.at[i] = p;
        if (i % kChunk == 0) s.chunk_base.push_back(p);
        if (i % kGroup == 0) s.gap.push_back((uint16_t)(p - s.chunk_base.back()));
        const bool tail = i + 300 >= n;
        p += kind == 0 ? 1 + rng() % kMaxLen : kind == 1 ? (tail ? kMaxLen : 1) : kMaxLen;
    }
    s.at[n] = p;
    s.chunk_base.push_back(p);
    return s;
}

// kCols columns of kRows rows a slab; whole: rows are whole groups.
struct Slabs {
    uint32_t rows, cols, parts, words, max_start;
    bool whole;
};

void check(const Slabs &k, uint64_t rows, uint64_t cols, const Stream &s) {
    const uint64_t n = rows * cols;
    const uint32_t step = k.whole ? k.cols : k.cols - kGroup;
    for (uint64_t r0 = 0; r0 < rows; r0 += k.rows)
        for (uint64_t c0 = 0; c0 < cols; c0 += step)
            for (uint32_t r = 0; r < k.rows; ++r) {
                // the tile starts at the group that its first value lies in
                const uint64_t e0 = r0 * cols + c0, t0 = e0 & ~(uint64_t)(kGroup - 1);
                const uint32_t row = (uint32_t)(umin64(r, rows - 1 - r0) * cols);
                const uint32_t left = (uint32_t)(n - t0), in_chunk = (uint32_t)t0 & (kChunk - 1);
                const uint32_t start = ((uint32_t)(e0 - t0) + row) & ~(kGroup - 1);
                const uint32_t to_end = ((left + kGroup - 1) & ~(kGroup - 1)) - start;
                const uint32_t len = k.whole ? umin32(k.cols, (uint32_t)(cols - c0)) : umin32(k.cols, to_end);
                const uint64_t first = t0 + start, end = umin64(first + len, n);
                const uint64_t ch0 = t0 / kChunk, g0 = t0 / kGroup;
                uint64_t wa = 0;
                for (uint32_t c = 0; c < k.parts; ++c) {
                    const SegRefs f = seg_refs(in_chunk, left, start, len, c);
                    CHECK(ch0 + f.chunk + 1 < s.chunk_base.size(), "base %u", f.chunk);
                    CHECK(g0 + f.a < s.gap.size() && g0 + f.b < s.gap.size() && g0 + f.e < s.gap.size(), "gap");
                    if (g_fail) return;
                    const uint64_t b0 = s.chunk_base[ch0 + f.chunk], b1 = s.chunk_base[ch0 + f.chunk + 1];
                    const uint64_t pa = (f.next & 1 ? b1 : b0) + s.gap[g0 + f.a];
                    const uint64_t pb = (f.next & 2 ? b1 : b0) + s.gap[g0 + f.b];
                    for (uint32_t h = 0; h < 2; ++h) {
                        const uint64_t e = first + kGroup * (2 * c + h);
                        CHECK(e >= first + len || (h ? pb : pa) == s.at[e], "%llu x %llu: group at %llu",
                              (unsigned long long)rows, (unsigned long long)cols, (unsigned long long)e);
                    }
                    if (c == 0) wa = seg_first_word(pa);
                    CHECK(pa - 32 * wa <= k.max_start && pb - 32 * wa <= k.max_start, "start clamped");
                    const uint32_t nw =
                        seg_staged(seg_end(f.next, (uint32_t)b0, (uint32_t)b1, s.gap[g0 + f.e], (uint32_t)s.bits()), wa,
                                   k.words);
                    const uint64_t want = ((s.at[end] + 31) >> 5) + 1 - wa;
                    CHECK(nw == want && want <= k.words, "%llu x %llu, elements %llu to %llu: %u words of %llu",
                          (unsigned long long)rows, (unsigned long long)cols, (unsigned long long)first,
                          (unsigned long long)end, nw, (unsigned long long)want);
                }
            }
}

}  // namespace

int main() {
    std::mt19937_64 rng(5);
    // words and clamps of the kernels' slices (afx_gated_gemm.hip; afx_gemm_t.hip: 56 words, 13 below the top kept)
    const Slabs gated{16, 256, 4, kSegWords, kSegMaxStart, true};
    const Slabs turned{32, 128, 2, 56, 32 * (55 - 13), true}, split{32, 128, 2, 56, 32 * (55 - 13), false};
    auto all = [&](uint64_t rows, uint64_t cols) {
        for (uint32_t kind = 0; kind < 3; ++kind) {
            const Stream s = stream(rows * cols, kind, rng);
            if (cols % kGroup == 0) {
                check(gated, rows, cols, s);
                check(turned, rows, cols, s);
            } else {
                check(split, rows, cols, s);
            }
        }
    };
    for (uint64_t rows = 1; rows <= 48; ++rows)
        for (uint64_t cols = 8; cols <= 360; cols += 8) all(rows, cols);
    for (int i = 0; i < 60; ++i) all(1 + rng() % 100, 8 * (1 + rng() % 700));
    // whatever bases and gaps a corrupt stream holds, no more words than the slice has
    for (int i = 0; i < 100000; ++i) {
        const uint32_t end = seg_end((uint32_t)rng(), (uint32_t)rng(), (uint32_t)rng(), (uint32_t)rng() & 0xFFFF, (uint32_t)rng());
        const uint64_t wa = seg_first_word(rng() >> rng() % 64);
        CHECK(seg_staged(end, wa, kSegWords) <= kSegWords, "%u words staged", seg_staged(end, wa, kSegWords));
    }
    if (g_fail) return 1;
    std::puts("segments ok");
    return 0;
}
