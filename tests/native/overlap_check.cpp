// overlap_check.cpp -- on the CPU, the test of whether two strided buffers
// share a byte (afx_internal.h: rows_overlap), against sets of bytes: exact
// for buffers of one stride and for single rows, and never missing a shared
// byte for others. Built with AddressSanitizer and UndefinedBehaviorSanitizer
// by tests/test_overlap.py; prints "overlap ok" and exits 0, else exits 1.
#include <cstdint>
#include <cstdio>
#include <random>
#include <set>

#include "afx_internal.h"

using namespace afx;

namespace {

const char *const kBase = reinterpret_cast<const char *>(uintptr_t{1} << 20);  // never dereferenced

std::set<uint64_t> bytes(uint64_t at, const RowSpan &s) {
    std::set<uint64_t> b;
    for (uint64_t r = 0; r < s.rows; ++r)
        for (uint64_t c = 0; c < s.width; ++c) b.insert(at + r * s.stride + c);
    return b;
}

bool share(const std::set<uint64_t> &a, const std::set<uint64_t> &b) {
    for (uint64_t v : a)
        if (b.count(v)) return true;
    return false;
}

}  // namespace

int main() {
    std::mt19937_64 rng(9);
    int fail = 0, disjoint = 0, shared = 0, interleaved = 0;
    for (int i = 0; i < 200000; ++i) {
        const uint64_t stride = 1 + rng() % 24, other = rng() % 3 ? stride : 1 + rng() % 24;
        const uint64_t at_a = rng() % 60, at_b = rng() % 60;
        const RowSpan a{kBase + at_a, rng() % 5, 1 + rng() % stride, stride};
        const RowSpan b{kBase + at_b, rng() % 5, 1 + rng() % other, other};
        const auto sa = bytes(at_a, a), sb = bytes(at_b, b);
        const bool want = share(sa, sb), got = rows_overlap(a, b);
        const bool exact = stride == other || (a.rows <= 1 && b.rows <= 1);
        if (got != rows_overlap(b, a) || (exact ? got != want : want && !got)) {
            if (fail++ < 10)
                std::fprintf(stderr, "overlap: %llu rows of %llu, stride %llu, at %llu and %llu of %llu, %llu, at %llu: %d\n",
                             (unsigned long long)a.rows, (unsigned long long)a.width, (unsigned long long)a.stride,
                             (unsigned long long)at_a, (unsigned long long)b.rows, (unsigned long long)b.width,
                             (unsigned long long)b.stride, (unsigned long long)at_b, got);
        }
        ++(want ? shared : disjoint);
        interleaved += !got && !sa.empty() && !sb.empty() && *sa.begin() < *sb.rbegin() && *sb.begin() < *sa.rbegin();
    }
    const RowSpan none{nullptr, 4, 8, 8}, some{kBase, 4, 8, 8}, huge{kBase, 1u << 23, 1u << 22, 1u << 24};
    if (rows_overlap(none, some) || rows_overlap(some, none) || !rows_overlap(huge, some)) ++fail;
    if (fail || !shared || !disjoint || !interleaved) return 1;
    std::puts("overlap ok");
    return 0;
}
