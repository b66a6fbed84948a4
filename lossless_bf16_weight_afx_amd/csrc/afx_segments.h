// afx_segments.h -- device pieces of the products that decode row segments of a
// coded matrix, several lanes a row, for the matrix cores
// (afx_gated_gemm.hip, afx_gemm_t.hip). Not installed.
//
// Loads are with kParts neighbouring lanes per row, so that a row's accesses
// fall into one cache line; decoding is with one row per lane. What the two
// orders hand over goes through LDS.
#pragma once

#include "afx_slab.h"

namespace afx {
namespace {

// Every lane gets the value of the first of its row's kParts (2 or 4) lanes.
template <int kParts>
__device__ inline uint64_t row_first(uint64_t v) {
    constexpr int kPick = kParts == 4 ? 0x00 : 0xA0;  // quad_perm 0,0,0,0 or 0,0,2,2
    const int lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)v, kPick, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(v >> 32), kPick, 0xF, 0xF, false);
    return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}

// A tile's place in its tensor: bases of its first element, so that a lane's
// own offsets stay 32-bit.
struct Tile {
    const uint64_t *base;   // chunk_base of the tile's first chunk
    const uint16_t *gap;    // gap of its first group
    const uint8_t *sm;      // its first sign/mantissa byte
    uint32_t in_chunk;      // its first element's place in that chunk
    uint32_t left;          // elements from its first to the tensor's end (at most 2^31)
};
__device__ inline Tile tile_at(const TensorDesc &T, uint64_t e0) {
    return Tile{T.chunk_base + (e0 >> 12), T.gap + (e0 >> 5), T.signmant + e0, (uint32_t)e0 & (kChunk - 1),
                (uint32_t)umin64(T.n - e0, 1u << 31)};
}

// A row's part of a slab: its elements [start, start + len), from the tile's
// first element.
struct Seg {
    uint32_t start, len;
};

// What the bit offsets of the lane's groups 2 c and 2 c + 1 of a segment and
// of its end are made of (afx_index.h), kept as loaded and added up only
// where used.
struct Bits {
    u32x4 base;        // u64 bit bases of the chunk that the segment starts in, and of the next
    uint32_t a, b, e;  // gaps of the lane's groups and of the group after the segment
    uint32_t next;     // SegRefs::next
};
__device__ inline Bits seg_bits(const Tile &t, const Seg &g, uint32_t c) {
    const SegRefs r = seg_refs(t.in_chunk, t.left, g.start, g.len, c);
    Bits b;
    __builtin_memcpy(&b.base, t.base + r.chunk, 16);  // (8-byte aligned; the entry after the last chunk's exists)
    b.a = t.gap[r.a];
    b.b = t.gap[r.b];
    b.e = t.gap[r.e];
    b.next = r.next;
    return b;
}

// A row segment's staged words [wa, wa + nw), and where the lane's groups
// start in them, in bits (16 each). Differences of positions are taken modulo
// 2^32: they are small, or, on a corrupt stream, clamped.
struct Words {
    uint64_t wa;
    uint32_t nw, starts;
};
template <int kParts, uint32_t kWords, uint32_t kMaxStart>
__device__ inline Words seg_words_of(const TensorDesc &T, const Bits &b) {
    const uint64_t b0 = ((uint64_t)b.base.y << 32) | b.base.x, bn = ((uint64_t)b.base.w << 32) | b.base.z;
    const uint64_t pa = (b.next & 1 ? bn : b0) + b.a;
    Words w;
    w.wa = seg_first_word(row_first<kParts>(pa));
    const uint32_t first = (uint32_t)w.wa << 5;
    w.nw = seg_staged(seg_end(b.next, b.base.x, b.base.z, b.e, T.reserved), w.wa, kWords);
    w.starts = min((uint32_t)pa - first, kMaxStart) |
               min((b.next & 2 ? b.base.z : b.base.x) + b.b - first, kMaxStart) << 16;
    static_assert(kMaxStart < 1u << 16, "a start fits 16 bits");
    return w;
}

// (`reserved`: the stream's length in bits, modulo 2^32)
inline TensorDesc tensor(const afx_info *info, const void *blob) {
    const uint8_t *b = static_cast<const uint8_t *>(blob);
    TensorDesc t{};
    t.code_len = b + info->off_code_len;
    t.chunk_base = reinterpret_cast<const uint64_t *>(b + info->off_chunk_base);
    t.gap = reinterpret_cast<const uint16_t *>(b + info->off_gap);
    t.signmant = b + info->off_signmant;
    t.exp = reinterpret_cast<const uint32_t *>(b + info->off_exp);
    t.n = info->n_elems;
    t.exp_words = info->exp_words;
    t.last_word4 = last_word4(info->exp_words);
    t.n_chunks = (uint32_t)info->n_chunks;
    t.reserved = (uint32_t)info->total_bits;
    return t;
}

}  // namespace
}  // namespace afx
