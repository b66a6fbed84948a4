// afx_gemm_t.hip -- y = d W for few tokens (gfx950), W restored and
// multiplied on the matrix cores without reaching memory: the transposed
// product, whose reduction runs along W's rows, one below the other.
//
// A wave's slab is 32 rows by 128 columns: 128 groups of 32 values, which
// decode on their own, two per lane (rows l mod 16 and 16 + l mod 16, columns
// from 32 (l / 16)). A lane then holds 32 columns of a row, while the matrix
// instruction wants 8 rows of a column: the restored slab goes through the
// wave's 8 KB of LDS and is read back transposed (ds_read_b64_tr_b16). The
// slab's tokens' operand is 32 rows wide whatever the columns, so it is one
// load per 16 tokens; the sums of 128 columns stay in registers (32 per 16
// tokens).
//
// The decode bounds this: of the 56 us that 16 tokens and a 5120 x 17408 matrix
// take (its coded bytes alone 20) vector instructions are issued for 28 (780 a
// slab), LDS is busy for 24, half of it in bank conflicts of the table's reads,
// and a wave waits for one of them, or for memory, in half of its time. 1.5
// times the coded bytes are read (a slab needs only a part of the lines that
// hold a row's gaps and code words; its neighbours come to them at other times).
//
// The slabs of a column tile, then of the next, are cut into one contiguous
// range per workgroup, whose waves take them in turn; the waves' sums are
// added through LDS, a tile's ranges by a last launch, in order: the same bits
// on every run.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "afx_gated_split.h"
#include "afx_gemm_t.h"
#include "afx_segments.h"

namespace afx {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kTRows = 32, kTCols = 128;  // a slab as it is decoded
constexpr uint32_t kTok = 16;                  // tokens of an operand
// Columns of a slab that are multiplied: all, or, where rows are not whole
// groups and so start up to 24 values into one, 96, which 4 groups cover
// wherever the row starts.
constexpr uint32_t slab_cols(bool whole) { return whole ? kTCols : kTCols - kGroup; }
constexpr uint32_t slab_units(bool whole) { return slab_cols(whole) / 16; }  // 16: columns of a matrix instruction
// Column slabs that a workgroup's waves take side by side. The lines that
// hold a row's code words and gaps are then read by waves of one CU at about
// the same time; more of them leave fewer waves to add their sums in LDS,
// and more sums for the join. 5120 x 17408, 16 tokens, with join: 1 68 us, 2
// 60, 4 61; both 17408 x 5120 matrices, 64 tokens: 140, 133, 141.
constexpr uint32_t kColWaves = 2;

// A row segment's code words in LDS, as afx_index.h stages those of 256
// columns: 128 codes of at most 12 bits, the first word's alignment and
// offset, a word of look-ahead.
constexpr uint32_t kRowWords = 56, kRowRev = kRowWords - 1, kRowSlice = kRowWords + 4;
constexpr uint32_t kRowMaxStart = 32 * (kRowRev - 13);
static_assert(kRowWords * 32 >= kTCols * kMaxLen + 5 * 32 && kRowRev % 4 == 3, "a segment's words fit its slice");
static_assert(chain_word(32 * kRowRev + kLead) + 1 < kRowSlice, "a chain's first words are in the slice");
static_assert(chain_word(32 * kRowRev + kLead - kRowMaxStart - 32 * kMaxLen) >= 1, "and its last, read ahead");

constexpr uint32_t kSmRow = kTCols + 16;       // a row's sign/mantissa bytes in LDS
constexpr uint32_t kStage = kTRows * (kSmRow + kTCols);  // bytes of LDS of a wave: the sign/mantissa bytes and half
                                                         // the restored slab
static_assert(kTRows * kRowSlice * 4 <= kStage && slab_units(true) * 64 * 16 <= kStage && kTRows * kSmRow % 256 == 0 &&
              kSmRow >= kTCols, "so do the words, or 16 tokens' sums; rows stay aligned to the banks");

struct TArgs {
    TensorDesc w[2];
    const uint16_t *d[2];
    uint64_t lda;
    float *part;  // [matrix][places][token blocks][column waves][unit][lane][4]
    uint64_t part_mat;  // floats from matrix to matrix
    uint32_t n_mats, m, rows, cols, ak, col_slabs;
    GatedSplit split;  // tiles of kColWaves column slabs; their slabs follow the rows
    float *y32;
    uint16_t *y16;
    uint64_t ldy;
    uint32_t add;
};

// Where 16 bytes (8 columns) of the restored slab lie in LDS: row r is 256
// bytes, its 32-byte unit u at u ^ (r & 3 | r >> 1 & 4), so that the rows
// which one transposing read takes are spread over all banks, and the halves
// of a unit swapped every other 4 rows, so that the writes are.
__device__ inline uint32_t row_swizzle(uint32_t r) { return (r & 3) | ((r >> 1) & 4); }
__device__ inline uint32_t piece_at(uint32_t r, uint32_t piece) {
    return r * (kTCols * 2) + 32 * ((piece >> 1) ^ row_swizzle(r)) + 16 * ((piece & 1) ^ ((r >> 2) & 1));
}

template <int kTB, int kWavesWG, bool kWhole>
__global__ __launch_bounds__(kWavesWG *kWave, kWavesWG / 4) void afx_gemm_t_kernel(const TArgs p) {
    constexpr uint32_t kRowWaves = kWavesWG / kColWaves, kCols = slab_cols(kWhole), kUnits = slab_units(kWhole);
    struct Lds {
        uint32_t plut[kLutEntries];  // 16 KB, at address 0 (afx_gemv_body.h)
        uint32_t stage[kWavesWG][kStage / 4];
        LutScratch scratch;
    };
    __shared__ __attribute__((aligned(1024))) Lds lds;
    const uint32_t lane = threadIdx.x & (kWave - 1), q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t wc = wave % kColWaves, wr = wave / kColWaves;
    // Block b runs on XCD b mod 8: an XCD takes neighbouring ranges of a matrix.
    const uint32_t mat = p.n_mats == 2 ? (blockIdx.x >> 3) & 1 : 0;
    const uint32_t k = p.n_mats == 2 ? (blockIdx.x >> 4) * 8 + (blockIdx.x & 7) : blockIdx.x;
    if (k >= p.split.ranges) return;
    const uint32_t range = xcd_rank(k, p.split.ranges);
    const TensorDesc T = mat ? p.w[1] : p.w[0];
    const uint16_t *d = mat ? p.d[1] : p.d[0];
    const uint32_t len = threadIdx.x < 256 ? T.code_len[threadIdx.x] : 0u;
    const uint32_t s0 = range_begin(p.split, range), s1 = range_begin(p.split, range + 1);
    const uint32_t blocks = p.split.tile_slabs;  // slabs down a tile
    const uint32_t tile0 = s0 / blocks, tile1 = (s1 - 1) / blocks;
    const uint32_t last_end = s1 - tile1 * blocks;

    // The wave's slabs in order: block b of tile t, kRowWaves apart.
    struct At {
        uint32_t t, b;
    };
    auto settle = [&](At a) {  // a, or where its tile has no such block the wave's next slab
        if (a.b < (a.t == tile1 ? last_end : blocks)) return a;
        const bool none = wr >= blocks || (a.t + 1 == tile1 && wr >= last_end);
        return At{none ? tile1 + 1 : a.t + 1, wr};
    };
    auto next = [&](At a) { return settle(At{a.t, a.b + kRowWaves}); };
    auto there = [&](At a) { return a.t <= tile1; };

    const uint32_t c = lane & 1, lrow = lane >> 1;  // the lane's half and row when loading code words
    uint8_t *stage = reinterpret_cast<uint8_t *>(lds.stage[wave]);
    uint32_t *seg_w = lds.stage[wave] + lrow * kRowSlice;
    const uint32_t *seg = lds.stage[wave] + (lane & 15) * kRowSlice;
    auto put = [&](uint32_t i, uint4 v) {  // words i .. i + 3, reversed
        *reinterpret_cast<uint4 *>(seg_w + kRowRev - 3 - i) = make_uint4(v.w, v.z, v.y, v.x);
    };
    auto col0_of = [&](At a) { return min(a.t * kColWaves + wc, p.col_slabs - 1) * kCols; };
    auto e0_of = [&](At a) { return (uint64_t)a.b * kTRows * p.cols + col0_of(a); };
    // (from the group that the slab's first value lies in)
    auto tile_of = [&](At a) { return tile_at(T, e0_of(a) & ~(uint64_t)(kGroup - 1)); };
    // Rows past the matrix repeat the last one.
    auto row_of = [&](At a, uint32_t r) { return umin32(r, p.rows - 1 - a.b * kTRows) * p.cols; };
    auto shift_of = [&](At a, uint32_t r) {  // columns between the first group's start and the slab's first
        return kWhole ? 0u : ((uint32_t)e0_of(a) + row_of(a, r)) & (kGroup - 1);
    };
    auto seg_of = [&](At a, uint32_t r) {
        if constexpr (kWhole) return Seg{row_of(a, r), umin32(kTCols, p.cols - col0_of(a))};
        const uint32_t start = (((uint32_t)e0_of(a) & (kGroup - 1)) + row_of(a, r)) & ~(kGroup - 1);
        const uint32_t left = (tile_of(a).left + kGroup - 1) & ~(kGroup - 1);  // the last group may be part empty
        return Seg{start, umin32(kTCols, left - start)};
    };

    Words words;
    Bits bits;
    u32x4 w0, w1, sm[4];
    auto load_bits = [&](At a) { bits = seg_bits(tile_of(a), seg_of(a, lrow), c); };
    auto load_words = [&] {
        w0 = __builtin_bit_cast(u32x4, load_words4(T, words.wa + 4 * c));
        w1 = __builtin_bit_cast(u32x4, load_words4(T, words.wa + 8 + 4 * c));
    };
    auto load_sm = [&](At a) {  // 8 lanes a row; read once: not kept in the caches
        const uint8_t *at = tile_of(a).sm;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const Seg g = seg_of(a, 8 * i + (lane >> 3));
            sm[i] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(at + g.start + umin32(16 * (lane & 7), g.len - 16)));
        }
    };
    // Tokens past the last, and rows past d's, come as zeros.
    constexpr uint32_t kPastEnd = 0x80000000u;
    const auto drsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(d), (short)0,
                                                         (int)(((p.m - 1) * p.lda + p.ak) * 2), 0x00020000);
    u32x4 dv[kTB];
    auto load_d = [&](At a) {
        const uint32_t row = a.b * kTRows + 8 * q;
#pragma unroll
        for (int i = 0; i < kTB; ++i) {
            const uint32_t t = kTok * i + (lane & 15);
            dv[i] = __builtin_amdgcn_raw_buffer_load_b128(
                drsrc, (int)(t < p.m && row < p.ak ? (uint32_t)(t * p.lda + row) * 2 : kPastEnd), 0, 0);
        }
    };

    At cur = settle(At{tile0, s0 - tile0 * blocks + wr}), nxt = cur;
    if (there(cur)) {
        load_bits(cur);
        words = seg_words_of<2, kRowWords, kRowMaxStart>(T, bits);
        load_words();
        nxt = next(cur);
        if (there(nxt)) load_bits(nxt);
    }
    [[clang::always_inline]] build_lut<kWavesWG * kWave, true>(len, lds.plut, lds.scratch);
    __syncthreads();

    f32x4 acc[kUnits][kTB];
    for (uint32_t t = tile0; t <= tile1; ++t) {
#pragma unroll
        for (uint32_t u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < kTB; ++i) acc[u][i] = f32x4{};
        while (cur.t == t) {
            // The words requested a slab ago (pinned here, or the compiler
            // moves their reversal, and so the wait for them, up to the request).
            asm volatile("" : "+v"(w0), "+v"(w1));
            put(4 * c, __builtin_bit_cast(uint4, w0));
            put(8 + 4 * c, __builtin_bit_cast(uint4, w1));
            for (uint32_t i = 16 + 4 * c; i < words.nw; i += 8) put(i, load_words4(T, words.wa + i));
            // The counters of the chains of the lane's groups: group q of rows
            // l mod 16 and 16 + l mod 16 (whose slice is 16 slices on).
            const int at = (int)(8 * (lane & 15) + 4 * (lane >> 5));  // lane 2 row + q / 2
            const uint32_t v1 = (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)words.starts);
            const uint32_t v2 = (uint32_t)__builtin_amdgcn_ds_bpermute(at + 128, (int)words.starts);
            const uint32_t shift = lane & 16;  // q odd: the high half
            const uint32_t r1 = 32 * kRowRev + kLead - ((v1 >> shift) & 0xFFFF);
            const uint32_t r2 = 32 * (kRowRev + 16 * kRowSlice) + kLead - ((v2 >> shift) & 0xFFFF);
            // All that is requested here arrives while the slab decodes: its
            // sign/mantissa bytes and tokens, the next slab's words, the one
            // after's offsets.
            load_sm(cur);
            const At aft = there(nxt) ? next(nxt) : nxt;
            if (there(nxt)) {
                words = seg_words_of<2, kRowWords, kRowMaxStart>(T, bits);
                load_words();
            }
            if (there(aft)) load_bits(aft);
            wave_sync();
            uint32_t ex[2][8];
            BufChain A = buf_chain(seg, r1), B = buf_chain(seg, r2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t a01, b01, a23, b23;
                pair_chain_steps(A, B, seg, lds.plut, a01, b01);
                pair_chain_steps(A, B, seg, lds.plut, a23, b23);
                ex[0][j] = join_entries(a01, a23);
                ex[1][j] = join_entries(b01, b23);
            }
            wave_sync();  // the staged words have been read
            // (LDS addresses are formed here, not held across the decode: registers)
            uint32_t ln = lane;
            asm volatile("" : "+v"(ln));
            uint8_t *sm_w = stage + (ln >> 3) * kSmRow + 16 * (ln & 7);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) *reinterpret_cast<u32x4 *>(sm_w + 8 * i * kSmRow) = sm[i];
            wave_sync();
            load_d(cur);
            // 16 rows at a time: the first 16 restored rows go behind the bytes,
            // the others in their place.
            const uint8_t *sm_r = stage + (ln & 15) * kSmRow + kGroup * (ln >> 4);
            // (piece j of a group changes bits 4 and 5 of the address)
            const uint32_t put_at = piece_at(ln & 15, 4 * (ln >> 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // rows past the matrix become zeros (their tokens' operand is, but 0 times infinity is not)
                const uint32_t in = cur.b * kTRows + 16 * h + (ln & 15) < p.rows ? ~0u : 0u;
                uint4 wf[4];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(sm_r + 16 * h * kSmRow + 8 * j);
                    join4(b.x & in, ex[h][2 * j] & in, wf[j].x, wf[j].y);
                    join4(b.y & in, ex[h][2 * j + 1] & in, wf[j].z, wf[j].w);
                    join4(b.z & in, ex[h][2 * j + 2] & in, wf[j + 1].x, wf[j + 1].y);
                    join4(b.w & in, ex[h][2 * j + 3] & in, wf[j + 1].z, wf[j + 1].w);
                }
                if (h == 1) wave_sync();  // the bytes have been read
                uint8_t *half = stage + (h == 0 ? kTRows * kSmRow : 0);
                const uint32_t first = 4 * (ln >> 4) - shift_of(cur, 16 * h + (ln & 15)) / 8;  // the lane's first piece
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    if constexpr (kWhole)
                        *reinterpret_cast<uint4 *>(half + (put_at ^ (16 * j))) = wf[j];
                    else if (first + j < kCols / 8)  // (before the slab: a large number)
                        *reinterpret_cast<uint4 *>(half + piece_at(ln & 15, first + j)) = wf[j];
                }
            }
            wave_sync();
            // Columns 16 u .. of rows 8 q .. 8 q + 7, transposed: 16 lanes read
            // 4 rows of a unit, 8 bytes each, and get 4 rows of a column each.
            asm volatile("" : "+v"(ln));
            const uint32_t row = 8 * ((ln >> 4) & 1) + ((ln & 15) >> 2);
            const uint32_t row_at = (ln & 32 ? 0 : kTRows * kSmRow) + row * (kTCols * 2) + 8 * (ln & 3);
            const uint32_t sw = 32 * row_swizzle(row);
#pragma unroll
            for (uint32_t u = 0; u < kUnits; ++u) {
                typedef __attribute__((address_space(3))) s16x4 *Lds4;
                const uint32_t a = row_at + ((32 * u) ^ sw);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(stage + a));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(stage + (a ^ 16) + 4 * (kTCols * 2)));
                const s16x8 w = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int i = 0; i < kTB; ++i)
                    acc[u][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, dv[i]), acc[u][i], 0, 0, 0);
            }
            wave_sync();  // the slab has been read: the next one's words may be staged
            cur = nxt;
            nxt = aft;
        }
        // The tile, or the range, ends: the waves' sums, in order, go to their
        // place. Value e of unit u is column 16 u + 4 q + e of token l mod 16.
        const uint64_t place = part_place(p.split, t, range - range_of(p.split, t * blocks), 0);
        f32x4 *out = reinterpret_cast<f32x4 *>(p.part + mat * p.part_mat) + place * kTB * kColWaves * (kUnits * kWave);
#pragma unroll
        for (int i = 0; i < kTB; ++i) {
#pragma unroll
            for (uint32_t u = 0; u < kUnits; ++u) reinterpret_cast<f32x4 *>(stage)[u * kWave + lane] = acc[u][i];
            __syncthreads();
            for (uint32_t f = threadIdx.x; f < kColWaves * kUnits * kWave; f += kWavesWG * kWave) {
                const uint32_t cw = f / (kUnits * kWave), e = f % (kUnits * kWave);
                f32x4 v = f32x4{};
                for (uint32_t w = 0; w < kRowWaves; ++w)
                    v += reinterpret_cast<const f32x4 *>(lds.stage[w * kColWaves + cw])[e];
                out[(i * kColWaves) * (kUnits * kWave) + f] = v;
            }
            __syncthreads();
        }
    }
}

// A slab's columns of 16 tokens: both matrices' ranges in order.
template <bool kWhole>
__global__ __launch_bounds__(slab_units(kWhole) * kWave) void afx_gemm_t_join_kernel(const TArgs p, uint32_t blocks) {
    constexpr uint32_t kCols = slab_cols(kWhole), kUnits = slab_units(kWhole);
    const uint32_t tile = blockIdx.x / kColWaves, cw = blockIdx.x % kColWaves, tb = blockIdx.y;
    const uint32_t lane = threadIdx.x % kWave, t = tb * kTok + (lane & 15);
    const uint32_t col = blockIdx.x * kCols + 16 * (threadIdx.x / kWave) + 4 * (lane >> 4);
    if (t >= p.m || col >= p.cols) return;
    const uint32_t first = range_of(p.split, tile * p.split.tile_slabs);
    const uint32_t n = range_of(p.split, (tile + 1) * p.split.tile_slabs - 1) - first + 1;
    f32x4 v = f32x4{};
    for (uint32_t mat = 0; mat < p.n_mats; ++mat) {
        const f32x4 *in = reinterpret_cast<const f32x4 *>(p.part + mat * p.part_mat) +
                          ((part_place(p.split, tile, 0, 0) * blocks + tb) * kColWaves + cw) * (kUnits * kWave) +
                          threadIdx.x;
#pragma unroll 8
        for (uint32_t o = 0; o < n; ++o) v += in[(uint64_t)o * blocks * kColWaves * (kUnits * kWave)];
    }
    if (p.y16) {
        uint16_t *y = p.y16 + t * p.ldy + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
    } else {
        float *y = p.y32 + t * p.ldy + col;
        if (((p.ldy & 3) | (reinterpret_cast<uintptr_t>(p.y32) & 15)) == 0) {
            f32x4 *y4 = reinterpret_cast<f32x4 *>(y);
            *y4 = p.add ? *y4 + v : v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = p.add ? y[e] + v[e] : v[e];
        }
    }
}

uint32_t token_blocks(uint32_t m) { return (m + kTok - 1) / kTok; }

// Waves of a workgroup: 128 registers a lane hold 16 tokens' sums, 256 more.
uint32_t workgroup_waves(uint32_t m) { return m <= kTok ? 16 : 8; }

// One workgroup per CU of 256, divided between the matrices, and no more than
// have a slab for each of their waves down a tile (1000 x 1000, 20 tokens: 24
// us with one slab a workgroup, 17 so). On a device with fewer CUs the rest
// follow: the split does not depend on the device.
bool whole_groups(uint64_t cols) { return cols % kGroup == 0; }
uint32_t col_slabs(uint64_t cols) {
    const uint32_t each = slab_cols(whole_groups(cols));
    return (uint32_t)((cols + each - 1) / each);
}
GatedSplit t_split(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    GatedSplit s{};
    s.waves = 1;
    s.tile_slabs = (uint32_t)((rows + kTRows - 1) / kTRows);
    s.tiles = s.row_tiles = (col_slabs(cols) + kColWaves - 1) / kColWaves;
    const uint64_t each = (uint64_t)s.tiles * s.tile_slabs / (workgroup_waves(m) / kColWaves);
    return with_ranges(s, (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(each, 256 / n_mats)));
}
uint64_t part_floats(const GatedSplit &s, uint64_t cols, uint32_t m) {
    return part_places(s) * token_blocks(m) * kColWaves * slab_cols(whole_groups(cols)) * kTok;
}

template <bool kWhole>
int launch(TArgs &p, uint32_t blocks, hipStream_t stream) {
    const void *fn = reinterpret_cast<const void *>(&afx_gemm_t_kernel<1, 16, kWhole>);
    if constexpr (kWhole) {
        if (blocks == 2) fn = reinterpret_cast<const void *>(&afx_gemm_t_kernel<2, 8, true>);
        if (blocks == 3) fn = reinterpret_cast<const void *>(&afx_gemm_t_kernel<3, 8, true>);
        if (blocks == 4) fn = reinterpret_cast<const void *>(&afx_gemm_t_kernel<4, 8, true>);
    }
    const uint32_t grid = p.n_mats * (p.n_mats == 2 ? (p.split.ranges + 7) / 8 * 8 : p.split.ranges);
    void *args[] = {&p};  // hipLaunchKernel reports this launch's own status
    if (hipLaunchKernel(fn, dim3(grid), dim3(workgroup_waves(p.m) * kWave), args, 0, stream) != hipSuccess) return AFX_E_HIP;
    void *join_args[] = {&p, &blocks};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_gemm_t_join_kernel<kWhole>), dim3(p.col_slabs, blocks),
                           dim3(slab_units(kWhole) * kWave), join_args, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

}  // namespace

uint64_t gemm_t_space(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    return n_mats * part_floats(t_split(rows, cols, n_mats, m), cols, m) * 4;
}

int launch_gemm_t(const GemmT &q, uint8_t *ws, hipStream_t stream) {
    TArgs p{};
    for (uint32_t i = 0; i < q.n_mats; ++i) {
        p.w[i] = tensor(q.info[i], q.blob[i]);
        p.d[i] = q.d[i];
    }
    p.lda = q.lda;
    p.split = t_split(q.rows, q.cols, q.n_mats, q.m);
    p.part = reinterpret_cast<float *>(ws);
    p.part_mat = part_floats(p.split, q.cols, q.m);
    p.n_mats = q.n_mats;
    p.m = q.m;
    p.rows = (uint32_t)q.rows;
    p.cols = (uint32_t)q.cols;
    p.ak = (uint32_t)((q.rows + 7) / 8 * 8);
    p.col_slabs = col_slabs(q.cols);
    p.y32 = q.y32;
    p.y16 = q.y16;
    p.ldy = q.ldy;
    p.add = q.add;
    const uint32_t blocks = token_blocks(q.m);
    return whole_groups(q.cols) ? launch<true>(p, blocks, stream) : launch<false>(p, blocks, stream);
}

}  // namespace afx
