// afx_gated_gemm.hip -- the gated block for up to 128 tokens (gfx950): both
// projections restored slab by slab into LDS and multiplied there on the
// matrix cores, then the activation and the product. No restored weight
// reaches memory.
//
// The restore and the multiplication of a slab (64 weight rows by 256
// columns) are those of afx_gemm.hip. Here a tile is 32 rows of the gate
// matrix (restored by waves 0 and 1, with its decode table) and the same 32
// rows of the up matrix (waves 2 and 3), so that a wave's two accumulators
// are g and u of the same outputs.
//
// Decoding bounds this, so the work is split evenly: the slabs of all tiles,
// in order, are cut into one contiguous range per resident workgroup, whose
// loads run ahead across the ends of tiles. A range's sums for a tile go to
// the workspace in FP32, and a second launch adds a tile's ranges in order
// and forms h: the same bits on every run.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "afx_act.h"
#include "afx_gated_gemm.h"
#include "afx_slab.h"

namespace afx {
namespace {

constexpr int kWaves = 4, kSlabThreads = kWaves * kWave;
constexpr uint32_t kSlabStride = kSlabCols * 2 + 16;  // bytes per restored row in LDS
static_assert(kSegRow * 4 <= kSlabStride, "a row's staged words fit its slab row");
static_assert(kSegWords * 32 >= kSlabCols * kMaxLen + 5 * 32, "a segment's words fit its slice");

struct SlabArgs {
    TensorDesc w[2];     // gate, up
    const uint16_t *x;   // BF16 [m, cols], row stride ldx
    float *part;         // [tiles][most ranges of a tile][m][64]
    uint64_t ldx;
    uint32_t m, rows, cols;
    GatedSplit split;
};

// Bit offsets of the lane's two groups of a row segment and of the segment's
// end, kept as loaded and added up only where used.
struct Bits {
    uint64_t b1, b2, be;
    uint32_t g1, g2, ge;
    bool last;  // the segment ends the tensor
};
struct Data {  // a segment's first 32 staged words and the lane's sign/mantissa bytes
    uint64_t wa;
    uint32_t nw;
    uint4 w0, w1;
    u32x4 s1a, s1b, s2a, s2b;
};
// Where the lane's groups of a slab (columns k0.. of a tile) lie: its groups
// start at elements e1, e2, its row's elements of the slab end at e_end. A
// row past the matrix repeats its last one and a group past a row's end
// repeats the row's last one: they are decoded, not used.
struct Seg {
    uint64_t e1, e2, e_end;
};
__device__ inline Seg segment(const SlabArgs &p, uint32_t tile, uint32_t k0, uint32_t row, uint32_t q4) {
    const uint64_t row_e = (uint64_t)min(tile * kGatedTileRows + row, p.rows - 1) * p.cols;
    const uint32_t last = p.cols - kGroup;
    return Seg{row_e + min(k0 + kGroup * q4, last), row_e + min(k0 + kGroup * (q4 + 4), last),
               row_e + min(k0 + kSlabCols, p.cols)};
}
// The slab after (tile, k0).
__device__ inline void next_slab(const SlabArgs &p, uint32_t &tile, uint32_t &k0) {
    k0 += kSlabCols;
    if (k0 >= p.cols) {
        k0 = 0;
        ++tile;
    }
}
__device__ inline Bits seg_bits(const TensorDesc &T, const Seg &g) {
    Bits b;
    b.last = g.e_end >= T.n;
    b.b1 = T.chunk_base[g.e1 >> 12];
    b.g1 = T.gap[g.e1 >> 5];
    b.b2 = T.chunk_base[g.e2 >> 12];
    b.g2 = T.gap[g.e2 >> 5];
    b.be = T.chunk_base[b.last ? T.n_chunks : g.e_end >> 12];
    b.ge = T.gap[b.last ? 0 : g.e_end >> 5];
    return b;
}
__device__ inline uint64_t bit1(const Bits &b) { return b.b1 + b.g1; }
__device__ inline uint64_t bit2(const Bits &b) { return b.b2 + b.g2; }
__device__ inline uint64_t bit_end(const Bits &b) { return b.be + (b.last ? 0u : b.ge); }
__device__ inline Data seg_data(const TensorDesc &T, const Seg &g, uint32_t q4, const Bits &b) {
    Data d;
    const uint64_t p_lo = quad_first(bit1(b)), p_hi = bit_end(b);
    d.wa = seg_first_word(p_lo);
    d.nw = seg_words(p_lo, p_hi);
    d.w0 = load_words4(T, d.wa + 4 * q4);
    d.w1 = load_words4(T, d.wa + 16 + 4 * q4);
    const u32x4 *sm1 = reinterpret_cast<const u32x4 *>(T.signmant + g.e1);
    const u32x4 *sm2 = reinterpret_cast<const u32x4 *>(T.signmant + g.e2);
    d.s1a = __builtin_nontemporal_load(sm1);
    d.s1b = __builtin_nontemporal_load(sm1 + 1);
    d.s2a = __builtin_nontemporal_load(sm2);
    d.s2b = __builtin_nontemporal_load(sm2 + 1);
    return d;
}

struct SlabLds {
    uint16_t lut[2][kLutEntries];                 // 16 KB
    uint8_t slab[2 * kGatedTileRows * kSlabStride];  // 33 KB
    LutScratch scratch[2];
};

// kWays waves share a block of 32 tokens, each multiplying its share of a
// slab's 16-column steps: 32 tokens a workgroup (kWays 4), 64 (2) or 128 (1).
template <int kWays>
__global__ __launch_bounds__(kSlabThreads, 3) void afx_gated_gemm_kernel(const SlabArgs p) {
    __shared__ __attribute__((aligned(16))) SlabLds lds;
    uint8_t *slab = lds.slab;
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t s0 = range_begin(p.split, blockIdx.x), s1 = range_begin(p.split, blockIdx.x + 1);

    // Restore: this lane's row of the tile (one quad per row) and its groups.
    const uint32_t q4 = lane & 3, lrow = wave * 16 + (lane >> 2);
    const uint32_t mat = wave >> 1, mrow = lrow & (kGatedTileRows - 1);
    const TensorDesc &T = p.w[mat];
    const uint16_t *lut = lds.lut[mat];
    uint32_t *seg = reinterpret_cast<uint32_t *>(slab + lrow * kSlabStride);
    uint8_t *out_row = slab + lrow * kSlabStride;
    // Multiply: this lane's token and the wave's steps.
    constexpr uint32_t kSteps = kSlabCols / 16 / kWays;
    constexpr uint32_t kPre = kWays == 1 ? 5 : kWays == 2 ? kSteps / 2 : kSteps;  // A steps fetched before the restore
    const uint32_t t_wave = (wave / kWays) * 32, ks0 = kSteps * (wave % kWays);
    const uint32_t tok = t_wave + (lane & 31);
    const bool tok_ok = tok < p.m, wave_mul = t_wave < p.m;
    const uint32_t kx = 16 * ks0 + 8 * (lane >> 5);  // the lane's first column in a slab
    const uint16_t *xa = p.x + (uint64_t)(tok_ok ? tok : 0) * p.ldx + kx;
    const uint8_t *b_row0 = slab + (lane & 31) * kSlabStride + 16 * (lane >> 5);
    const uint8_t *b_row1 = b_row0 + 32 * kSlabStride;

    const uint32_t len0 = p.w[0].code_len[threadIdx.x], len1 = p.w[1].code_len[threadIdx.x];
    uint32_t tile = s0 / p.split.tile_slabs, k0 = (s0 - tile * p.split.tile_slabs) * kSlabCols;
    uint32_t tile_n = tile, k0_n = k0;  // the slab after
    if (s0 + 1 < s1) next_slab(p, tile_n, k0_n);
    Bits bits_c = seg_bits(T, segment(p, tile, k0, mrow, q4));
    Data data_c = seg_data(T, segment(p, tile, k0, mrow, q4), q4, bits_c);
    Bits bits_n = seg_bits(T, segment(p, tile_n, k0_n, mrow, q4));
    build_lut<kSlabThreads>(len0, lds.lut[0], lds.scratch[0]);
    build_lut<kSlabThreads>(len1, lds.lut[1], lds.scratch[1]);
    __syncthreads();
    f32x16 acc[2] = {f32x16{}, f32x16{}};
    for (uint32_t s = s0; s < s1; ++s) {
        put_seg4(seg, 4 * q4, data_c.w0);
        put_seg4(seg, 16 + 4 * q4, data_c.w1);
        for (uint32_t i = 32 + 4 * q4; i < data_c.nw; i += 16) put_seg4(seg, i, load_words4(T, data_c.wa + i));
        // the next slab's words, the one after's offsets, this slab's tokens
        Data data_n = data_c;
        if (s + 1 < s1) data_n = seg_data(T, segment(p, tile_n, k0_n, mrow, q4), q4, bits_n);
        Bits bits_nn = bits_n;
        if (s + 2 < s1) {
            uint32_t tile_nn = tile_n, k0_nn = k0_n;
            next_slab(p, tile_nn, k0_nn);
            bits_nn = seg_bits(T, segment(p, tile_nn, k0_nn, mrow, q4));
        }
        bf16x8 xv[kSteps];
        auto load_step = [&](uint32_t ks) { return load_a(xa + k0 + 16 * ks, tok_ok && k0 + kx + 16 * ks < p.cols); };
        if (wave_mul) {
#pragma unroll
            for (uint32_t ks = 0; ks < kPre; ++ks) xv[ks] = load_step(ks);
        }
        wave_sync();
        uint32_t ex1[8], ex2[8];
        decode_groups(seg, seg_chain_r0(bit1(bits_c), data_c.wa), seg_chain_r0(bit2(bits_c), data_c.wa), lut, ex1,
                      ex2);
        wave_sync();  // the row's staged words have been read: its slab row may be written
        // columns past the row's end become zeros
        const uint32_t in1 = k0 + kGroup * q4 < p.cols ? ~0u : 0u, in2 = k0 + kGroup * (q4 + 4) < p.cols ? ~0u : 0u;
        const uint32_t b1[8] = {data_c.s1a.x, data_c.s1a.y, data_c.s1a.z, data_c.s1a.w,
                                data_c.s1b.x, data_c.s1b.y, data_c.s1b.z, data_c.s1b.w};
        const uint32_t b2[8] = {data_c.s2a.x, data_c.s2a.y, data_c.s2a.z, data_c.s2a.w,
                                data_c.s2b.x, data_c.s2b.y, data_c.s2b.z, data_c.s2b.w};
        uint4 *o1 = reinterpret_cast<uint4 *>(out_row + 64 * q4);
        uint4 *o2 = reinterpret_cast<uint4 *>(out_row + 64 * (q4 + 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 v1, v2;
            join4(b1[2 * j], ex1[2 * j], v1.x, v1.y);
            join4(b1[2 * j + 1], ex1[2 * j + 1], v1.z, v1.w);
            join4(b2[2 * j], ex2[2 * j], v2.x, v2.y);
            join4(b2[2 * j + 1], ex2[2 * j + 1], v2.z, v2.w);
            o1[j] = make_uint4(v1.x & in1, v1.y & in1, v1.z & in1, v1.w & in1);
            o2[j] = make_uint4(v2.x & in2, v2.y & in2, v2.z & in2, v2.w & in2);
        }
        __syncthreads();  // the slab is complete
        if (wave_mul) {
#pragma unroll
            for (uint32_t ks = 0; ks < kSteps; ++ks) {
                if (ks + kPre < kSteps) xv[ks + kPre] = load_step(ks + kPre);
                const uint32_t kb = 32 * (ks0 + ks);
                const bf16x8 w0 = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(b_row0 + kb));
                const bf16x8 w1 = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(b_row1 + kb));
                acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xv[ks], w0, acc[0], 0, 0, 0);
                acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xv[ks], w1, acc[1], 0, 0, 0);
            }
        }
        __syncthreads();  // every wave is done with the slab and its staged words
        bits_c = bits_n;
        bits_n = bits_nn;
        data_c = data_n;
        const uint32_t tile_c = tile;
        tile = tile_n;
        k0 = k0_n;
        next_slab(p, tile_n, k0_n);
        if (tile == tile_c && s + 1 < s1) continue;
        // The tile, or the range, ends: its sums go to their place.
        if constexpr (kWays > 1) {
            // the waves that share a token block add up in LDS, in their order
            static_assert(kWaves * 2 * 16 * kWave * 4 <= sizeof(SlabLds::slab), "partial sums fit the slab");
            float *mine = reinterpret_cast<float *>(slab) + wave * (2 * 16 * kWave);
            if (wave_mul && wave % kWays != 0) {
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    mine[v * kWave + lane] = acc[0][v];
                    mine[(16 + v) * kWave + lane] = acc[1][v];
                }
            }
            __syncthreads();
            if (wave % kWays == 0) {
#pragma unroll
                for (int w = 1; w < kWays; ++w) {
                    const float *pw = mine + w * (2 * 16 * kWave);
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        acc[0][v] += pw[v * kWave + lane];
                        acc[1][v] += pw[(16 + v) * kWave + lane];
                    }
                }
            }
            __syncthreads();  // before the next slab's words are staged there
        }
        if (wave_mul && wave % kWays == 0) {
            const uint32_t slot = tile_c * p.split.most + (blockIdx.x - range_of(p.split, tile_c * p.split.tile_slabs));
            uint32_t l = lane;
            asm volatile("" : "+v"(l));  // (the addresses are not kept in registers through the loop)
            const uint32_t t0 = t_wave + 4 * (l >> 5);
            float *out = p.part + ((uint64_t)slot * p.m + t0) * (2 * kGatedTileRows) + (l & 31);
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const uint32_t dt = 8 * (v / 4) + (v & 3);  // accumulator v is token t0 + dt
                if (t0 + dt < p.m) {
                    out[dt * (2 * kGatedTileRows)] = acc[0][v];
                    out[dt * (2 * kGatedTileRows) + kGatedTileRows] = acc[1][v];
                }
            }
        }
        acc[0] = acc[1] = f32x16{};
    }
}

// h of one tile and 8 tokens: the tile's ranges in order.
template <uint32_t kAct>
__global__ __launch_bounds__(256) void afx_gated_gemm_join_kernel(const SlabArgs p, const GatedGemm q) {
    const uint32_t tile = blockIdx.x, t = blockIdx.y * 8 + threadIdx.x / 32, c = threadIdx.x % 32;
    const uint32_t f = tile * kGatedTileRows + c;
    if (t >= p.m || f >= p.rows) return;
    const uint32_t first = range_of(p.split, tile * p.split.tile_slabs);
    const uint32_t n = range_of(p.split, (tile + 1) * p.split.tile_slabs - 1) - first + 1;
    float g = 0.f, u = 0.f;
    for (uint32_t o = 0; o < n; ++o) {
        const float *v = p.part + (((uint64_t)tile * p.split.most + o) * p.m + t) * (2 * kGatedTileRows) + c;
        g += v[0];
        u += v[kGatedTileRows];
    }
    q.h[(uint64_t)t * q.ldh + f] = __builtin_bit_cast(uint16_t, (__bf16)(act<kAct>(g) * u));
    if (q.g) {
        q.g[(uint64_t)t * q.ldgu + f] = __builtin_bit_cast(uint16_t, (__bf16)g);
        q.u[(uint64_t)t * q.ldgu + f] = __builtin_bit_cast(uint16_t, (__bf16)u);
    }
}

TensorDesc tensor(const afx_info *info, const void *blob) {
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
    return t;
}

}  // namespace

uint64_t gated_gemm_space(uint64_t rows, uint64_t cols, uint32_t m) {
    const GatedSplit s = gated_split(rows, cols);
    return (uint64_t)s.tiles * s.most * m * 2 * kGatedTileRows * 4;
}

int launch_gated_gemm(const afx_gated &w, const GatedGemm &q, uint8_t *ws, hipStream_t stream) {
    SlabArgs p{};
    p.w[0] = tensor(w.gate_info, w.gate_blob_dev);
    p.w[1] = tensor(w.up_info, w.up_blob_dev);
    p.x = q.x;
    p.part = reinterpret_cast<float *>(ws);
    p.ldx = q.ldx;
    p.m = q.m;
    p.rows = (uint32_t)w.rows;
    p.cols = (uint32_t)w.cols;
    p.split = gated_split(w.rows, w.cols);
    const void *fn = q.m <= 32   ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<4>)
                     : q.m <= 64 ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<2>)
                                 : reinterpret_cast<const void *>(&afx_gated_gemm_kernel<1>);
    void *args[] = {&p};
    if (hipLaunchKernel(fn, dim3(p.split.ranges), dim3(kSlabThreads), args, 0, stream) != hipSuccess) return AFX_E_HIP;
    const void *join = w.act == AFX_ACT_SILU
                           ? reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_SILU>)
                       : w.act == AFX_ACT_GELU_TANH
                           ? reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_GELU_TANH>)
                           : reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_GELU>);
    GatedGemm out = q;
    void *jargs[] = {&p, &out};
    return hipLaunchKernel(join, dim3(p.split.tiles, (q.m + 7) / 8), dim3(256), jargs, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

}  // namespace afx
