// afx_gated_gemm.hip -- the gated block for up to 128 tokens (gfx950): both
// projections restored and multiplied on the matrix cores, then the
// activation and the product. No restored weight reaches memory, or LDS.
//
// A slab is 16 weight rows by 256 columns: 128 groups of 32 values, which
// decode on their own, two per lane. Lane l takes row l mod 16 and the
// groups q = l / 16 and q + 4 of it; the 32 values of a group, 8 at a time,
// are then just what lane l feeds v_mfma_f32_16x16x32_bf16 for row l mod 16,
// if its four lanes per row may take any 32 columns between them, and they
// may: the order of a sum's terms is free as long as the tokens' operand has
// the same. So x is first copied into that order, each operand's 1 KB in one
// piece (x's own rows, 2 cols bytes apart, would fall into a few sets of the
// L1).
//
// What bounds it: at 16 tokens (two 17408 x 5120 matrices, 89 us; their coded
// bytes alone 40) vector instructions are issued for 47 us and LDS is busy for
// 42, 61% of that in bank conflicts of the table's reads. Neither is full: a
// wave's chains wait for one and the other in turn, and four waves a SIMD
// hide only part of it. From there on the tokens' operands add to it (48
// tokens: 118). So the waves are independent of each other: every wave stages
// its own rows' code words, reads the workgroup's pair table, and shares no
// barrier after that is built. They do go through the same columns at about the same time, so that
// the CU's L1 serves most of their tokens' operands. The slabs of all tiles
// (16 rows per wave), in order, are cut into one contiguous range per
// workgroup; a range's sums for a tile go to the workspace in FP32, and a
// last launch adds a tile's ranges in order and forms h: the same bits on
// every run.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "afx_act.h"
#include "afx_gated_gemm.h"
#include "afx_segments.h"

namespace afx {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kTok = kGatedTokenBlock;
constexpr uint32_t kSlabSteps = kSlabCols / 32;  // matrix instructions per slab and token block
static_assert(kSegWords * 32 >= kSlabCols * kMaxLen + 5 * 32, "a segment's words fit its slice");

struct SlabArgs {
    TensorDesc w[2];     // gate, up
    const uint16_t *xp;  // x in operand order: [slab][step][token block][lane][8]
    float *part[2];      // [part_places][token blocks][16 tokens][16 rows]
    uint32_t m, rows, cols, blocks;  // blocks: token blocks
    GatedSplit split;
};

// Operand step (half, j) of a slab: lane l holds columns 128 half + 32 (l /
// 16) + 8 j .. + 7 of token l mod 16.
__global__ __launch_bounds__(256) void afx_gated_pack_kernel(const uint16_t *x, uint64_t ldx, uint32_t m,
                                                             uint32_t cols, uint32_t blocks, uint16_t *out) {
    // one wave per operand; operand o of (slab, step, token block)
    const uint32_t o = blockIdx.x * 4 + threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const uint32_t tb = o % blocks, step = o / blocks % kSlabSteps, slab = o / blocks / kSlabSteps;
    const uint32_t col = slab * kSlabCols + 128 * (step / 4) + 32 * (lane / 16) + 8 * (step % 4);
    const uint32_t t = tb * kTok + lane % 16;
    if (slab * kSlabCols >= cols) return;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < m && col < cols) v = *reinterpret_cast<const uint4 *>(x + t * ldx + col);
    *reinterpret_cast<uint4 *>(out + ((uint64_t)o * kWave + lane) * 8) = v;
}

// The counters of the chains of the lane's groups q and q + 4 of row l mod 16.
__device__ inline void chain_starts(uint32_t starts, uint32_t lane, uint32_t &r1, uint32_t &r2) {
    const int at = (int)(16 * (lane & 15) + 4 * (lane >> 5));  // lane 4 row + q / 2
    const uint32_t v1 = (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)starts);
    const uint32_t v2 = (uint32_t)__builtin_amdgcn_ds_bpermute(at + 8, (int)starts);
    const uint32_t shift = lane & 16;  // q odd: the high half
    r1 = 32 * kSegRev + kLead - ((v1 >> shift) & 0xFFFF);
    r2 = 32 * kSegRev + kLead - ((v2 >> shift) & 0xFFFF);
}

// The 32 exponent codes of the lane's two groups through the pair table (the
// chains start kLead bits early, so the pad word above the staged words may
// be read, never used).
__device__ inline void decode_pairs(const uint32_t *seg, uint32_t r1, uint32_t r2, const uint32_t *plut,
                                    uint32_t (&ex1)[8], uint32_t (&ex2)[8]) {
    BufChain A = buf_chain(seg, r1), B = buf_chain(seg, r2);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        uint32_t a01, b01, a23, b23;
        pair_chain_steps(A, B, seg, plut, a01, b01);
        pair_chain_steps(A, B, seg, plut, a23, b23);
        ex1[q] = join_entries(a01, a23);
        ex2[q] = join_entries(b01, b23);
    }
}

// A row's sign/mantissa bytes in the wave's stage slice, after the decode.
constexpr uint32_t kSmRow = kSlabCols + 16;
static_assert(16 * kSmRow <= 16 * kSegRow * 4, "they fit the slice");

template <int kWavesWG>
struct SlabLds {
    uint32_t plut[kLutEntries];               // 16 KB, at address 0 (afx_gemv_body.h)
    uint32_t stage[kWavesWG][16 * kSegRow];   // 6.9 KB a wave
    LutScratch scratch;
};

// kTB: token blocks of 16. One workgroup runs on a CU: 16 waves up to 64 tokens
// (128 registers), 8 above, whose token operands take more of the LDS.
template <int kTB>
__global__ __launch_bounds__(gated_waves(kTB) *kWave, gated_waves(kTB) / 4)
void afx_gated_gemm_kernel(const SlabArgs p) {
    constexpr int kWavesWG = gated_waves(kTB);
    __shared__ __attribute__((aligned(16))) SlabLds<kWavesWG> lds;
    // Where a slab's token operands come from: the L1 (each 16 tokens cost 15
    // us more on 17408 x 5120: the L1's rate), or LDS, where they are put once
    // for all waves, which then wait for each other twice a slab (20 us, then
    // 5 us per 16 tokens). Measured, L1 and LDS: 16 tokens 91 and 111 us, 32 105
    // and 117, 48 121 and 122, 64 134 and 125.
    constexpr bool kDirect = kTB <= 3;
    __shared__ __attribute__((aligned(16))) uint8_t xs[kDirect ? 16 : kSlabSteps * kTB * 1024];
    const uint32_t lane = threadIdx.x & (kWave - 1), q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t mat = blockIdx.x & 1, range = blockIdx.x >> 1;
    const TensorDesc T = mat ? p.w[1] : p.w[0];
    const uint32_t len = threadIdx.x < 256 ? T.code_len[threadIdx.x] : 0u;
    const uint32_t s0 = range_begin(p.split, range), s1 = range_begin(p.split, range + 1);

    const uint32_t c = lane & 3, lrow = lane >> 2;  // the lane's part and row when loading
    uint32_t *seg_w = lds.stage[wave] + lrow * kSegRow;
    const uint32_t *seg = lds.stage[wave] + (lane & 15) * kSegRow;
    uint8_t *sm_w = reinterpret_cast<uint8_t *>(lds.stage[wave]) + lrow * kSmRow + 16 * c;
    const uint8_t *sm_r = reinterpret_cast<const uint8_t *>(lds.stage[wave]) + (lane & 15) * kSmRow + kGroup * q;
    uint32_t tile = s0 / p.split.tile_slabs, k0 = (s0 - tile * p.split.tile_slabs) * kSlabCols;
    // The wave's 16 rows of tile t, and the lane's part of a slab. Rows past
    // the matrix repeat its last ones; their sums are not used.
    auto rows_of = [&](uint32_t t) { return min(t * p.split.waves + wave, p.split.row_tiles - 1); };
    auto tile_of = [&](uint32_t t) { return tile_at(T, (uint64_t)rows_of(t) * kGatedWaveRows * p.cols); };
    auto segment = [&](uint32_t t, uint32_t k) {
        return Seg{umin32(lrow, p.rows - 1 - rows_of(t) * kGatedWaveRows) * p.cols + k, umin32(kSlabCols, p.cols - k)};
    };
    auto next = [&](uint32_t &t, uint32_t &k) {  // the slab after
        k += kSlabCols;
        if (k >= p.cols) {
            k = 0;
            ++t;
        }
    };
    uint32_t tile_n = tile, k0_n = k0;  // the slab after
    if (s0 + 1 < s1) next(tile_n, k0_n);
    Words words;
    Bits bits;
    u32x4 w0, w1, sm[4];  // the lane's 8 of the row's first 32 words; 4 of 16 times 16 sign/mantissa bytes
    auto load_bits = [&](uint32_t t, uint32_t k) {
        bits = seg_bits(tile_of(t), segment(t, k), c);
    };
    auto load_words = [&] {
        w0 = __builtin_bit_cast(u32x4, load_words4(T, words.wa + 4 * c));
        w1 = __builtin_bit_cast(u32x4, load_words4(T, words.wa + 16 + 4 * c));
    };
    auto load_sm = [&](uint32_t t, uint32_t k) {  // read once: not kept in the caches
        const Seg g = segment(t, k);
        const uint8_t *row = tile_of(t).sm;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            sm[i] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4 *>(row + g.start + min(64 * i + 16 * c, g.len - 16)));
    };
    load_bits(tile, k0);
    words = seg_words_of<4, kSegWords, kSegMaxStart>(T, bits);
    load_words();
    load_bits(tile_n, k0_n);
    [[clang::always_inline]] build_lut<kWavesWG * kWave, true>(len, lds.plut, lds.scratch);
    __syncthreads();
    const bool active = wave < p.split.waves;
    if (kDirect && !active) return;
    f32x4 acc[kTB];
#pragma unroll
    for (int b = 0; b < kTB; ++b) acc[b] = f32x4{};
    const auto xrsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(p.xp), (short)0, (int)(p.split.tile_slabs * kSlabSteps * kTB * 1024), 0x00020000);
    for (uint32_t s = s0; s < s1; ++s) {
        // The words requested a slab ago (pinned here, or the compiler moves
        // their reversal, and so the wait for them, up to the request).
        asm volatile("" : "+v"(w0), "+v"(w1));
        put_seg4(seg_w, 4 * c, __builtin_bit_cast(uint4, w0));
        put_seg4(seg_w, 16 + 4 * c, __builtin_bit_cast(uint4, w1));
        for (uint32_t i = 32 + 4 * c; i < words.nw; i += 16) put_seg4(seg_w, i, load_words4(T, words.wa + i));
        uint32_t r1, r2;
        chain_starts(words.starts, lane, r1, r2);
        if constexpr (!kDirect) {
            __syncthreads();  // every wave is done with the last slab's token operands
            for (uint32_t o = wave; o < kSlabSteps * kTB; o += kWavesWG)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    xrsrc, (__attribute__((address_space(3))) void *)(xs + o * 1024), 16,
                    (int)((k0 / kSlabCols * kSlabSteps * kTB + o) * 1024 + lane * 16), 0, 0, 0);
        }
        // All that is requested here arrives while the slab decodes: its
        // sign/mantissa bytes, the next slab's words, the one after's offsets.
        load_sm(tile, k0);
        if (s + 1 < s1) {
            words = seg_words_of<4, kSegWords, kSegMaxStart>(T, bits);
            load_words();
        }
        if (s + 2 < s1) {
            uint32_t t2 = tile_n, k2 = k0_n;
            next(t2, k2);
            load_bits(t2, k2);
        }
        wave_sync();
        uint32_t ex1[8], ex2[8];
        decode_pairs(seg, r1, r2, lds.plut, ex1, ex2);
        wave_sync();  // the staged words have been read
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) *reinterpret_cast<u32x4 *>(sm_w + 64 * i) = sm[i];
        wave_sync();
        // columns past the row's end become zeros
        const uint32_t in1 = k0 + kGroup * q < p.cols ? ~0u : 0u, in2 = k0 + kGroup * (q + 4) < p.cols ? ~0u : 0u;
        uint4 wf[kSlabSteps];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const uint4 m1 = *reinterpret_cast<const uint4 *>(sm_r + 8 * j);
            const uint4 m2 = *reinterpret_cast<const uint4 *>(sm_r + 128 + 8 * j);
            join4(m1.x & in1, ex1[2 * j] & in1, wf[j].x, wf[j].y);
            join4(m1.y & in1, ex1[2 * j + 1] & in1, wf[j].z, wf[j].w);
            join4(m1.z & in1, ex1[2 * j + 2] & in1, wf[j + 1].x, wf[j + 1].y);
            join4(m1.w & in1, ex1[2 * j + 3] & in1, wf[j + 1].z, wf[j + 1].w);
            join4(m2.x & in2, ex2[2 * j] & in2, wf[4 + j].x, wf[4 + j].y);
            join4(m2.y & in2, ex2[2 * j + 1] & in2, wf[4 + j].z, wf[4 + j].w);
            join4(m2.z & in2, ex2[2 * j + 2] & in2, wf[5 + j].x, wf[5 + j].y);
            join4(m2.w & in2, ex2[2 * j + 3] & in2, wf[5 + j].z, wf[5 + j].w);
        }
        wave_sync();  // the bytes have been read: the next slab's words may be staged
        if constexpr (kDirect) {
            __builtin_amdgcn_sched_barrier(0);  // (not requested before the decode: registers)
            constexpr uint32_t kAhead = kTB == 1 ? 6 : kTB == 2 ? 3 : kTB == 3 ? 2 : 1;
            u32x4 xv[kSlabSteps][kTB];
            auto load_step = [&](uint32_t st) {
#pragma unroll
                for (int b = 0; b < kTB; ++b)
                    xv[st][b] = __builtin_amdgcn_raw_buffer_load_b128(
                        xrsrc, (int)(lane * 16), (int)((k0 / kSlabCols * kSlabSteps * kTB + st * kTB + b) * 1024), 0);
            };
#pragma unroll
            for (uint32_t st = 0; st < kAhead; ++st) load_step(st);
#pragma unroll
            for (uint32_t st = 0; st < kSlabSteps; ++st) {
                if (st + kAhead < kSlabSteps) load_step(st + kAhead);
                __builtin_amdgcn_sched_barrier(0);  // (the compiler would request them later)
#pragma unroll
                for (int b = 0; b < kTB; ++b)
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, wf[st]), __builtin_bit_cast(bf16x8, xv[st][b]), acc[b], 0, 0, 0);
            }
        } else {
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's share of the operands is in LDS
            __syncthreads();                     // and every wave's
            if (active) {
#pragma unroll
                for (uint32_t st = 0; st < kSlabSteps; ++st)
#pragma unroll
                    for (int b = 0; b < kTB; ++b) {
                        const uint4 xv = *reinterpret_cast<const uint4 *>(xs + (st * kTB + b) * 1024 + lane * 16);
                        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[st]),
                                                                         __builtin_bit_cast(bf16x8, xv), acc[b], 0, 0, 0);
                    }
            }
        }
        const uint32_t tile_c = tile;
        tile = tile_n;
        k0 = k0_n;
        next(tile_n, k0_n);
        if (tile == tile_c && s + 1 < s1) continue;
        // The tile, or the range, ends: its sums go to their place. The
        // lane's four are rows 4 q .. of token l mod 16.
        const uint64_t place =
            part_place(p.split, tile_c, range - range_of(p.split, tile_c * p.split.tile_slabs), wave);
        f32x4 *out = reinterpret_cast<f32x4 *>(p.part[mat]) + place * kTB * kWave + 4 * (lane & 15) + q;
#pragma unroll
        for (int b = 0; b < kTB; ++b) {
            if (active) out[b * kWave] = acc[b];
            acc[b] = f32x4{};
        }
    }
}

// h of 16 rows and 16 tokens: the tile's ranges in order.
template <uint32_t kAct>
__global__ __launch_bounds__(256) void afx_gated_gemm_join_kernel(const SlabArgs p, const GatedGemm q) {
    const uint32_t tile = blockIdx.x / p.split.waves, wave = blockIdx.x % p.split.waves;
    const uint32_t f = blockIdx.x * kGatedWaveRows + threadIdx.x % 16, t = blockIdx.y * kTok + threadIdx.x / 16;
    if (t >= p.m || f >= p.rows) return;
    const uint32_t first = range_of(p.split, tile * p.split.tile_slabs);
    const uint32_t n = range_of(p.split, (tile + 1) * p.split.tile_slabs - 1) - first + 1;
    float g = 0.f, u = 0.f;
    for (uint32_t o = 0; o < n; ++o) {
        const uint64_t at = (part_place(p.split, tile, o, wave) * p.blocks + blockIdx.y) * 256 + threadIdx.x;
        g += p.part[0][at];
        u += p.part[1][at];
    }
    q.h[(uint64_t)t * q.ldh + f] = __builtin_bit_cast(uint16_t, (__bf16)(act<kAct>(g) * u));
    if (q.g) {
        q.g[(uint64_t)t * q.ldgu + f] = __builtin_bit_cast(uint16_t, (__bf16)g);
        q.u[(uint64_t)t * q.ldgu + f] = __builtin_bit_cast(uint16_t, (__bf16)u);
    }
}

uint64_t align_up(uint64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
uint64_t part_bytes(const GatedSplit &s, uint32_t m) {
    return align_up(part_places(s) * gated_token_blocks(m) * kTok * kGatedWaveRows * 4);
}
uint64_t packed_bytes(const GatedSplit &s, uint32_t m) {
    return (uint64_t)s.tile_slabs * kSlabCols * gated_token_blocks(m) * kTok * 2;
}

bool launch(const void *fn, dim3 grid, uint32_t threads, void **args, hipStream_t stream) {
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, stream) == hipSuccess;
}

}  // namespace

uint64_t gated_gemm_space(uint64_t rows, uint64_t cols, uint32_t m) {
    const GatedSplit s = gated_split(rows, cols, m);
    return 2 * part_bytes(s, m) + align_up(packed_bytes(s, m));
}

int launch_gated_gemm(const afx_gated &w, const GatedGemm &q, uint8_t *ws, hipStream_t stream) {
    SlabArgs p{};
    p.w[0] = tensor(w.gate_info, w.gate_blob_dev);
    p.w[1] = tensor(w.up_info, w.up_blob_dev);
    p.split = gated_split(w.rows, w.cols, q.m);
    const uint64_t pb = part_bytes(p.split, q.m);
    p.part[0] = reinterpret_cast<float *>(ws);
    p.part[1] = reinterpret_cast<float *>(ws + pb);
    uint16_t *packed = reinterpret_cast<uint16_t *>(ws + 2 * pb);
    p.xp = packed;
    p.m = q.m;
    p.rows = (uint32_t)w.rows;
    p.cols = (uint32_t)w.cols;
    p.blocks = gated_token_blocks(q.m);
    const uint32_t waves = gated_waves(p.blocks);
    const uint16_t *x = q.x;
    uint64_t ldx = q.ldx;
    void *pack_args[] = {&x, &ldx, &p.m, &p.cols, &p.blocks, &packed};
    const uint32_t operands = p.split.tile_slabs * kSlabSteps * p.blocks;
    if (!launch(reinterpret_cast<const void *>(&afx_gated_pack_kernel), dim3((operands + 3) / 4), 256, pack_args, stream))
        return AFX_E_HIP;
    const void *fn = p.blocks == 1   ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<1>)
                     : p.blocks == 2 ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<2>)
                     : p.blocks == 3 ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<3>)
                     : p.blocks == 4 ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<4>)
                     : p.blocks == 6 ? reinterpret_cast<const void *>(&afx_gated_gemm_kernel<6>)
                                     : reinterpret_cast<const void *>(&afx_gated_gemm_kernel<8>);
    void *args[] = {&p};
    if (!launch(fn, dim3(2 * p.split.ranges), waves * kWave, args, stream)) return AFX_E_HIP;
    const void *join = w.act == AFX_ACT_SILU
                           ? reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_SILU>)
                       : w.act == AFX_ACT_GELU_TANH
                           ? reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_GELU_TANH>)
                           : reinterpret_cast<const void *>(&afx_gated_gemm_join_kernel<AFX_ACT_GELU>);
    GatedGemm out = q;
    void *join_args[] = {&p, &out};
    return launch(join, dim3(p.split.row_tiles, p.blocks), 256, join_args, stream) ? AFX_OK : AFX_E_HIP;
}

}  // namespace afx
