// afx_mm.hip -- products of BF16 activations with restored BF16 weights on
// the matrix cores (gfx950): the dense half of the gated feed-forward block
// for many tokens, and of the transposed products.
//
//   gated       g = x Wg^T, u = x Wu^T, h = act(g) u     (W rows contiguous in k)
//   transposed  y = d0 W0 [+ d1 W1]                      (W rows are the reduction)
//
// A workgroup of 8 waves takes BM tokens and 256 weight rows (gated: 128 of
// each matrix, interleaved by 32 so that a wave holds g and u of the same
// outputs) or 256 columns (transposed), 64 reduction steps at a time. Tiles
// go from memory to LDS without passing through registers (buffer loads to
// LDS, 16 bytes a lane), double-buffered: the next tile is requested right
// after the barrier that frees its buffer and has a whole tile's matrix
// instructions to arrive. Weights are the A operand of
// v_mfma_f32_16x16x32_bf16 and tokens the B operand, so that a lane's four
// accumulators are four consecutive outputs of one token.
//
// LDS layouts (the loads write lanes' 16 bytes contiguously, so the order is
// set by which 16 bytes each lane asks for):
//   * rows of 64 k (128 bytes): 16-byte chunk c of row r sits at chunk c ^
//     ((r >> 1) & 7), so that the 16 rows a 16-lane phase reads cover all 64
//     banks once;
//   * transposed weights, rows of 256 columns (512 bytes): 32-byte unit q of
//     row k sits at unit q ^ ((k & 3) | (k >> 1 & 4)); the operand's 8
//     consecutive k of one column come from two ds_read_b64_tr_b16 (a 16-lane
//     group reads 4 rows of 16 columns and gets them transposed).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "afx_act.h"
#include "afx_mm.h"

namespace afx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMmWave = 64, kMmWaves = 8, kMmThreads = kMmWave * kMmWaves;
constexpr uint32_t kBN = 256;          // weight rows (or columns) of a tile
constexpr uint32_t kBK = kMmTileK;     // reduction steps of a tile
constexpr int kBufferFlags = 0x00020000;  // raw buffer, 32-bit data format

struct MmArgs {
    const uint16_t *a;      // tokens [m, ak], row stride lda
    const uint16_t *w0, *w1;
    uint64_t lda, ldw;
    uint32_t m, n;          // tokens; outputs per token
    uint32_t ak, wk;        // reduction steps held by a; by each matrix
    uint32_t k_tiles0;      // k-tiles of the first matrix
    uint32_t k_tiles;       // k-tiles of all matrices
    uint32_t splits;        // the reduction is cut into this many ranges of k-tiles
    uint32_t m_tiles, n_tiles;
    uint16_t *h, *g, *u;    // BF16 outputs
    float *y32;
    uint64_t ldh, ldgu;     // ldh: also y32's
    uint32_t add;
};

enum MmEpilogue { kEpiGated, kEpiBf16, kEpiF32, kEpiPartial };

__device__ inline uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Four consecutive BF16 outputs of one token; n4 <= 4 of them exist.
__device__ inline void store4(uint16_t *p, const float (&v)[4], uint32_t n4, bool vec) {
    if (vec && n4 >= 4) {
        const uint32_t lo = to_bf16(v[0]) | ((uint32_t)to_bf16(v[1]) << 16);
        const uint32_t hi = to_bf16(v[2]) | ((uint32_t)to_bf16(v[3]) << 16);
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < n4) p[i] = to_bf16(v[i]);
    }
}

// 16 bytes per lane from rsrc + off straight into LDS at `to` (wave-uniform)
// + 16 lane.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint8_t *to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 16, (int)off, 0, 0,
                                             0);
}
__device__ inline __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t end) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)end, kBufferFlags);
}

template <int BM, bool kNN, int kEpi, uint32_t kAct>
__global__ __launch_bounds__(kMmThreads, 2) void afx_mm_kernel(const MmArgs p) {
    constexpr int kTokInstr = BM / 64;  // DMA instructions per wave for the token tile
    constexpr int kMT = BM / 32;        // 16-token fragments per wave
    __shared__ __attribute__((aligned(1024))) uint8_t tok0[BM * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t tok1[BM * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t wt0[kBN * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t wt1[kBN * kBK * 2];

    const uint32_t lane = threadIdx.x & (kMmWave - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kMmWave);
    // Block b runs on XCD b mod 8: the token tiles of one weight tile follow
    // each other there, so that its L2 fetches the weights once.
    const uint32_t xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
    const uint32_t split = idx / (p.m_tiles * ((p.n_tiles + 7) / 8));
    const uint32_t rest = idx % (p.m_tiles * ((p.n_tiles + 7) / 8));
    const uint32_t nt = (rest / p.m_tiles) * 8 + xcd;
    if (nt >= p.n_tiles || split >= p.splits) return;
    const uint32_t m0 = (rest % p.m_tiles) * BM;
    constexpr uint32_t kOutN = kEpi == kEpiGated ? kBN / 2 : kBN;  // outputs per token of a tile
    const uint32_t n0 = nt * kOutN;
    const uint32_t kt_lo = (uint32_t)((uint64_t)p.k_tiles * split / p.splits);
    const uint32_t kt_hi = (uint32_t)((uint64_t)p.k_tiles * (split + 1) / p.splits);

    // ---- what this lane loads -------------------------------------------
    // Every buffer resource ends where its rows end: a load past that end
    // puts zeros into LDS. So tokens past the last, weight rows past the
    // last and reduction steps past the last (given an offset past every
    // end) come as zeros, whatever memory holds there. (Columns past the
    // last of a transposed tile may hold the next row's; they are not stored.)
    constexpr uint32_t kPastEnd = 0x80000000u;
    // rows of 64 k: instruction i covers rows 64 i + 8 wave + lane / 8
    const uint32_t lr = 8 * wave + (lane >> 3);
    const uint32_t lc = (lane & 7) ^ ((lr >> 1) & 7);  // 64 i leaves the swizzle unchanged
    const uint16_t *a_base = p.a + (uint64_t)m0 * p.lda;
    const uint32_t a_end = (uint32_t)(((min((uint32_t)BM, p.m - m0) - 1) * p.lda + p.ak) * 2);
    uint32_t a_off[kTokInstr];
#pragma unroll
    for (int i = 0; i < kTokInstr; ++i) a_off[i] = (uint32_t)((64u * i + lr) * p.lda * 2) + 16 * lc;
    uint32_t w_off[4];
    const uint16_t *w_base = nullptr;  // rows contiguous in k: the wave's matrix at row n0
    uint32_t w_end = 0;
    if constexpr (!kNN) {
        // LDS row 64 i + 8 wave + ..: 32 rows of gate (waves 0-3), then 32 of up
        w_base = (wave < 4 ? p.w0 : p.w1) + (uint64_t)n0 * p.ldw;
        w_end = (uint32_t)(((min(kBN / 2, p.n - n0) - 1) * p.ldw + p.wk) * 2);
        const uint32_t r = 8 * (wave & 3) + (lane >> 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) w_off[i] = (uint32_t)((32u * i + r) * p.ldw * 2) + 16 * lc;
    } else {
        // rows of 256 columns: instruction i covers rows 16 i + 2 wave + lane / 32
        const uint32_t wk_row = 2 * wave + (lane >> 5);
        const uint32_t sw = (wk_row & 3) | ((wk_row >> 1) & 4);
        const uint32_t c = ((((lane & 31) >> 1) ^ sw) << 1) | (lane & 1);  // 8-column chunk
#pragma unroll
        for (int i = 0; i < 4; ++i) w_off[i] = (uint32_t)((16u * i + wk_row) * p.ldw * 2) + 16 * c;
    }

    // Request k-tile kt into a buffer.
    auto stage = [&](uint32_t kt, uint8_t *tok, uint8_t *wt) {
        const uint32_t ak0 = kt * kBK;
        uint8_t *tok_w = tok + wave * 1024, *wt_w = wt + wave * 1024;
        const auto ra = buffer(a_base, a_end);
        // steps come in whole chunks of 8
        const uint32_t step = 2 * ak0 + (ak0 + 8 * lc < p.ak ? 0u : kPastEnd);
#pragma unroll
        for (int i = 0; i < kTokInstr; ++i) load_to_lds(ra, a_off[i] + step, tok_w + i * 8192);
        if constexpr (!kNN) {
            const auto rw = buffer(w_base, w_end);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_to_lds(rw, w_off[i] + step, wt_w + i * 8192);
        } else {
            const bool second = kt >= p.k_tiles0;
            const uint32_t k0 = (kt - (second ? p.k_tiles0 : 0u)) * kBK;
            const auto rw = buffer((second ? p.w1 : p.w0) + (uint64_t)k0 * p.ldw + n0,
                                   (uint32_t)(((min(kBK, p.wk - k0) - 1) * p.ldw + (p.n - n0)) * 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) load_to_lds(rw, w_off[i], wt_w + i * 8192);
        }
    };

    // ---- what this lane multiplies ----------------------------------------
    const uint32_t wn = wave & 3, wm = wave >> 2;  // the wave's 64 weight rows and BM / 2 tokens
    const uint32_t fr = lane & 15, fk = lane >> 4;
    f32x4 acc[4][kMT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kMT; ++j) acc[i][j] = f32x4{};
    auto frag = [&](const uint8_t *tile, uint32_t row, uint32_t ks) {
        const uint32_t c = (4 * ks + fk) ^ ((row >> 1) & 7);
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(tile + row * 128 + 16 * c));
    };
    auto frag_t = [&](uint8_t *tile, uint32_t col0, uint32_t ks) {  // 8 k of column col0 + lane % 16
        const uint32_t k = 32 * ks + 8 * fk + (fr >> 2);
        const uint32_t unit = (col0 >> 4) ^ ((k & 3) | ((k >> 1) & 4));
        uint8_t *q = tile + k * 512 + 32 * unit + 8 * (fr & 3);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)q);
        const s16x4 hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(q + 4 * 512));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto compute = [&](uint8_t *tok, uint8_t *wt) {
#pragma unroll
        for (uint32_t ks = 0; ks < kBK / 32; ++ks) {
            bf16x8 w[4], t[kMT];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = kNN ? frag_t(wt, 64 * wn + 16 * i, ks) : frag(wt, 64 * wn + 16 * i + fr, ks);
#pragma unroll
            for (int j = 0; j < kMT; ++j) t[j] = frag(tok, (BM / 2) * wm + 16 * j + fr, ks);
#pragma unroll
            for (int j = 0; j < kMT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], t[j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time: both do not fit the registers
        }
    };
    // Every wave's loads into the buffer to be read have landed, and every
    // wave is done with the other one.
    auto tile_ready = [&] {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
    };

    stage(kt_lo, tok0, wt0);
    for (uint32_t kt = kt_lo; kt + 1 < kt_hi; kt += 2) {
        tile_ready();
        stage(kt + 1, tok1, wt1);
        compute(tok0, wt0);
        tile_ready();
        if (kt + 2 < kt_hi) stage(kt + 2, tok0, wt0);
        compute(tok1, wt1);
    }
    if ((kt_hi - kt_lo) & 1) {
        tile_ready();
        compute(tok0, wt0);
    }

    // ---- outputs: accumulator v of lane l is weight row 16 i + 4 (l / 16) +
    // v and token 16 j + l % 16 ------------------------------------------------
#pragma unroll
    for (int j = 0; j < kMT; ++j) {
        const uint32_t t = m0 + (BM / 2) * wm + 16 * j + fr;
        if (t >= p.m) continue;
        if constexpr (kEpi == kEpiGated) {
            const bool vec = ((p.ldh | p.ldgu) & 3) == 0 &&
                             ((reinterpret_cast<uintptr_t>(p.h) | reinterpret_cast<uintptr_t>(p.g) |
                               reinterpret_cast<uintptr_t>(p.u)) & 7) == 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t f = n0 + 32 * wn + 16 * i + 4 * fk;
                if (f >= p.n) continue;
                const uint32_t n4 = p.n - f;
                float g[4], u[4], h[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    g[v] = acc[i][j][v];
                    u[v] = acc[i + 2][j][v];
                    h[v] = act<kAct>(g[v]) * u[v];
                }
                store4(p.h + (uint64_t)t * p.ldh + f, h, n4, vec);
                if (p.g) {
                    store4(p.g + (uint64_t)t * p.ldgu + f, g, n4, vec);
                    store4(p.u + (uint64_t)t * p.ldgu + f, u, n4, vec);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = n0 + 64 * wn + 16 * i + 4 * fk;
                if (c >= p.n) continue;  // n is a multiple of 8
                if constexpr (kEpi == kEpiBf16) {
                    const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store4(p.h + (uint64_t)t * p.ldh + c, v, 4,
                           (p.ldh & 3) == 0 && (reinterpret_cast<uintptr_t>(p.h) & 7) == 0);
                } else if constexpr (kEpi == kEpiF32) {
                    float *y = p.y32 + (uint64_t)t * p.ldh + c;  // 4-byte aligned
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = p.add ? y[v] + acc[i][j][v] : acc[i][j][v];
                } else {  // partial sums of this range, [splits, m, n]
                    float *y = p.y32 + ((uint64_t)split * p.m + t) * p.n + c;
                    *reinterpret_cast<f32x4 *>(y) = acc[i][j];
                }
            }
        }
    }
}

// The partial sums of every range, added in their order: the same result on
// every run.
template <bool kBf16>
__global__ __launch_bounds__(256) void afx_mm_join_kernel(const float *part, uint32_t splits, uint32_t m, uint32_t n,
                                                          void *out, uint64_t ld, uint32_t add) {
    const uint64_t total = (uint64_t)m * n;
    for (uint64_t i = 4 * ((uint64_t)blockIdx.x * 256 + threadIdx.x); i < total; i += 4ull * 256 * gridDim.x) {
        f32x4 s = *reinterpret_cast<const f32x4 *>(part + i);
        for (uint32_t k = 1; k < splits; ++k) s += *reinterpret_cast<const f32x4 *>(part + k * total + i);
        const uint64_t t = i / n, c = i % n;  // n is a multiple of 8: four outputs of one token
        if constexpr (kBf16) {
            uint16_t *y = static_cast<uint16_t *>(out) + t * ld + c;
            for (int v = 0; v < 4; ++v) y[v] = to_bf16(s[v]);
        } else {
            float *y = static_cast<float *>(out) + t * ld + c;
            for (int v = 0; v < 4; ++v) y[v] = add ? y[v] + s[v] : s[v];
        }
    }
}

uint32_t tokens_per_tile(uint32_t m) { return m <= 64 ? 64 : m <= 128 ? 128 : 256; }

// How many ranges the reduction is cut into: as many as still fit one
// workgroup per CU, each of at least 8 k-tiles.
uint32_t transposed_splits(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    const uint64_t bm = tokens_per_tile(m);
    const uint64_t tiles = ((m + bm - 1) / bm) * ((cols + kBN - 1) / kBN);
    const uint64_t k_tiles = n_mats * (mm_pad_k(rows) / kBK);
    return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(256 / tiles, k_tiles / 8));
}

template <int BM, bool kNN, int kEpi, uint32_t kAct>
int launch(MmArgs &p, hipStream_t stream) {
    const uint32_t out_n = kEpi == kEpiGated ? kBN / 2 : kBN;
    p.m_tiles = (p.m + BM - 1) / BM;
    p.n_tiles = (p.n + out_n - 1) / out_n;
    const uint64_t blocks = (uint64_t)p.m_tiles * ((p.n_tiles + 7) / 8) * 8 * p.splits;
    if (blocks >= (1ull << 31)) return AFX_E_UNSUPPORTED;
    void *args[] = {&p};  // hipLaunchKernel reports this launch's own status
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_mm_kernel<BM, kNN, kEpi, kAct>),
                           dim3((unsigned)blocks), dim3(kMmThreads), args, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

template <bool kNN, int kEpi, uint32_t kAct = 0>
int launch_for_tokens(MmArgs &p, hipStream_t stream) {
    switch (tokens_per_tile(p.m)) {
        case 64: return launch<64, kNN, kEpi, kAct>(p, stream);
        case 128: return launch<128, kNN, kEpi, kAct>(p, stream);
        default: return launch<256, kNN, kEpi, kAct>(p, stream);
    }
}

}  // namespace

int launch_mm_gated(const MmGated &q, hipStream_t stream) {
    MmArgs p{};
    p.a = q.x;
    p.lda = q.ldx;
    p.w0 = q.wg;
    p.w1 = q.wu;
    p.ldw = q.cols;
    p.m = q.m;
    p.n = (uint32_t)q.rows;
    p.ak = p.wk = (uint32_t)q.cols;
    p.k_tiles0 = p.k_tiles = (uint32_t)(mm_pad_k(q.cols) / kBK);
    p.splits = 1;
    p.h = q.h;
    p.ldh = q.ldh;
    p.g = q.g;
    p.u = q.u;
    p.ldgu = q.ldgu;
    switch (q.act) {
        case AFX_ACT_SILU: return launch_for_tokens<false, kEpiGated, AFX_ACT_SILU>(p, stream);
        case AFX_ACT_GELU_TANH: return launch_for_tokens<false, kEpiGated, AFX_ACT_GELU_TANH>(p, stream);
        default: return launch_for_tokens<false, kEpiGated, AFX_ACT_GELU>(p, stream);
    }
}

uint64_t mm_transposed_partial(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    const uint32_t s = transposed_splits(rows, cols, n_mats, m);
    return s > 1 ? (uint64_t)s * m * cols * 4 : 0;
}

int launch_mm_transposed(const MmTransposed &q, hipStream_t stream) {
    MmArgs p{};
    p.a = q.a;
    p.lda = q.lda;
    p.w0 = q.w[0];
    p.w1 = q.w[1];
    p.ldw = q.cols;
    p.m = q.m;
    p.n = (uint32_t)q.cols;
    p.wk = (uint32_t)q.rows;
    p.k_tiles0 = (uint32_t)(mm_pad_k(q.rows) / kBK);
    p.k_tiles = p.k_tiles0 * q.n_mats;
    p.ak = q.n_mats == 2 ? p.k_tiles * kBK : (uint32_t)q.rows;
    p.splits = transposed_splits(q.rows, q.cols, q.n_mats, q.m);
    p.add = q.add;
    p.ldh = q.ldy;
    if (p.splits == 1) {
        p.h = q.y16;
        p.y32 = q.y32;
        return q.y16 ? launch_for_tokens<true, kEpiBf16>(p, stream) : launch_for_tokens<true, kEpiF32>(p, stream);
    }
    p.y32 = q.partial;
    const int rc = launch_for_tokens<true, kEpiPartial>(p, stream);
    if (rc != AFX_OK) return rc;
    const uint64_t quads = (uint64_t)q.m * q.cols / 4;
    const dim3 grid((unsigned)std::min<uint64_t>((quads + 255) / 256, 4096));
    const float *part = q.partial;
    void *out = q.y16 ? static_cast<void *>(q.y16) : static_cast<void *>(q.y32);
    uint32_t splits = p.splits, m = q.m, n = p.n, add = q.add;
    uint64_t ld = q.ldy;
    void *args[] = {&part, &splits, &m, &n, &out, &ld, &add};
    const void *fn = q.y16 ? reinterpret_cast<const void *>(&afx_mm_join_kernel<true>)
                           : reinterpret_cast<const void *>(&afx_mm_join_kernel<false>);
    return hipLaunchKernel(fn, grid, dim3(256), args, 0, stream) == hipSuccess ? AFX_OK : AFX_E_HIP;
}

}  // namespace afx
