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
// v_mfma_f32_32x32x16_bf16 and tokens the B operand, so that a lane's four
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
//
// The gated product reads 128 bytes of each of 256 rows, so its operands come
// as panels (afx_panels.h: at 64 tokens and 17408 x 5112 weights 97 us, 142
// from row-major ones); the transposed product reads 512 bytes of each of 64
// weight rows and takes row-major weights (1024 tokens: 353 us, 370 from
// panels) and tokens as they are.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "afx_act.h"
#include "afx_mm.h"

namespace afx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMmWave = 64, kMmWaves = 8, kMmThreads = kMmWave * kMmWaves;
constexpr uint32_t kBN = 256;          // weight rows (or columns) of a tile
constexpr uint32_t kBK = kMmTileK;     // reduction steps of a tile
constexpr int kBufferFlags = 0x00020000;  // raw buffer, 32-bit data format

// How a launch's tiles are laid out. The tiles of n_full weight tiles (whole
// rounds of one workgroup per CU) take the whole reduction; those of the
// n_rest others, which would leave CUs idle in a last round, are cut into
// `splits` ranges of the reduction, whose sums a second launch adds in order.
// A unit is a weight tile, or one range of one of the rest; its token tiles
// follow each other on one XCD, whose L2 then fetches the weights once.
struct MmPlan {
    uint32_t bm, m_tiles, n_full, n_rest, splits;  // bm: tokens of a tile
};

struct MmArgs {
    const uint16_t *a0, *a1;  // gated: a0 tokens' panels; transposed: tokens of each matrix [m, ak], row stride lda
    const uint16_t *w0, *w1;  // gated: panels; transposed: row-major, n columns
    uint64_t lda;
    uint32_t m, n;            // tokens; outputs per token
    uint32_t rows, ak;        // weight rows; transposed: steps held by a row of a0
    uint32_t k_tiles0;        // k-tiles of the first matrix
    uint32_t k_tiles;         // k-tiles of all matrices
    MmPlan plan;
    uint16_t *h, *g, *u;      // BF16 outputs
    float *y32;
    float *partial;           // [n_rest][splits][m_tiles][accumulators of a tile's lanes]
    uint64_t ldh, ldgu;       // ldh: also y32's
    uint32_t add;
};

enum MmEpilogue { kEpiGated, kEpiBf16, kEpiF32 };

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

// The outputs of one 32-token fragment: accumulator v of acc[i] of lane l is
// weight row 32 i + 8 (v / 4) + 4 (l / 32) + v mod 4 of the wave's 64, and
// token t (l mod 32 of the fragment). Here accumulators 4 q .. 4 q + 3 of both.
template <int kEpi, uint32_t kAct>
__device__ inline void write_outputs(const MmArgs &p, uint32_t n0, uint32_t wn, uint32_t half, uint32_t t, uint32_t q,
                                     const f32x4 (&acc)[2]) {
    if (t >= p.m) return;
    if constexpr (kEpi == kEpiGated) {
        const bool vec = ((p.ldh | p.ldgu) & 3) == 0 &&
                         ((reinterpret_cast<uintptr_t>(p.h) | reinterpret_cast<uintptr_t>(p.g) |
                           reinterpret_cast<uintptr_t>(p.u)) & 7) == 0;
        const uint32_t f = n0 + 32 * wn + 8 * q + 4 * half;
        if (f >= p.n) return;
        const uint32_t n4 = p.n - f;
        float g[4], u[4], h[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            g[v] = acc[0][v];
            u[v] = acc[1][v];
            h[v] = act<kAct>(g[v]) * u[v];
        }
        store4(p.h + (uint64_t)t * p.ldh + f, h, n4, vec);
        if (p.g) {
            store4(p.g + (uint64_t)t * p.ldgu + f, g, n4, vec);
            store4(p.u + (uint64_t)t * p.ldgu + f, u, n4, vec);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = n0 + 64 * wn + 32 * i + 8 * q + 4 * half;
            if (c >= p.n) continue;  // n is a multiple of 8
            if constexpr (kEpi == kEpiBf16) {
                const float v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
                store4(p.h + (uint64_t)t * p.ldh + c, v, 4,
                       (p.ldh & 3) == 0 && (reinterpret_cast<uintptr_t>(p.h) & 7) == 0);
            } else {
                float *y = p.y32 + (uint64_t)t * p.ldh + c;
                if (((p.ldh & 3) | (reinterpret_cast<uintptr_t>(p.y32) & 15)) == 0) {
                    f32x4 *y4 = reinterpret_cast<f32x4 *>(y);
                    *y4 = p.add ? *y4 + acc[i] : acc[i];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = p.add ? y[e] + acc[i][e] : acc[i][e];
                }
            }
        }
    }
}

template <int BM, bool kNN, int kEpi, uint32_t kAct>
__global__ __launch_bounds__(kMmThreads, 2) void afx_mm_kernel(const MmArgs p) {
    constexpr int kTokInstr = BM / 64;  // DMA instructions per wave for the token tile
    constexpr int kMT = BM / 64;        // 32-token fragments per wave
    __shared__ __attribute__((aligned(1024))) uint8_t tok0[BM * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t tok1[BM * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t wt0[kBN * kBK * 2];
    __shared__ __attribute__((aligned(1024))) uint8_t wt1[kBN * kBK * 2];

    const uint32_t lane = threadIdx.x & (kMmWave - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kMmWave);
    // Block b runs on XCD b mod 8.
    const uint32_t unit = (blockIdx.x >> 3) / p.plan.m_tiles * 8 + (blockIdx.x & 7);
    const uint32_t mt = (blockIdx.x >> 3) % p.plan.m_tiles, m0 = mt * BM;
    const bool rest = unit >= p.plan.n_full;
    const uint32_t r = unit - p.plan.n_full;  // of the rest: weight tile r / splits, range r mod splits
    if (rest && r >= p.plan.n_rest * p.plan.splits) return;
    const uint32_t nt = rest ? p.plan.n_full + r / p.plan.splits : unit;
    constexpr uint32_t kOutN = kEpi == kEpiGated ? kBN / 2 : kBN;  // outputs per token of a tile
    const uint32_t n0 = nt * kOutN;
    const uint32_t splits = rest ? p.plan.splits : 1, split = rest ? r % p.plan.splits : 0;
    const uint32_t kt_lo = (uint32_t)((uint64_t)p.k_tiles * split / splits);
    const uint32_t kt_hi = (uint32_t)((uint64_t)p.k_tiles * (split + 1) / splits);

    // ---- what this lane loads -------------------------------------------
    // Every buffer resource ends where its rows do: a load past that end puts
    // zeros into LDS. So tokens, weight rows and reduction steps (given an
    // offset past every end) past the last come as zeros, whatever memory
    // holds there. (Columns past the last of a transposed tile are the next
    // row's; their outputs are not stored.)
    constexpr uint32_t kPastEnd = 0x80000000u;
    // Instruction i of a wave covers rows 64 i + 8 wave + lane / 8 of 64 steps.
    const uint32_t lr = 8 * wave + (lane >> 3);
    const uint32_t lc = (lane & 7) ^ ((lr >> 1) & 7);  // 64 i leaves the swizzle unchanged
    const uint32_t a_row = kNN ? (uint32_t)(p.lda * 2) : 128u;  // bytes from row to row
    const uint32_t a_off = a_row * lr + 16 * lc;
    const uint32_t a_end = kNN ? (uint32_t)(((min((uint32_t)BM, p.m - m0) - 1) * p.lda + p.ak) * 2) : (p.m - m0) * 128;
    uint32_t w_off, w_end = 0;
    if constexpr (!kNN) {
        // LDS row 64 i + 8 wave + ..: 32 rows of gate (waves 0-3), then 32 of up
        w_off = 128 * (8 * (wave & 3) + (lane >> 3)) + 16 * lc;
        w_end = (p.n - n0) * 128;
    } else {
        // rows of 256 columns: instruction i covers rows 16 i + 2 wave + lane / 32
        const uint32_t wk_row = 2 * wave + (lane >> 5);
        const uint32_t sw = (wk_row & 3) | ((wk_row >> 1) & 4);
        w_off = wk_row * (2 * p.n) + 32 * (((lane & 31) >> 1) ^ sw) + 16 * (lane & 1);
    }

    // Request k-tile kt into a buffer.
    auto stage = [&](uint32_t kt, uint8_t *tok, uint8_t *wt) {
        const bool second = kNN && kt >= p.k_tiles0;
        const uint32_t kl = kt - (second ? p.k_tiles0 : 0u), k0 = kl * kBK;  // within the matrix
        uint8_t *tok_w = tok + wave * 1024, *wt_w = wt + wave * 1024;
        const auto ra = kNN ? buffer((second ? p.a1 : p.a0) + m0 * p.lda, a_end)
                            : buffer(p.a0 + ((uint64_t)kl * p.m + m0) * kBK, a_end);
        // (transposed: steps come in whole chunks of 8)
        const uint32_t a_step = kNN ? 2 * k0 + (k0 + 8 * lc < p.ak ? 0u : kPastEnd) : 0u;
#pragma unroll
        for (int i = 0; i < kTokInstr; ++i) load_to_lds(ra, a_off + 64 * i * a_row + a_step, tok_w + i * 8192);
        if constexpr (!kNN) {
            const auto rw = buffer((wave < 4 ? p.w0 : p.w1) + ((uint64_t)kl * p.rows + n0) * kBK, w_end);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_to_lds(rw, w_off + i * 4096, wt_w + i * 8192);
        } else {
            const auto rw = buffer((second ? p.w1 : p.w0) + (uint64_t)k0 * p.n + n0,
                                   (uint32_t)(((min(kBK, p.rows - k0) - 1) * (uint64_t)p.n + (p.n - n0)) * 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) load_to_lds(rw, w_off + i * 32 * p.n, wt_w + i * 8192);
        }
    };

    // ---- what this lane multiplies ----------------------------------------
    const uint32_t wn = wave & 3, wm = wave >> 2;  // the wave's 64 weight rows and BM / 2 tokens
    const uint32_t fr = lane & 31, half = lane >> 5;
    f32x16 acc[2][kMT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < kMT; ++j) acc[i][j] = f32x16{};
    // Row row0 + l mod 32, 8 of the tile's steps from 16 ks + 8 (l / 32).
    auto frag = [&](const uint8_t *tile, uint32_t row0, uint32_t ks) {
        const uint32_t row = row0 + fr, c = (2 * ks + half) ^ ((row >> 1) & 7);
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(tile + row * 128 + 16 * c));
    };
    // The same of columns l mod 32 and 32 + l mod 32 of the wave's 64 of a
    // transposed tile. (The four reads and their wait are one block: through
    // the compiler's builtin, every transposing read would wait for all loads
    // into LDS, whichever buffer they fill.)
    auto frags_t = [&](uint8_t *tile, uint32_t ks, bf16x8 (&f)[2]) {
        const uint32_t k = 16 * ks + 8 * half + ((lane & 15) >> 2);
        const uint32_t unit = 4 * wn + ((lane >> 4) & 1), sw = (k & 3) | ((k >> 1) & 4);
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)tile + k * 512 +
                            8 * (lane & 3);
        s16x4 v0, v1, v2, v3;
        asm volatile("ds_read_b64_tr_b16 %0, %4\n\t"
                     "ds_read_b64_tr_b16 %1, %4 offset:2048\n\t"
                     "ds_read_b64_tr_b16 %2, %5\n\t"
                     "ds_read_b64_tr_b16 %3, %5 offset:2048\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3)
                     : "v"(at + 32 * (unit ^ sw)), "v"(at + 32 * ((unit + 2) ^ sw))
                     : "memory");
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        f[0] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
        f[1] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(v2, v3, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    // A k-tile is 4 kMT slots: slot j of step ks (16 of the tile's 64)
    // multiplies token fragment j with the step's two weight fragments. Its
    // fragments were read kLead slots before, so that the matrix cores need
    // not wait for LDS; the last kLead slots read the next tile's first
    // fragments. Before those, the tile is done with its buffers.
    constexpr int kSlots = 4 * kMT, kLead = kMT > 3 ? 3 : kMT, kRing = 4;
    bf16x8 w[2][2], t[kRing];  // weight fragments of two steps; a ring of token fragments
    // What slot n (of this tile, or past kSlots of the next) multiplies.
    auto read = [&](int n, uint8_t *tok, uint8_t *wt) {
        const int ks = n / kMT, j = n % kMT;
        t[n % kRing] = frag(tok, (BM / 2) * wm + 32 * j, ks % 4);
        if (j == 0) {
            if constexpr (kNN) {
                frags_t(wt, ks % 4, w[ks % 2]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) w[ks % 2][i] = frag(wt, 64 * wn + 32 * i, ks % 4);
            }
        }
    };
    // Slot s of the tile in tok, wt; tok_n, wt_n: the next tile's, if there is one.
    auto slot = [&](int s, uint8_t *tok, uint8_t *wt, uint8_t *tok_n, uint8_t *wt_n, auto has_next) {
        const int n = s + kLead;  // the slot whose fragments are read now
        if (n < kSlots)
            read(n, tok, wt);
        else if (has_next)
            read(n, tok_n, wt_n);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            acc[i][s % kMT] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[s / kMT % 2][i], t[s % kRing], acc[i][s % kMT], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto first_slots = [&](uint8_t *tok, uint8_t *wt) {
#pragma unroll
        for (int s = 0; s < kSlots - kLead; ++s) slot(s, tok, wt, tok, wt, std::false_type{});
    };
    // The last slots of k-tile kt and the first of the next.
    auto on_to_next = [&](uint32_t kt, uint8_t *tok, uint8_t *wt, uint8_t *tok_n, uint8_t *wt_n) {
        // This wave holds all it reads of the tile, and its loads of the next
        // one have landed; then every wave's.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __syncthreads();
        if (kt + 2 < kt_hi) stage(kt + 2, tok, wt);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = kSlots - kLead; s < kSlots; ++s) slot(s, tok, wt, tok_n, wt_n, std::true_type{});
        first_slots(tok_n, wt_n);
    };
    auto last_slots = [&](uint8_t *tok, uint8_t *wt) {
#pragma unroll
        for (int s = kSlots - kLead; s < kSlots; ++s) slot(s, tok, wt, tok, wt, std::false_type{});
    };
    stage(kt_lo, tok0, wt0);
    if (kt_lo + 1 < kt_hi) stage(kt_lo + 1, tok1, wt1);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kLead; ++n) read(n, tok0, wt0);
    first_slots(tok0, wt0);
    uint32_t kt = kt_lo;
    for (; kt + 2 < kt_hi; kt += 2) {
        on_to_next(kt, tok0, wt0, tok1, wt1);
        on_to_next(kt + 1, tok1, wt1, tok0, wt0);
    }
    if (kt + 1 < kt_hi) {
        on_to_next(kt, tok0, wt0, tok1, wt1);
        last_slots(tok1, wt1);
    } else {
        last_slots(tok0, wt0);
    }

    // ---- outputs, or a range's sums as they lie in the lanes ------------------
    f32x4 *out = reinterpret_cast<f32x4 *>(p.partial) + ((uint64_t)r * p.plan.m_tiles + mt) * (8 * kMT * kMmThreads);
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            if (splits == 1) {
                write_outputs<kEpi, kAct>(p, n0, wn, half, m0 + (BM / 2) * wm + 32 * j + fr, q, v);
            } else {
                out[(8 * j + 2 * q) * kMmThreads + threadIdx.x] = v[0];
                out[(8 * j + 2 * q + 1) * kMmThreads + threadIdx.x] = v[1];
            }
        }
}

// One 32-token fragment of every wave of one of the rest's tiles (kQ 4), or a
// quarter of it for 2 of the waves (kQ 1): the ranges' sums added in their
// order (the same bits on every run), then the outputs.
constexpr uint32_t join_threads(int q) { return q == 4 ? kMmThreads : kMmThreads / 4; }
constexpr uint32_t join_parts(int q) { return q == 4 ? 1 : 16; }
template <int BM, int kEpi, uint32_t kAct, int kQ>
__global__ __launch_bounds__(join_threads(kQ)) void afx_mm_join_kernel(const MmArgs p) {
    constexpr uint32_t kMT = BM / 64, kParts = join_parts(kQ);
    const uint32_t part = blockIdx.x % kParts, q0 = part % 4, j = blockIdx.x / kParts % kMT;
    const uint32_t mt = blockIdx.x / (kParts * kMT) % p.plan.m_tiles, nr = blockIdx.x / (kParts * kMT) / p.plan.m_tiles;
    const uint32_t thread = part / 4 * join_threads(kQ) + threadIdx.x;  // of the tile's workgroup
    const uint32_t lane = thread & (kMmWave - 1), wave = thread / kMmWave;
    f32x4 acc[kQ][2] = {};
    const uint64_t range = (uint64_t)p.plan.m_tiles * (8 * kMT * kMmThreads);  // from one to the next
    const f32x4 *in = reinterpret_cast<const f32x4 *>(p.partial) + nr * p.plan.splits * range +
                      (uint64_t)mt * (8 * kMT * kMmThreads) + (8 * j + 2 * q0) * kMmThreads + thread;
    constexpr int kAtOnce = 8 / kQ;  // ranges requested together
#pragma unroll kAtOnce
    for (uint32_t s = 0; s < p.plan.splits; ++s)
#pragma unroll
        for (int k = 0; k < 2 * kQ; ++k) acc[k / 2][k % 2] += in[s * range + k * kMmThreads];
    constexpr uint32_t kOutN = kEpi == kEpiGated ? kBN / 2 : kBN;
#pragma unroll
    for (int k = 0; k < kQ; ++k)
        write_outputs<kEpi, kAct>(p, (p.plan.n_full + nr) * kOutN, wave & 3, lane >> 5,
                                  mt * BM + (BM / 2) * (wave >> 2) + 32 * j + (lane & 31), q0 + k, acc[k]);
}

// A CU runs one workgroup of these tiles, 32 CUs share an XCD. (On another
// device the launches do the same work in another number of rounds: the plan,
// and so the workspace and the order of the sums, do not depend on it.)
constexpr uint32_t kXcds = 8, kXcdCus = 32;
constexpr uint32_t kLeastRange = 4;  // k-tiles: a range's start and join take about as long

MmPlan plan_for(uint32_t bm, uint32_t m, uint64_t n, uint32_t out_n, uint64_t k_tiles) {
    MmPlan p{};
    p.bm = bm;
    p.m_tiles = (m + bm - 1) / bm;
    const uint32_t n_tiles = (uint32_t)((n + out_n - 1) / out_n);
    // weight tiles of a round: what every XCD's CUs take at once
    const uint32_t round = kXcds * std::max(1u, kXcdCus / p.m_tiles);
    p.n_full = n_tiles / round * round;
    p.n_rest = n_tiles - p.n_full;
    p.splits = 1;
    if (p.n_rest == 0) return p;
    const uint32_t most = (uint32_t)std::max<uint64_t>(1, k_tiles / kLeastRange);
    while (p.splits < most && (p.n_rest * (p.splits + 1) + kXcds - 1) / kXcds * p.m_tiles <= kXcdCus) ++p.splits;
    return p;
}

// Tokens of a tile: 64, 128 or 256, whichever is estimated to take least. A
// k-tile takes about 1.2, 1.4 and 1.75 us of them (17408 x 5112 weights, as
// many tokens: 97, 110 and 138 us), so that large tiles win where they fill
// the CUs, small ones where large ones would not. The sums of ranges cost
// about 4 us and their bytes' way to memory and back. (Gated, with join:
// 1000 x 600 weights, 200 tokens 11.7 us, 16.9 with the largest tile; 3000 x
// 1000, 600 tokens: 21 and 32; 17408 x 5120, 256 tokens, where the two are
// estimated alike: 141 and 136.)
MmPlan mm_plan(uint32_t m, uint64_t n, uint32_t out_n, uint64_t k_tiles) {
    MmPlan best{};
    double least = 0;
    for (uint32_t bm = 64; bm <= 256; bm *= 2) {
        const MmPlan p = plan_for(bm, m, n, out_n, k_tiles);
        const auto rounds = [&](uint64_t units) { return (double)((units * p.m_tiles + 255) / 256); };
        double tiles = rounds(p.n_full) * (double)k_tiles, us = 0;
        if (p.n_rest) tiles += rounds((uint64_t)p.n_rest * p.splits) * (double)((k_tiles + p.splits - 1) / p.splits);
        if (p.splits > 1) us += 4 + (double)p.n_rest * p.splits * p.m_tiles * bm * kBN * 8 / 4.9e6;
        us += tiles * (bm == 64 ? 1.2 : bm == 128 ? 1.4 : 1.75);
        if (bm == 64 || us < least) {
            best = p;
            least = us;
        }
        if (m <= bm) break;  // a larger tile would be part empty
    }
    return best;
}

uint64_t partial_bytes(const MmPlan &p) {
    return p.splits > 1 ? (uint64_t)p.n_rest * p.splits * p.m_tiles * p.bm * kBN * 4 : 0;
}

template <int BM, bool kNN, int kEpi, uint32_t kAct>
int launch(MmArgs &p, hipStream_t stream) {
    const MmPlan &q = p.plan;
    const uint64_t units = (uint64_t)q.n_full + q.n_rest * q.splits;
    const uint64_t blocks = (units + kXcds - 1) / kXcds * kXcds * q.m_tiles;
    if (blocks >= (1ull << 31)) return AFX_E_UNSUPPORTED;
    void *args[] = {&p};  // hipLaunchKernel reports this launch's own status
    if (hipLaunchKernel(reinterpret_cast<const void *>(&afx_mm_kernel<BM, kNN, kEpi, kAct>), dim3((unsigned)blocks),
                        dim3(kMmThreads), args, 0, stream) != hipSuccess)
        return AFX_E_HIP;
    if (q.splits == 1) return AFX_OK;
    // Whole fragments write whole lines (64 tiles of 256 tokens, gated: 16 us,
    // 23 in quarters); few of them leave CUs idle and are divided (6 tiles of
    // 64 tokens, 32 ranges: 13.8 us, 4.6 divided).
    const uint32_t frags = q.n_rest * q.m_tiles * (BM / 64);
    const bool whole = frags >= 256;
    const void *join = whole ? reinterpret_cast<const void *>(&afx_mm_join_kernel<BM, kEpi, kAct, 4>)
                             : reinterpret_cast<const void *>(&afx_mm_join_kernel<BM, kEpi, kAct, 1>);
    return hipLaunchKernel(join, dim3(frags * join_parts(whole ? 4 : 1)), dim3(join_threads(whole ? 4 : 1)), args, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

template <bool kNN, int kEpi, uint32_t kAct = 0>
int launch_for_tokens(MmArgs &p, hipStream_t stream) {
    switch (p.plan.bm) {
        case 64: return launch<64, kNN, kEpi, kAct>(p, stream);
        case 128: return launch<128, kNN, kEpi, kAct>(p, stream);
        default: return launch<256, kNN, kEpi, kAct>(p, stream);
    }
}

MmPlan gated_plan(uint64_t rows, uint64_t cols, uint32_t m) { return mm_plan(m, rows, kBN / 2, panel_count(cols)); }
MmPlan transposed_plan(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    return mm_plan(m, cols, kBN, n_mats * panel_count(rows));
}

}  // namespace

uint64_t mm_gated_partial(uint64_t rows, uint64_t cols, uint32_t m) {
    return partial_bytes(gated_plan(rows, cols, m));
}
uint64_t mm_transposed_partial(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m) {
    return partial_bytes(transposed_plan(rows, cols, n_mats, m));
}

int launch_mm_gated(const MmGated &q, hipStream_t stream) {
    MmArgs p{};
    p.a0 = q.x;
    p.w0 = q.wg;
    p.w1 = q.wu;
    p.m = q.m;
    p.n = p.rows = (uint32_t)q.rows;
    p.k_tiles0 = p.k_tiles = (uint32_t)panel_count(q.cols);
    p.plan = gated_plan(q.rows, q.cols, q.m);
    p.partial = q.partial;
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

int launch_mm_transposed(const MmTransposed &q, hipStream_t stream) {
    MmArgs p{};
    p.a0 = q.a[0];
    p.a1 = q.a[1];
    p.w0 = q.w[0];
    p.w1 = q.w[1];
    p.m = q.m;
    p.n = (uint32_t)q.cols;
    p.rows = (uint32_t)q.rows;
    p.lda = q.lda;
    p.ak = (uint32_t)((q.rows + 7) / 8 * 8);
    p.k_tiles0 = (uint32_t)panel_count(q.rows);
    p.k_tiles = p.k_tiles0 * q.n_mats;
    p.plan = transposed_plan(q.rows, q.cols, q.n_mats, q.m);
    p.partial = q.partial;
    p.add = q.add;
    p.h = q.y16;
    p.y32 = q.y32;
    p.ldh = q.ldy;
    return q.y16 ? launch_for_tokens<true, kEpiBf16>(p, stream) : launch_for_tokens<true, kEpiF32>(p, stream);
}

}  // namespace afx
