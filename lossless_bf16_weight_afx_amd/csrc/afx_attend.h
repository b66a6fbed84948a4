// afx_attend.h -- what the kernels of the attention over a paged cache share.
//
// Query rows. A token's query heads that read one key-value head are rows of
// one matrix: row rr of a batch row's key-value head kvh is token rr / group,
// query head kvh * group + rr % group. All rows of a head share its keys and
// values, so that a cached value is read once for all of them.
//
// Scores are in powers of two: s2 = (q k) scale2, weights 2^(s2 - M), with
// scale2 = |scale| log2(e); the scale's sign goes to q (a scale of 0 makes q 0
// and scale2 1), so that the largest product is the largest score and minus
// infinity stays what it is.
//
// Infinite and NaN values. In a tile of tokens that all rows see, the matrix
// cores bring them to all rows. In one that some rows do not see, 0 times them
// would be NaN: they are multiplied as 0, and added after the last tile to the
// outputs of the rows that see them (as they are: a weight would not make them
// finite). The other rows' sums are those of any finite value in their place,
// bit for bit.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_paged.h"

namespace afx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kFewTokens = 32;    // tokens of a wave's tile in the kernel for few query rows
// Waves of 32 query rows of a workgroup in the kernel for many, by a head's
// dimensions in units of 32: two on a SIMD while their registers allow it.
constexpr uint32_t many_waves(int kc) { return kc <= 4 ? 8 : 4; }
constexpr uint32_t kMaxSplits = 256;   // parts that a row's tokens are cut into
// Tokens that a sequence may have: positions are int32, and both kernels look
// up pages, and count, up to 512 positions behind a sequence's last.
constexpr uint64_t kMaxPositions = (1ull << 31) - 1024;

struct AttendArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    const int32_t *table, *len, *seqs, *starts;
    uint64_t q_stride, out_stride, table_stride;
    uint32_t m, n_rows, n_seqs, max_pages, n_pages, page_shift, q_heads, kv_heads, group, d, causal, window;
    float scale2;
    uint32_t q_and, q_xor;  // what makes q of two of its values
    // Batch rows of at most few_rows query rows a head go to the kernel for few
    // rows: their tokens are cut into parts of few_part tokens (more where that
    // makes more than few_splits). The others' tiles are cut into many_splits
    // equal parts.
    uint32_t few_rows, few_part, few_splits, many_tiles, many_splits;
    // Sums of parts: few: [n_rows][kv_heads][few_rows][few_splits], many: [m][q_heads][many_splits], of d unnormalised
    // outputs, and M and the sum of weights.
    float *few_o, *many_o;
    float2 *few_ml, *many_ml;
};

// A batch row's sequence, its new tokens and its length.
struct BatchRow {
    uint32_t seq, from, n, len;
    __device__ BatchRow() {}
    __device__ BatchRow(const AttendArgs &a, uint32_t r) {
        seq = a.seqs ? (uint32_t)a.seqs[r] : r;
        from = (uint32_t)min(max(a.starts[r], 0), (int32_t)a.m);
        const uint32_t to = (uint32_t)min(max(a.starts[r + 1], 0), (int32_t)a.m);
        n = to > from ? to - from : 0;
        len = seq < a.n_seqs ? (uint32_t)min((int64_t)max(a.len[seq], 0), (int64_t)a.max_pages << a.page_shift) : 0;
    }
    // The positions that new token i sees: begin .. end - 1.
    __device__ int32_t begin(const AttendArgs &a, uint32_t i) const {
        const int64_t at = (int64_t)len - n + i;
        return a.window ? (int32_t)min(max(at - (int64_t)a.window + 1, (int64_t)0), (int64_t)len) : 0;
    }
    __device__ int32_t end(const AttendArgs &a, uint32_t i) const {
        const int64_t at = (int64_t)len - n + i;
        return a.causal ? (int32_t)max(at + 1, (int64_t)0) : (int32_t)len;
    }
};

// The positions seen by a batch row that the kernel for few rows takes, from
// a multiple of its tile on, and their parts.
struct FewRange {
    int32_t base, end;
    uint32_t part, splits;  // tokens of a part (of the last one: the rest), number of parts
    __device__ FewRange(const AttendArgs &a, const BatchRow &row) {
        base = row.begin(a, 0) & ~(int32_t)(kFewTokens - 1);
        end = max(row.end(a, row.n - 1), base);
        const uint32_t n = (uint32_t)(end - base);
        part = a.few_part;
        // (a row longer than was told is cut into as many parts as there is room for, all alike)
        if (a.few_splits > 1 && n > a.few_splits * a.few_part + kFewTokens)
            part = ((n + a.few_splits - 1) / a.few_splits + 127) & ~127u;
        // (more rows than there is room for come out of one part)
        splits = row.n * a.group <= a.few_rows ? min(max((n + part - 1) / part, 1u), a.few_splits) : 1;
    }
};

// 8 dimensions from `dim` on of a query row.
__device__ inline bf16x8 load_q(const AttendArgs &a, const uint16_t *q, uint32_t dim) {
    u32x4 f = *reinterpret_cast<const u32x4 *>(q + min(dim, a.d - 8));
    f = (f & a.q_and) ^ a.q_xor;
    if (dim >= a.d) f = u32x4{0, 0, 0, 0};
    return __builtin_bit_cast(bf16x8, f);
}

// The same value, of which the compiler knows nothing: what a rare path
// computes from it is computed there, and holds no registers around it.
__device__ inline uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ inline uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ inline float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline uint32_t pack2(float lo, float hi) { return to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16); }
__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// Two BF16 values with infinities and NaN as zeros, and whether a value is one.
__device__ inline uint32_t finite2(uint32_t v) {
    const uint32_t odd = ((v & 0x7F807F80u) + 0x00800080u) >> 15 & 0x00010001u;  // (only all ones carry into bit 15)
    return v & ~(odd * 0xFFFFu);
}
__device__ inline bool odd(uint16_t v) { return (v & 0x7F80u) == 0x7F80u; }
// ln of the sum of e^score, from M and the sum of weights
__device__ inline float lse_of(float top, float sum) {
    return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

int launch_attend_few(const AttendArgs &a, hipStream_t stream);
int launch_attend_many(const AttendArgs &a, hipStream_t stream);

}  // namespace afx
