// afx_gated_gemm.h -- the gated block for up to 128 tokens
// (afx_gated_gemm.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_gated_split.h"
#include "afx_internal.h"

namespace afx {

constexpr uint32_t kGatedGemmTokens = 128;

struct GatedGemm {
    const uint16_t *x;   // BF16 [m, cols], row stride ldx
    uint64_t ldx;
    uint32_t m;          // 1..kGatedGemmTokens
    uint16_t *h, *g, *u; // BF16 [m, rows], row strides ldh, ldgu; g, u may be NULL
    uint64_t ldh, ldgu;
};

// Token blocks of 16 that a call for m tokens computes (a kernel each for 1 to
// 4, 6 and 8).
constexpr uint32_t kGatedTokenBlock = 16;
constexpr uint32_t gated_token_blocks(uint32_t m) {
    const uint32_t b = (m + kGatedTokenBlock - 1) / kGatedTokenBlock;
    return b <= 4 ? b : (b + 1) / 2 * 2;
}

// Waves of a workgroup. One workgroup of each matrix on each of 128 CUs: both
// matrices fill 256. (On a device with fewer CUs the rest follow; the split,
// and so the workspace and the order of the sums, do not depend on the
// device.)
constexpr uint32_t gated_waves(uint32_t blocks) { return blocks <= 4 ? 16 : 8; }
inline GatedSplit gated_split(uint64_t rows, uint64_t cols, uint32_t m) {
    return split_slabs(rows, cols, 128, gated_waves(gated_token_blocks(m)));
}

// cols: a multiple of 32 (a row of whole groups).
uint64_t gated_gemm_space(uint64_t rows, uint64_t cols, uint32_t m);
int launch_gated_gemm(const afx_gated &w, const GatedGemm &q, uint8_t *ws, hipStream_t stream);

}  // namespace afx
