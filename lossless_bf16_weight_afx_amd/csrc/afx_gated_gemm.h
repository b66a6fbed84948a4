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

// Three workgroups on each of 256 CUs run at once. (On a device with fewer
// CUs the rest follow; the split, and so the workspace and the order of the
// sums, do not depend on the device.)
inline GatedSplit gated_split(uint64_t rows, uint64_t cols) { return split_slabs(rows, cols, 3 * 256); }

// cols: a multiple of 32 (a row of whole groups).
uint64_t gated_gemm_space(uint64_t rows, uint64_t cols, uint32_t m);
int launch_gated_gemm(const afx_gated &w, const GatedGemm &q, uint8_t *ws, hipStream_t stream);

}  // namespace afx
