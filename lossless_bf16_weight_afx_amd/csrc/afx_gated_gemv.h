// afx_gated_gemv.h -- the gated block for one to four tokens
// (afx_gated_gemv.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_internal.h"

namespace afx {

constexpr uint32_t kGatedGemvTokens = 4;

struct GatedGemv {
    const uint16_t *x;   // BF16 [m, cols], row stride ldx
    uint64_t ldx;
    uint32_t m;          // 1..kGatedGemvTokens
    uint16_t *h, *g, *u; // BF16 [m, rows], row strides ldh, ldgu; g, u may be NULL
    uint64_t ldh, ldgu;
};

uint64_t gated_gemv_space(uint64_t rows, uint64_t cols, uint32_t m);
int launch_gated_gemv(const afx_gated &w, const GatedGemv &q, uint8_t *ws, hipStream_t stream);

}  // namespace afx
