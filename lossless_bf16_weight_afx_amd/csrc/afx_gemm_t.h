// afx_gemm_t.h -- products with coded matrices along their rows, for few
// tokens (afx_gemm_t.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_internal.h"

namespace afx {

// Tokens taken, where rows are whole groups of the coded format and where not.
constexpr uint32_t kGemmTTokens = 64, kGemmTTokensSplit = 16;

// y (+)= d[0] W[0] [+ d[1] W[1]].
struct GemmT {
    const afx_info *info[2];
    const void *blob[2];
    uint32_t n_mats;
    uint64_t rows, cols;   // cols: a multiple of 8
    const uint16_t *d[2];  // BF16 [m, rows], row stride lda, 16-byte aligned rows; rows up to the next
                           // multiple of 8 are read and must be 0
    uint64_t lda;
    uint32_t m;            // 1..kGemmTTokens or kGemmTTokensSplit
    float *y32;            // FP32 [m, cols], row stride ldy, overwritten or (add) added to;
    uint16_t *y16;         // or BF16
    uint64_t ldy;
    bool add;
};

uint64_t gemm_t_space(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m);
int launch_gemm_t(const GemmT &q, uint8_t *ws, hipStream_t stream);

}  // namespace afx
