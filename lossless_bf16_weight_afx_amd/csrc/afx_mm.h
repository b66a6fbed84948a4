// afx_mm.h -- the product of BF16 activations with restored BF16 weights on
// the matrix cores (afx_mm.hip), as the gated feed-forward block and the
// transposed product use it. Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_panels.h"

namespace afx {

constexpr uint32_t kMmTileK = kPanelCols;  // reduction steps of a k-tile

// h = act(x wg^T) * (x wu^T).
struct MmGated {
    const uint16_t *x;       // panels of BF16 [m, cols]
    uint32_t m;
    const uint16_t *wg, *wu; // panels of BF16 [rows, cols]
    uint64_t rows, cols;
    uint32_t act;
    uint16_t *h;             // BF16 [m, rows], row stride ldh
    uint64_t ldh;
    uint16_t *g, *u;         // BF16 [m, rows], row stride ldgu, or NULL
    uint64_t ldgu;
    float *partial;          // mm_gated_partial(...) bytes
};

// y = a[0] w[0] (+ a[1] w[1]).
struct MmTransposed {
    const uint16_t *a[2];    // BF16 [m, rows], row stride lda, 16-byte aligned rows; rows up to the next
                             // multiple of 8 are read and must be 0
    uint64_t lda;
    uint32_t m;
    const uint16_t *w[2];    // BF16 [rows, cols], restored
    uint32_t n_mats;
    uint64_t rows, cols;
    float *y32;              // FP32 [m, cols], row stride ldy (one of y32, y16)
    uint16_t *y16;           // BF16
    uint64_t ldy;
    bool add;                // y32 += instead of =
    float *partial;          // mm_transposed_partial(...) bytes
};

uint64_t mm_gated_partial(uint64_t rows, uint64_t cols, uint32_t m);
uint64_t mm_transposed_partial(uint64_t rows, uint64_t cols, uint32_t n_mats, uint32_t m);
int launch_mm_gated(const MmGated &p, hipStream_t stream);
int launch_mm_transposed(const MmTransposed &p, hipStream_t stream);

}  // namespace afx
