// afx_panels.h -- matrices as panels of 64 columns: element (r, c) of [rows,
// cols] is at panel c / 64, row r, place c mod 64, each panel [rows][64]; the
// columns past the last are zeros. Not installed.
//
// The matrix-core products read a tile as 128 bytes of each of many rows. In
// a row-major matrix those rows are a power of two or so apart (10240 bytes
// for 5120 columns) and fall into 2 of an L2's 16 channels; in a panel they
// follow each other.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_internal.h"

namespace afx {

constexpr uint32_t kPanelCols = 64;
constexpr uint64_t panel_count(uint64_t cols) { return (cols + kPanelCols - 1) / kPanelCols; }
constexpr uint64_t panel_bytes(uint64_t rows, uint64_t cols) { return panel_count(cols) * rows * kPanelCols * 2; }

// A coded matrix to restore. rows < 2^21, cols < 2^22 and a multiple of 8.
struct PanelJob {
    const afx_info *info;
    const void *blob_dev;
    uint64_t rows, cols;
    uint16_t *out;  // panel_bytes(rows, cols)
};

// Restores both matrices (of the same size) and copies the rows of a [m,
// cols] (BF16, row stride ld, a multiple of 8; 16-byte aligned) to panels.
int launch_panels(const PanelJob (&jobs)[2], const uint16_t *a, uint64_t ld, uint32_t m, uint16_t *out,
                  hipStream_t stream);

}  // namespace afx
