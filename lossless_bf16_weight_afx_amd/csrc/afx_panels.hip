// afx_panels.hip -- coded matrices restored into panels of 64 columns
// (afx_panels.h), and activations copied into them, for the matrix-core
// products (gfx950).
#include <hip/hip_runtime.h>

#include "afx_device.h"
#include "afx_panels.h"

namespace afx {
namespace {

// Restored values go to panels. T.reserved holds the matrix's columns, a
// multiple of 8, so that 8 values from a multiple of 8 on are in one row and
// panel.
struct OutPlace {
    uint16_t *out;
    uint64_t rows, row0;
    uint32_t cols, c0;  // the chunk starts at row0, column c0
    __device__ OutPlace(const TensorDesc &T, uint64_t e0)
        : out(T.out), rows(T.n / T.reserved), row0(e0 / T.reserved), cols(T.reserved),
          c0((uint32_t)(e0 - row0 * T.reserved)) {}
    __device__ uint16_t *at(uint32_t i) const {
        uint32_t c = c0 + i, d;
        if (cols >= kChunk) {  // (uniform) the chunk reaches into one more row at most
            d = c >= cols ? 1u : 0u;
            c -= d ? cols : 0u;
        } else {
            d = c / cols;
            c -= d * cols;
        }
        return out + ((c / kPanelCols) * rows + row0 + d) * kPanelCols + c % kPanelCols;
    }
};

}  // namespace
}  // namespace afx

#include "afx_restore_body.h"

namespace afx {
namespace {

// Zeros in the last panel's columns past the matrix's.
__global__ __launch_bounds__(256) void afx_panel_pad_kernel(uint16_t *panel, uint64_t rows, uint32_t used) {
    const uint64_t r = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (r >= rows) return;
    for (uint32_t c = used; c < kPanelCols; c += 8)
        *reinterpret_cast<uint4 *>(panel + r * kPanelCols + c) = make_uint4(0, 0, 0, 0);
}

// 8 values per thread; a wave reads 1 KB of a row and writes 8 panels' 128
// bytes of it.
__global__ __launch_bounds__(256) void afx_pack_panels_kernel(const uint16_t *a, uint64_t ld, uint32_t m, uint64_t cols,
                                                              uint64_t padded, uint16_t *out) {
    const uint64_t c = 8 * ((uint64_t)blockIdx.x * 256 + threadIdx.x);
    if (c >= padded) return;
    for (uint64_t t = blockIdx.y; t < m; t += gridDim.y) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < cols) v = *reinterpret_cast<const uint4 *>(a + t * ld + c);
        *reinterpret_cast<uint4 *>(out + ((c / kPanelCols) * m + t) * kPanelCols + c % kPanelCols) = v;
    }
}

bool launch(const void *fn, dim3 grid, uint32_t threads, void **args, hipStream_t stream) {
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, stream) == hipSuccess;
}

}  // namespace

int launch_restore_panels(const PanelJob *jobs, uint32_t n, hipStream_t stream) {
    Batch batch;
    batch.n_tensors = n;
    uint64_t chunks[2];
    uint32_t lo[2], hi[2];
    for (uint32_t t = 0; t < n; ++t) {
        batch.t[t] = describe(afx_job{jobs[t].info, jobs[t].blob_dev, jobs[t].out, 0});
        batch.t[t].reserved = (uint32_t)jobs[t].cols;
        chunks[t] = jobs[t].info->n_chunks;
    }
    int max_blocks = 0;
    const int rc = max_blocks_for_current_device(&max_blocks);
    if (rc != AFX_OK) return rc;
    const uint32_t grid = split_grid(chunks, n, n, (uint32_t)max_blocks, lo, hi);
    for (uint32_t t = 0; t < n; ++t) {
        batch.t[t].blk_lo = lo[t];
        batch.t[t].blk_hi = hi[t];
    }
    void *args[] = {&batch};
    if (!launch(reinterpret_cast<const void *>(&afx_decode_kernel), dim3(grid), kThreads, args, stream)) return AFX_E_HIP;
    for (uint32_t t = 0; t < n; ++t) {
        uint32_t used = (uint32_t)(jobs[t].cols % kPanelCols);
        if (!used) continue;
        uint64_t rows = jobs[t].rows;
        uint16_t *panel = jobs[t].out + jobs[t].cols / kPanelCols * rows * kPanelCols;
        void *pad_args[] = {&panel, &rows, &used};
        if (!launch(reinterpret_cast<const void *>(&afx_panel_pad_kernel), dim3((unsigned)((rows + 255) / 256)), 256,
                    pad_args, stream))
            return AFX_E_HIP;
    }
    return AFX_OK;
}

int launch_pack_panels(const uint16_t *a, uint64_t ld, uint32_t m, uint64_t cols, uint16_t *out, hipStream_t stream) {
    uint64_t padded = panel_count(cols) * kPanelCols;
    void *args[] = {&a, &ld, &m, &cols, &padded, &out};
    return launch(reinterpret_cast<const void *>(&afx_pack_panels_kernel),
                  dim3((unsigned)((padded / 8 + 255) / 256), std::min(m, 32768u)), 256, args, stream)
               ? AFX_OK
               : AFX_E_HIP;
}

}  // namespace afx
