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

struct PackArgs {
    const uint16_t *a;  // [m, cols], row stride ld
    uint64_t ld, cols, padded;
    uint16_t *out;
    uint16_t *w[2];     // panels of two coded matrices [rows, cols]
    uint64_t rows;
    uint32_t m;
};

// Activations to panels, 8 values per thread: a wave reads 1 KB of a row and
// writes 8 panels' 128 bytes of it. And zeros in the last panel's columns of
// both matrices past theirs (the restore writes only theirs).
__global__ __launch_bounds__(256) void afx_pack_panels_kernel(const PackArgs p) {
    const uint64_t c = 8 * ((uint64_t)blockIdx.x * 256 + threadIdx.x);
    if (c < p.padded)
        for (uint64_t t = blockIdx.y; t < p.m; t += gridDim.y) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (c < p.cols) v = *reinterpret_cast<const uint4 *>(p.a + t * p.ld + c);
            *reinterpret_cast<uint4 *>(p.out + ((c / kPanelCols) * p.m + t) * kPanelCols + c % kPanelCols) = v;
        }
    if (p.cols == p.padded) return;
    const uint64_t last = p.cols / kPanelCols * p.rows * kPanelCols, threads = (uint64_t)gridDim.x * gridDim.y * 256;
    for (uint64_t r = ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; r < 2 * p.rows; r += threads) {
        uint16_t *row = (r < p.rows ? p.w[0] : p.w[1]) + last + (r < p.rows ? r : r - p.rows) * kPanelCols;
        for (uint32_t k = p.cols % kPanelCols; k < kPanelCols; k += 8)
            *reinterpret_cast<uint4 *>(row + k) = make_uint4(0, 0, 0, 0);
    }
}

bool launch(const void *fn, dim3 grid, uint32_t threads, void **args, hipStream_t stream) {
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, stream) == hipSuccess;
}

}  // namespace

int launch_panels(const PanelJob (&jobs)[2], const uint16_t *a, uint64_t ld, uint32_t m, uint16_t *out,
                  hipStream_t stream) {
    constexpr uint32_t n = 2;
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
    PackArgs p{};
    p.a = a;
    p.ld = ld;
    p.cols = jobs[0].cols;
    p.padded = panel_count(p.cols) * kPanelCols;
    p.out = out;
    p.w[0] = jobs[0].out;
    p.w[1] = jobs[1].out;
    p.rows = jobs[0].rows;
    p.m = m;
    void *pack_args[] = {&p};
    return launch(reinterpret_cast<const void *>(&afx_pack_panels_kernel),
                  dim3((unsigned)((p.padded / 8 + 255) / 256), std::min(m, 32768u)), 256, pack_args, stream)
               ? AFX_OK
               : AFX_E_HIP;
}

}  // namespace afx
