// afx_gemv.hip -- the restore fused into its consumer (gfx950): y += W x for a
// weight matrix W held only in its coded form.
//
// "Why Weight Offloading Slows Inference" (section "Lossless compression")
// reconstructs a coded weight's bits ahead of the computation that uses it.
// Restoring into HBM and then multiplying writes the BF16 matrix (2 bytes per
// value) and reads it back; for the matrix-vector products of token-by-token
// generation, which read every weight once per token, that traffic is the
// cost. Here each wave restores a chunk exactly as afx_decode.hip does, up to
// the exponent bytes in LDS, and multiplies the restored values by the
// activations in registers: HBM sees the coded matrix (~1.39 bytes per value)
// and nothing else.
//
// W is row-major [rows, cols] (the blob's element order), x is BF16 [m, cols]
// and y is FP32 [m, rows], both row-major; m is 1, 2 or 4 (a handful of
// tokens). The products of two BF16 values are exact in FP32; sums are FP32:
// per lane over 8 consecutive values, two products at a time
// (v_dot2_f32_bf16, which on this hardware measures within one rounding per
// addition), then across the wave, then into y with atomic adds (in no fixed
// order).
//
// Work decomposition and decode as in the restore: one 16-wave workgroup per
// CU, chunks round the workgroups, claimed one at a time by the waves from an
// LDS counter, code words staged a chunk ahead, decoded through the pair
// table.
#include <hip/hip_runtime.h>

#include "afx_gemv_body.h"

namespace afx {
namespace {

// y += the chunk's sums, with atomic adds (in no fixed order).
template <int M>
__device__ inline void GemvSink::put(const GemvArgs &a, uint64_t, uint64_t row0, uint32_t d, int m, float s) {
    atomicAdd(a.y + (uint64_t)m * a.rows + row0 + d, s);
}

template <int M>
int launch_gemv(GemvBatch &batch, hipStream_t stream) {
    bool all_long = true;
    for (uint32_t t = 0; t < batch.n; ++t) all_long &= batch.j[t].cols >= kChunk;
    return all_long ? launch_gemv_kernel<M, true>(batch, stream) : launch_gemv_kernel<M, false>(batch, stream);
}

int check_gemv_job(const afx_gemv_job &j, uint32_t m) {
    int rc = check_info(j.info);
    if (rc != AFX_OK) return rc;
    const afx_info *info = j.info;
    if (j.cols == 0 || info->n_elems % j.cols || info->n_elems / j.cols != j.rows) return AFX_E_INVALID_ARG;
    if (info->n_elems == 0) return AFX_OK;  // nothing to add
    if (!j.blob_dev) return AFX_E_INVALID_ARG;
    if (j.cols % 8 || j.cols >= (1ull << 31)) return AFX_E_UNSUPPORTED;  // x rows are read by byte offset
    if (m != 1 && m != 2 && m != 4) return AFX_E_UNSUPPORTED;
    if (!j.x_dev || !j.y_dev) return AFX_E_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(j.blob_dev) | reinterpret_cast<uintptr_t>(j.x_dev)) & 15) return AFX_E_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(j.y_dev) & 3) return AFX_E_MISALIGNED;
    return AFX_OK;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" int afx_restore_gemv_batch_async(const afx_gemv_job *jobs, size_t n_jobs, uint32_t m, void *stream) {
    if (!jobs && n_jobs) return AFX_E_INVALID_ARG;
    for (size_t i = 0; i < n_jobs; ++i) {
        const int rc = check_gemv_job(jobs[i], m);
        if (rc != AFX_OK) return rc;
    }
    if (fused_outputs_overlap_inputs(jobs, n_jobs, m)) return AFX_E_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    for (size_t i = 0; i < n_jobs;) {
        GemvBatch batch;
        batch.n = 0;
        for (; i < n_jobs && batch.n < kMaxGemvJobs; ++i)
            if (jobs[i].info->n_elems) batch.j[batch.n++] = gemv_args(jobs[i]);
        int rc = AFX_OK;
        switch (m) {
            case 1: rc = launch_gemv<1>(batch, s); break;
            case 2: rc = launch_gemv<2>(batch, s); break;
            default: rc = launch_gemv<4>(batch, s); break;
        }
        if (rc != AFX_OK) return rc;
    }
    return AFX_OK;
}

extern "C" int afx_restore_gemv_async(const afx_info *info, const void *blob_dev, uint64_t rows, uint64_t cols,
                                      const uint16_t *x_dev, uint32_t m, float *y_dev, void *stream) {
    const afx_gemv_job job{info, blob_dev, rows, cols, x_dev, y_dev};
    return afx_restore_gemv_batch_async(&job, 1, m, stream);
}
