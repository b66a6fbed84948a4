// afx_gated_gemv.hip -- the gated block for one to four tokens (gfx950): both
// projections restored and multiplied by the matrix-vector kernel, then the
// activation and the product.
//
// Token-by-token generation reads every weight once per token, so the coded
// bytes and their decoding bound it; no restored weight reaches memory. The
// two projections are one launch over both matrices, split by chunks as the
// restore is. A chunk's sums per row go to their own place in the workspace
// (at most 2 rows a chunk for rows of 4096 columns or more: 0.7 MB for the
// two 17408 x 5120 matrices) instead of into an atomic add, and a second,
// small launch adds each row's sums in the order of its chunks and forms h:
// the same bits on every run.
#include "afx_gemv_body.h"

#include "afx_act.h"
#include "afx_gated_gemv.h"

namespace afx {
namespace {

// Rows that a chunk's 4096 values can touch, for rows of cols values.
constexpr uint64_t chunk_rows(uint64_t cols) { return (kChunk - 1) / cols + 2; }

// a.y: [chunks][chunk_rows][M]; a.rows holds chunk_rows here.
template <int M>
__device__ inline void GemvSink::put(const GemvArgs &a, uint64_t lc, uint64_t, uint32_t d, int m, float s) {
    a.y[(lc * a.rows + d) * M + m] = s;
}

struct JoinArgs {
    const float *gate, *up;  // as written by GemvSink
    uint16_t *h, *g, *u;
    uint64_t ldh, ldgu, rows;
    uint32_t cols, chunk_rows;
};

template <int M>
__device__ inline void row_sums(const float *part, uint64_t row, const JoinArgs &p, float (&s)[M]) {
    const uint64_t e0 = row * p.cols, e1 = e0 + p.cols - 1;
#pragma unroll
    for (int m = 0; m < M; ++m) s[m] = 0.f;
    for (uint64_t c = e0 / kChunk; c <= e1 / kChunk; ++c) {
        const uint64_t d = row - c * kChunk / p.cols;
        const float *v = part + (c * p.chunk_rows + d) * M;
#pragma unroll
        for (int m = 0; m < M; ++m) s[m] += v[m];
    }
}

template <int M, uint32_t kAct>
__global__ __launch_bounds__(64) void afx_gated_join_kernel(const JoinArgs p) {
    const uint64_t row = (uint64_t)blockIdx.x * 64 + threadIdx.x;
    if (row >= p.rows) return;
    float g[M], u[M];
    row_sums<M>(p.gate, row, p, g);
    row_sums<M>(p.up, row, p, u);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        p.h[m * p.ldh + row] = __builtin_bit_cast(uint16_t, (__bf16)(act<kAct>(g[m]) * u[m]));
        if (p.g) {
            p.g[m * p.ldgu + row] = __builtin_bit_cast(uint16_t, (__bf16)g[m]);
            p.u[m * p.ldgu + row] = __builtin_bit_cast(uint16_t, (__bf16)u[m]);
        }
    }
}

// Token rows moved next to each other (the matrix-vector kernel reads
// contiguous ones), 8 values per thread.
__global__ __launch_bounds__(256) void afx_pack_rows_kernel(const uint16_t *x, uint64_t stride, uint64_t cols,
                                                            uint16_t *out) {
    const uint64_t c = 8 * ((uint64_t)blockIdx.x * 256 + threadIdx.x);
    if (c >= cols) return;
    *reinterpret_cast<uint4 *>(out + blockIdx.y * cols + c) =
        *reinterpret_cast<const uint4 *>(x + blockIdx.y * stride + c);
}

template <int M, uint32_t kAct>
int launch_join(JoinArgs &a, hipStream_t stream) {
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_gated_join_kernel<M, kAct>),
                           dim3((unsigned)((a.rows + 63) / 64)), dim3(64), args, 0, stream) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

template <int M>
int launch_tokens(GemvBatch &batch, JoinArgs &a, uint32_t act, bool all_long, hipStream_t stream) {
    const int rc = all_long ? launch_gemv_kernel<M, true>(batch, stream) : launch_gemv_kernel<M, false>(batch, stream);
    if (rc != AFX_OK) return rc;
    switch (act) {
        case AFX_ACT_SILU: return launch_join<M, AFX_ACT_SILU>(a, stream);
        case AFX_ACT_GELU_TANH: return launch_join<M, AFX_ACT_GELU_TANH>(a, stream);
        default: return launch_join<M, AFX_ACT_GELU>(a, stream);
    }
}

uint64_t align_up(uint64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
uint64_t part_bytes(uint64_t rows, uint64_t cols, uint32_t m) {
    return align_up((rows * cols + kChunk - 1) / kChunk * chunk_rows(cols) * m * 4);
}

}  // namespace

uint64_t gated_gemv_space(uint64_t rows, uint64_t cols, uint32_t m) {
    return 2 * part_bytes(rows, cols, m) + (m > 1 ? align_up((uint64_t)m * cols * 2) : 0);
}

int launch_gated_gemv(const afx_gated &w, const GatedGemv &q, uint8_t *ws, hipStream_t stream) {
    const uint64_t pb = part_bytes(w.rows, w.cols, q.m);
    const uint16_t *x = q.x;
    if (q.m > 1 && q.ldx != w.cols) {
        uint16_t *out = reinterpret_cast<uint16_t *>(ws + 2 * pb);
        uint64_t stride = q.ldx, cols = w.cols;
        void *args[] = {&x, &stride, &cols, &out};
        if (hipLaunchKernel(reinterpret_cast<const void *>(&afx_pack_rows_kernel),
                            dim3((unsigned)((cols / 8 + 255) / 256), q.m), dim3(256), args, 0, stream) != hipSuccess)
            return AFX_E_HIP;
        x = out;
    }
    GemvBatch batch;
    batch.n = 2;
    batch.j[0] = gemv_args({w.gate_info, w.gate_blob_dev, w.rows, w.cols, x, reinterpret_cast<float *>(ws)});
    batch.j[1] = gemv_args({w.up_info, w.up_blob_dev, w.rows, w.cols, x, reinterpret_cast<float *>(ws + pb)});
    batch.j[0].rows = batch.j[1].rows = chunk_rows(w.cols);
    JoinArgs a{};
    a.gate = batch.j[0].y;
    a.up = batch.j[1].y;
    a.h = q.h;
    a.g = q.g;
    a.u = q.u;
    a.ldh = q.ldh;
    a.ldgu = q.ldgu;
    a.rows = w.rows;
    a.cols = (uint32_t)w.cols;
    a.chunk_rows = (uint32_t)chunk_rows(w.cols);
    const bool all_long = w.cols >= kChunk;
    switch (q.m) {
        case 1: return launch_tokens<1>(batch, a, w.act, all_long, stream);
        case 2: return launch_tokens<2>(batch, a, w.act, all_long, stream);
        case 3: return launch_tokens<3>(batch, a, w.act, all_long, stream);
        default: return launch_tokens<4>(batch, a, w.act, all_long, stream);
    }
}

}  // namespace afx
