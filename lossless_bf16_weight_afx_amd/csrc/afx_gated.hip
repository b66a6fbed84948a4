// afx_gated.hip -- the gated feed-forward block over coded weights, its
// gradients, and the transposed product with a coded matrix (gfx950).
//
//   h = act(x Wg^T) * (x Wu^T)
//   dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu
//   y = d W
//
// "Why Weight Offloading Slows Inference" (section "Lossless compression")
// reconstructs a coded weight's bits ahead of the computation that uses it;
// these are the computations of a layer's feed-forward half around the
// products of afx_gemv.hip and afx_gemm.hip. The weights are coded and so
// constants: gradients are formed for the activations only.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "afx_act.h"
#include "afx_gated_gemm.h"
#include "afx_gated_gemv.h"
#include "afx_gemm_t.h"
#include "afx_mm.h"

namespace afx {
namespace {

constexpr uint64_t kMaxRows = 1ull << 21, kMaxCols = 1ull << 22, kMaxStride = 1ull << 22;
constexpr uint32_t kMaxTokens = 1u << 23;

uint64_t align_up(uint64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// ---- dg, du ------------------------------------------------------------------
struct GradArgs {
    const float *dh;
    const uint16_t *g, *u;
    uint16_t *dg, *du;    // the caller's, or NULL
    uint16_t *wdg, *wdu;  // [m, padded] for the product, zeros past the row, or NULL
    uint64_t ldh, ldgu, padded;
    uint32_t m, rows;
    uint32_t vec;         // every row starts aligned for four values at once
};

__device__ inline float bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Elementwise, four values per thread; bound by memory (4 + 2 + 2 bytes read,
// 4 or 8 written per value). The values go to the matrix cores as BF16: dg
// and du are rounded once here, before dx is summed in FP32. That costs dx as
// much as its own rounding does (1.7e-3 of its norm each, 2.4e-3 together;
// measured at 37 and 1024 tokens), and a second BF16 term for what the
// rounding leaves would double the matrix instructions; so dx is the gradient
// from the dg and du that the caller gets.
template <uint32_t kAct>
__global__ __launch_bounds__(256) void afx_gated_grad_kernel(const GradArgs p) {
    const uint32_t f = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (f >= p.padded) return;
    for (uint64_t t = blockIdx.y; t < p.m; t += gridDim.y) {
        uint16_t dg[4] = {}, du[4] = {};
        if (f < p.rows) {
            float dh[4] = {}, g[4] = {}, u[4] = {};
            const float *dhp = p.dh + t * p.ldh + f;
            const uint16_t *gp = p.g + t * p.ldgu + f, *up = p.u + t * p.ldgu + f;
            if (p.vec && f + 4 <= p.rows) {
                const float4 v = *reinterpret_cast<const float4 *>(dhp);
                const uint2 a = *reinterpret_cast<const uint2 *>(gp), b = *reinterpret_cast<const uint2 *>(up);
                dh[0] = v.x, dh[1] = v.y, dh[2] = v.z, dh[3] = v.w;
                g[0] = bf16((uint16_t)a.x), g[1] = __uint_as_float(a.x & 0xFFFF0000u);
                g[2] = bf16((uint16_t)a.y), g[3] = __uint_as_float(a.y & 0xFFFF0000u);
                u[0] = bf16((uint16_t)b.x), u[1] = __uint_as_float(b.x & 0xFFFF0000u);
                u[2] = bf16((uint16_t)b.y), u[3] = __uint_as_float(b.y & 0xFFFF0000u);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    if (f + i < p.rows) dh[i] = dhp[i], g[i] = bf16(gp[i]), u[i] = bf16(up[i]);
            }
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                float a, da;
                act_grad<kAct>(g[i], a, da);  // (past the row all three inputs are zero, and so both results)
                dg[i] = to_bf16(dh[i] * u[i] * da);
                du[i] = to_bf16(dh[i] * a);
            }
        }
        const uint2 dgv = make_uint2(dg[0] | ((uint32_t)dg[1] << 16), dg[2] | ((uint32_t)dg[3] << 16));
        const uint2 duv = make_uint2(du[0] | ((uint32_t)du[1] << 16), du[2] | ((uint32_t)du[3] << 16));
        if (p.wdg) {  // (padded is a multiple of 8)
            *reinterpret_cast<uint2 *>(p.wdg + t * p.padded + f) = dgv;
            *reinterpret_cast<uint2 *>(p.wdu + t * p.padded + f) = duv;
        }
        if (p.dg) {
            uint16_t *a = p.dg + t * p.ldgu + f, *b = p.du + t * p.ldgu + f;
            if (p.vec && f + 4 <= p.rows) {
                *reinterpret_cast<uint2 *>(a) = dgv;
                *reinterpret_cast<uint2 *>(b) = duv;
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    if (f + i < p.rows) a[i] = dg[i], b[i] = du[i];
            }
        }
    }
}

int launch_grad(const GradArgs &p, uint32_t act, hipStream_t stream) {
    GradArgs a = p;
    void *args[] = {&a};
    const void *fn = act == AFX_ACT_SILU        ? reinterpret_cast<const void *>(&afx_gated_grad_kernel<AFX_ACT_SILU>)
                     : act == AFX_ACT_GELU_TANH ? reinterpret_cast<const void *>(&afx_gated_grad_kernel<AFX_ACT_GELU_TANH>)
                                                : reinterpret_cast<const void *>(&afx_gated_grad_kernel<AFX_ACT_GELU>);
    const dim3 grid((unsigned)((p.padded / 4 + 255) / 256), std::min(p.m, 32768u));
    return hipLaunchKernel(fn, grid, dim3(256), args, 0, stream) == hipSuccess ? AFX_OK : AFX_E_HIP;
}

// ---- argument checks ---------------------------------------------------------
// A caller's buffer: m rows of `width` elements; or `bytes` in one piece.
RowSpan span(const void *p, uint32_t m, uint64_t stride, uint64_t width, uint64_t elem) {
    return RowSpan{p, m, width * elem, stride * elem};
}
RowSpan piece(const void *p, uint64_t bytes) { return RowSpan{p, bytes ? 1u : 0u, bytes, bytes}; }
bool any_overlap(const RowSpan *a, size_t na, const RowSpan *b, size_t nb) {
    for (size_t i = 0; i < na; ++i)
        for (size_t k = 0; k < nb; ++k)
            if (rows_overlap(a[i], b[k])) return true;
    return false;
}
bool pairs_overlap(const RowSpan *a, size_t n) {
    for (size_t i = 0; i < n; ++i)
        if (any_overlap(a + i, 1, a + i + 1, n - i - 1)) return true;
    return false;
}
bool misaligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

int check_matrix(const afx_info *info, const void *blob, uint64_t rows, uint64_t cols) {
    const int rc = check_info(info);
    if (rc != AFX_OK) return rc;
    if (!blob || rows == 0 || cols == 0) return AFX_E_INVALID_ARG;
    if (info->n_elems % cols || info->n_elems / cols != rows) return AFX_E_INVALID_ARG;
    if (cols % 8 || rows >= kMaxRows || cols >= kMaxCols) return AFX_E_UNSUPPORTED;
    return misaligned(blob, 16) ? AFX_E_MISALIGNED : AFX_OK;
}

int check_sizes(uint64_t rows, uint64_t cols, uint32_t m) {
    if (rows == 0 || cols == 0) return AFX_E_INVALID_ARG;
    return cols % 8 || rows >= kMaxRows || cols >= kMaxCols || m > kMaxTokens ? AFX_E_UNSUPPORTED : AFX_OK;
}

// Which kernels run a forward call. One to four tokens: the matrix-vector
// kernel. It and the next one, 3 tokens: two 17408 x 5120 matrices 81 and 89
// us, 300 x 17408 19 and 43; 4 tokens: 88 and 89, 20 and 43, 8192 x 4096 42 and
// 41, the worst for it 17408 x 512, 28 and 25; where the next one cannot run
// (17408 x 5112, 4 tokens), 88 and, restored first, 223. Up to 128: the fused
// matrix-core kernel, if rows hold whole groups of the coded format (it and
// restored first, two 17408 x 5120 matrices: 16 tokens 92 and 214, 128 177 and
// 229; 4096 x 2048, 128: 33 and 39; its sums and operands have no room for
// more). Else the matrices are restored to the workspace and multiplied there.
enum GatedPath { kPathGemv, kPathGemm, kPathRestore };
GatedPath gated_path(uint64_t cols, uint32_t m) {
    if (m <= kGatedGemvTokens) return kPathGemv;
    return m <= kGatedGemmTokens && cols % kGroup == 0 ? kPathGemm : kPathRestore;
}

// Whether a transposed product takes the coded matrices as they are, or has
// them restored to the workspace first. Fused and restored, rows of whole
// groups: the gradient of two 17408 x 5120 matrices, 16 tokens 103 and 191
// us, 64 125 and 200; 5120 x 17408, 64 tokens: 75 and 108; 1024 x 1024, 64: 18
// and 22. (Above 64 the fused kernel's sums would not fit its registers.) Other
// rows decode a third more: 5120 x 17400, 16 tokens: 75 and 104, two 4100 x
// 1528 26 and 32; but 37 tokens and two 4100 x 1528 matrices 37 and 34, 64 and
// 17408 x 5112 202 and 206.
bool transposed_fused(uint64_t cols, uint32_t m) {
    return m <= (cols % kGroup == 0 ? kGemmTTokens : kGemmTTokensSplit);
}

// Where the pieces of a gated call's workspace lie, and its size.
struct GatedSpace {
    uint64_t wg, wu, a0, a1, partial, bytes;  // a0: x as panels; or dg, and a1: du
};
uint64_t pad8(uint64_t v) { return (v + 7) / 8 * 8; }
GatedSpace gated_space(uint64_t rows, uint64_t cols, uint32_t m, bool backward) {
    GatedSpace s{};
    if (m == 0) return s;
    const GatedPath path = gated_path(cols, m);
    if (!backward && path != kPathRestore) {
        s.bytes = path == kPathGemv ? gated_gemv_space(rows, cols, m) : gated_gemm_space(rows, cols, m);
        return s;
    }
    const bool fused = backward && transposed_fused(cols, m);
    const uint64_t w = fused ? 0 : align_up(backward ? 2 * rows * cols : panel_bytes(rows, cols));
    const uint64_t a = align_up(backward ? 2 * m * pad8(rows) : panel_bytes(m, cols));
    s.wu = w;
    s.a0 = 2 * w;
    s.a1 = s.a0 + (backward ? a : 0);
    s.partial = s.a1 + a;
    s.bytes = s.partial +
              align_up(fused      ? gemm_t_space(rows, cols, 2, m)
                       : backward ? mm_transposed_partial(rows, cols, 2, m)
                                  : mm_gated_partial(rows, cols, m));
    return s;
}

int check_gated(const afx_gated *w, uint32_t m) {
    if (!w) return AFX_E_INVALID_ARG;
    int rc = check_matrix(w->gate_info, w->gate_blob_dev, w->rows, w->cols);
    if (rc != AFX_OK) return rc;
    rc = check_matrix(w->up_info, w->up_blob_dev, w->rows, w->cols);
    if (rc != AFX_OK) return rc;
    if (w->act > AFX_ACT_GELU) return AFX_E_INVALID_ARG;
    return m > kMaxTokens ? AFX_E_UNSUPPORTED : AFX_OK;
}

uint16_t *u16_at(void *ws, uint64_t at) { return reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + at); }

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_restore_gated_workspace(uint64_t rows, uint64_t cols, uint32_t m, int backward, size_t *bytes) {
    if (!bytes) return AFX_E_INVALID_ARG;
    const int rc = check_sizes(rows, cols, m);
    if (rc != AFX_OK) return rc;
    *bytes = gated_space(rows, cols, m, backward != 0).bytes;
    return AFX_OK;
}

int afx_restore_gated_async(const afx_gated *w, uint32_t m, const uint16_t *x_dev, uint64_t x_stride, uint16_t *h_dev,
                            uint64_t h_stride, uint16_t *g_dev, uint16_t *u_dev, uint64_t gu_stride, void *ws_dev,
                            size_t ws_bytes, void *stream) {
    int rc = check_gated(w, m);
    if (rc != AFX_OK) return rc;
    if (!g_dev != !u_dev) return AFX_E_INVALID_ARG;
    if (m == 0) return AFX_OK;
    const GatedSpace sp = gated_space(w->rows, w->cols, m, false);
    if (!x_dev || !h_dev || (!ws_dev && sp.bytes)) return AFX_E_INVALID_ARG;
    if (x_stride < w->cols || h_stride < w->rows || (g_dev && gu_stride < w->rows)) return AFX_E_INVALID_ARG;
    if (x_stride % 8 || x_stride >= kMaxStride || h_stride >= kMaxStride || (g_dev && gu_stride >= kMaxStride))
        return AFX_E_UNSUPPORTED;
    if (misaligned(x_dev, 16) || misaligned(ws_dev, 16) || misaligned(h_dev, 2) || misaligned(g_dev, 2) ||
        misaligned(u_dev, 2))
        return AFX_E_MISALIGNED;
    if (ws_bytes < sp.bytes) return AFX_E_BUFFER_TOO_SMALL;
    const RowSpan in[] = {piece(w->gate_blob_dev, w->gate_info->blob_bytes),
                          piece(w->up_blob_dev, w->up_info->blob_bytes),
                          span(x_dev, m, x_stride, w->cols, 2)};
    const RowSpan out[] = {span(h_dev, m, h_stride, w->rows, 2), span(g_dev, m, gu_stride, w->rows, 2),
                           span(u_dev, m, gu_stride, w->rows, 2), piece(ws_dev, sp.bytes)};
    if (any_overlap(in, 3, out, 4) || pairs_overlap(out, 4)) return AFX_E_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(ws_dev);
    const uint64_t gus = g_dev ? gu_stride : 0;
    const GatedPath path = gated_path(w->cols, m);
    if (path == kPathGemv) return launch_gated_gemv(*w, {x_dev, x_stride, m, h_dev, g_dev, u_dev, h_stride, gus}, ws, s);
    if (path == kPathGemm) return launch_gated_gemm(*w, {x_dev, x_stride, m, h_dev, g_dev, u_dev, h_stride, gus}, ws, s);
    const PanelJob jobs[2] = {{w->gate_info, w->gate_blob_dev, w->rows, w->cols, u16_at(ws, sp.wg)},
                              {w->up_info, w->up_blob_dev, w->rows, w->cols, u16_at(ws, sp.wu)}};
    rc = launch_panels(jobs, x_dev, x_stride, m, u16_at(ws, sp.a0), s);
    if (rc != AFX_OK) return rc;
    MmGated p{};
    p.x = u16_at(ws, sp.a0);
    p.m = m;
    p.wg = u16_at(ws, sp.wg);
    p.wu = u16_at(ws, sp.wu);
    p.rows = w->rows;
    p.cols = w->cols;
    p.act = w->act;
    p.h = h_dev;
    p.ldh = h_stride;
    p.g = g_dev;
    p.u = u_dev;
    p.ldgu = gus;
    p.partial = reinterpret_cast<float *>(ws + sp.partial);
    return launch_mm_gated(p, s);
}

int afx_restore_gated_backward_async(const afx_gated *w, uint32_t m, const float *dh_dev, uint64_t dh_stride,
                                     const uint16_t *g_dev, const uint16_t *u_dev, uint64_t gu_stride,
                                     uint16_t *dx_dev, uint64_t dx_stride, uint16_t *dg_dev, uint16_t *du_dev,
                                     void *ws_dev, size_t ws_bytes, void *stream) {
    int rc = check_gated(w, m);
    if (rc != AFX_OK) return rc;
    if (!dg_dev != !du_dev) return AFX_E_INVALID_ARG;
    if (m == 0) return AFX_OK;
    const GatedSpace sp = gated_space(w->rows, w->cols, m, true);
    if (!dh_dev || !g_dev || !u_dev || !dx_dev || !ws_dev) return AFX_E_INVALID_ARG;
    if (dh_stride < w->rows || gu_stride < w->rows || dx_stride < w->cols) return AFX_E_INVALID_ARG;
    if (dh_stride >= kMaxStride || gu_stride >= kMaxStride || dx_stride >= kMaxStride) return AFX_E_UNSUPPORTED;
    if (misaligned(dh_dev, 4) || misaligned(g_dev, 2) || misaligned(u_dev, 2) || misaligned(dx_dev, 2) ||
        misaligned(dg_dev, 2) || misaligned(du_dev, 2) || misaligned(ws_dev, 16))
        return AFX_E_MISALIGNED;
    if (ws_bytes < sp.bytes) return AFX_E_BUFFER_TOO_SMALL;
    const RowSpan gu[] = {span(g_dev, m, gu_stride, w->rows, 2), span(u_dev, m, gu_stride, w->rows, 2)};
    const RowSpan in[] = {piece(w->gate_blob_dev, w->gate_info->blob_bytes),
                          piece(w->up_blob_dev, w->up_info->blob_bytes),
                          span(dh_dev, m, dh_stride, w->rows, 4)};
    const RowSpan out[] = {span(dx_dev, m, dx_stride, w->cols, 2), span(dg_dev, m, gu_stride, w->rows, 2),
                           span(du_dev, m, gu_stride, w->rows, 2), piece(ws_dev, sp.bytes)};
    if (any_overlap(in, 3, out, 4) || pairs_overlap(out, 4)) return AFX_E_INVALID_ARG;
    // g and u may be replaced in place by dg and du, and only so
    if (any_overlap(gu, 2, out, 1) || any_overlap(gu, 2, out + 3, 1)) return AFX_E_INVALID_ARG;
    if ((dg_dev != g_dev && any_overlap(gu, 1, out + 1, 1)) || any_overlap(gu, 1, out + 2, 1) ||
        (du_dev != u_dev && any_overlap(gu + 1, 1, out + 2, 1)) || any_overlap(gu + 1, 1, out + 1, 1))
        return AFX_E_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(ws_dev);
    GradArgs a{};
    a.dh = dh_dev;
    a.g = g_dev;
    a.u = u_dev;
    a.dg = dg_dev;
    a.du = du_dev;
    // The product reads the caller's dg and du if their rows are whole
    // 16-byte pieces, else copies in the workspace.
    const bool direct = dg_dev && w->rows % 8 == 0 && gu_stride % 8 == 0 && !misaligned(dg_dev, 16) &&
                        !misaligned(du_dev, 16);
    if (!direct) {
        a.wdg = u16_at(ws, sp.a0);
        a.wdu = u16_at(ws, sp.a1);
    }
    a.ldh = dh_stride;
    a.ldgu = gu_stride;
    a.padded = pad8(w->rows);
    a.m = m;
    a.rows = (uint32_t)w->rows;
    a.vec = dh_stride % 4 == 0 && gu_stride % 4 == 0 && !misaligned(dh_dev, 16) && !misaligned(g_dev, 8) &&
            !misaligned(u_dev, 8) && !misaligned(dg_dev, 8) && !misaligned(du_dev, 8);
    rc = launch_grad(a, w->act, s);
    if (rc != AFX_OK) return rc;
    const uint16_t *dg = direct ? dg_dev : a.wdg, *du = direct ? du_dev : a.wdu;
    const uint64_t lda = direct ? gu_stride : a.padded;
    if (transposed_fused(w->cols, m))
        return launch_gemm_t({{w->gate_info, w->up_info}, {w->gate_blob_dev, w->up_blob_dev}, 2, w->rows, w->cols,
                              {dg, du}, lda, m, nullptr, dx_dev, dx_stride, false}, ws + sp.partial, s);
    const size_t bytes = 2 * w->rows * w->cols;
    const afx_job jobs[2] = {{w->gate_info, w->gate_blob_dev, u16_at(ws, sp.wg), bytes},
                             {w->up_info, w->up_blob_dev, u16_at(ws, sp.wu), bytes}};
    rc = afx_decode_layer_async(jobs, 2, s);
    if (rc != AFX_OK) return rc;
    MmTransposed p{};
    p.a[0] = dg;
    p.a[1] = du;
    p.lda = lda;
    p.m = m;
    p.w[0] = u16_at(ws, sp.wg);
    p.w[1] = u16_at(ws, sp.wu);
    p.n_mats = 2;
    p.rows = w->rows;
    p.cols = w->cols;
    p.y16 = dx_dev;
    p.ldy = dx_stride;
    p.partial = reinterpret_cast<float *>(ws + sp.partial);
    return launch_mm_transposed(p, s);
}

int afx_restore_gemm_t_workspace(uint64_t rows, uint64_t cols, uint32_t m, size_t *bytes) {
    if (!bytes) return AFX_E_INVALID_ARG;
    const int rc = check_sizes(rows, cols, m);
    if (rc != AFX_OK) return rc;
    if (rows % 8) return AFX_E_UNSUPPORTED;
    *bytes = m == 0                     ? 0
             : transposed_fused(cols, m) ? align_up(gemm_t_space(rows, cols, 1, m))
                                         : align_up(2 * rows * cols) +
                                               align_up(mm_transposed_partial(rows, cols, 1, m));
    return AFX_OK;
}

int afx_restore_gemm_t_async(const afx_info *info, const void *blob_dev, uint64_t rows, uint64_t cols,
                             const uint16_t *d_dev, uint32_t m, float *y_dev, int add, void *ws_dev, size_t ws_bytes,
                             void *stream) {
    int rc = check_matrix(info, blob_dev, rows, cols);
    if (rc != AFX_OK) return rc;
    size_t need = 0;
    rc = afx_restore_gemm_t_workspace(rows, cols, m, &need);
    if (rc != AFX_OK) return rc;
    if (m == 0) return AFX_OK;
    if (!d_dev || !y_dev || !ws_dev) return AFX_E_INVALID_ARG;
    if (misaligned(d_dev, 16) || misaligned(y_dev, 4) || misaligned(ws_dev, 16)) return AFX_E_MISALIGNED;
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
    const RowSpan in[] = {piece(blob_dev, info->blob_bytes), span(d_dev, m, rows, rows, 2)};
    const RowSpan out[] = {span(y_dev, m, cols, cols, 4), piece(ws_dev, need)};
    if (any_overlap(in, 2, out, 2) || pairs_overlap(out, 2)) return AFX_E_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (transposed_fused(cols, m))
        return launch_gemm_t({{info, nullptr}, {blob_dev, nullptr}, 1, rows, cols, {d_dev, nullptr}, rows, m, y_dev,
                              nullptr, cols, add != 0}, static_cast<uint8_t *>(ws_dev), s);
    const afx_job job{info, blob_dev, ws_dev, 2 * rows * cols};
    rc = afx_decode_layer_async(&job, 1, s);
    if (rc != AFX_OK) return rc;
    MmTransposed p{};
    p.a[0] = d_dev;
    p.lda = rows;
    p.m = m;
    p.w[0] = u16_at(ws_dev, 0);
    p.n_mats = 1;
    p.rows = rows;
    p.cols = cols;
    p.y32 = y_dev;
    p.ldy = cols;
    p.add = add != 0;
    p.partial = reinterpret_cast<float *>(u16_at(ws_dev, align_up(2 * rows * cols)));
    return launch_mm_transposed(p, s);
}

}  // extern "C"
