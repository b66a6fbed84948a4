/*
 * afx.h -- C ABI of libafx: lossless BF16 weight blobs restored on the GPU.
 *
 * The operation. "Why Weight Offloading Slows Inference" (section "Three
 * steps for each weight", Eq. (1)) puts an unpack step, t_unpack, between
 * reading a stored weight and using it; section "Lossless compression"
 * entropy-codes the BF16 exponent field without loss (a minimum-redundancy
 * prefix code, that page's reference [2]), so that each weight's original
 * 16 bits must be reconstructed before it is used. This library performs that
 * reconstruction on an
 * AMD Instinct MI355X (gfx950), after the compressed bytes have been copied
 * to device memory, and writes the BF16 bit patterns into a caller buffer.
 *
 * Blob format (version 1), little-endian; every section starts on a
 * 256-byte boundary and the blob length is a multiple of 256:
 *   [0,256)        header: "AFX1", u32 version = 1, u64 n, u64 total_bits,
 *                  u64 exp_words, u32 ndim, u32 4096, u32 32, u32 12,
 *                  u32 n_symbols, 12 zero bytes, u64 shape[4] at byte 64, zeros
 *   code_len[256]  u8 code length of each exponent value (0 = unused, <= 12)
 *   chunk_base     u64 x (n_chunks + 1): bit position where each 4096-element
 *                  chunk starts; the last entry equals total_bits
 *   gap            u16 x n_groups: start of each 32-element group, in bits
 *                  after its chunk's base
 *   signmant       u8 x n: (sign << 7) | mantissa7 of each element
 *   exp            u32 x exp_words: the canonical code stream of the 8-bit
 *                  exponent fields, MSB first in each word, then zero words
 * Element i is ((signmant[i] & 0x80) << 8) | (exponent << 7) |
 * (signmant[i] & 0x7F). The code is canonical: symbols ordered by (length,
 * value) take consecutive codes; a tensor with one exponent value uses one
 * 1-bit code.
 *
 * Conventions. Every function returns AFX_OK (0) or a negative afx_status,
 * never aborts and never prints. Argument and format errors are detected
 * before any HIP call and leave every output untouched. The library keeps no
 * pointer after a call returns and allocates no device memory.
 */
#ifndef AFX_H
#define AFX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define AFX_ABI_VERSION 1u
#define AFX_FORMAT_VERSION 1u
#define AFX_CHUNK_ELEMS 4096u
#define AFX_GROUP_ELEMS 32u
#define AFX_MAX_CODE_LEN 12u
#define AFX_MAX_JOBS_PER_LAUNCH 32u

typedef enum afx_status {
    AFX_OK = 0,
    AFX_E_INVALID_ARG = -1,     /* NULL pointer, zero-size or inconsistent argument */
    AFX_E_BAD_MAGIC = -2,       /* blob does not start with "AFX1" */
    AFX_E_BAD_VERSION = -3,     /* unknown format version or fixed-field value */
    AFX_E_CORRUPT = -4,         /* inconsistent header, code lengths, bases or gaps */
    AFX_E_BUFFER_TOO_SMALL = -5,/* blob shorter than its header says, or output too small */
    AFX_E_MISALIGNED = -6,      /* device pointer not 16-byte aligned */
    AFX_E_HIP = -7,             /* a HIP runtime call failed (launch or execution) */
    AFX_E_UNSUPPORTED = -8,     /* request beyond what the library supports */
    AFX_E_IO = -9,              /* a file could not be opened or read in full */
    AFX_E_HOST_MEMORY = -10     /* host memory for the call's own work could not be had */
} afx_status;
/* No entry point throws, aborts or prints: the host-side calls that allocate
 * working memory (the encoder, the host unpack, the file reader) return
 * AFX_E_HOST_MEMORY when it cannot be had, and run on fewer threads when
 * threads cannot be started. */

/* What afx_query reports about a blob. Offsets are in bytes from the blob's
 * first byte; sizes count elements unless named *_bytes. */
typedef struct afx_info {
    uint32_t abi_version;     /* AFX_ABI_VERSION of the library that filled it */
    uint32_t format_version;  /* 1 */
    uint64_t n_elems;         /* BF16 elements restored */
    uint64_t decoded_bytes;   /* 2 * n_elems */
    uint64_t blob_bytes;      /* bytes of the blob, a multiple of 256 */
    uint64_t total_bits;      /* length of the exponent code stream */
    uint64_t exp_words;       /* u32 words of the exp section, padding included */
    uint64_t n_chunks;        /* ceil(n / 4096) */
    uint64_t n_groups;        /* ceil(n / 32) */
    uint32_t ndim;            /* 0..4 */
    uint32_t n_symbols;       /* exponent values in use */
    uint64_t shape[4];        /* unused dimensions are 0 */
    uint32_t chunk_elems;     /* 4096 */
    uint32_t group_elems;     /* 32 */
    uint32_t max_code_len;    /* 12 */
    uint32_t longest_code;    /* longest length actually used */
    uint64_t off_code_len, off_chunk_base, off_gap, off_signmant, off_exp;
} afx_info;

/* One tensor of a batch. */
typedef struct afx_job {
    const afx_info *info;  /* filled by afx_query from a host copy of the blob */
    const void *blob_dev;  /* device copy of the same blob, 16-byte aligned */
    void *out_dev;         /* device output of n_elems u16 (BF16), 16-byte aligned */
    size_t out_bytes;      /* capacity of out_dev in bytes, >= 2 * n_elems */
} afx_job;

/* afx_query: inspect a blob held in host memory (pageable or pinned).
 * Checks the header, the code lengths (each <= 12; Kraft sum exactly 1 when
 * two or more values are used, a single 1-bit code otherwise), the chunk
 * bases (start at 0, non-decreasing, at most 12 bits per element, end at
 * total_bits) and the group gaps (0 at each chunk start, non-decreasing,
 * within the chunk), then fills *info. Host only, no HIP call.
 * Errors: AFX_E_INVALID_ARG (NULL), AFX_E_BUFFER_TOO_SMALL (blob_bytes short),
 * AFX_E_BAD_MAGIC, AFX_E_BAD_VERSION, AFX_E_CORRUPT. */
int afx_query(const void *blob_host, size_t blob_bytes, afx_info *info);

/* afx_decode_tensor: restore one tensor and wait for it.
 * info comes from afx_query on a host copy of the blob whose device copy is
 * blob_dev. Writes exactly 2 * n_elems bytes at out_dev and nothing else.
 * stream is a hipStream_t (NULL = the default stream); the call enqueues the
 * decode on it and then synchronizes that stream, so asynchronous kernel
 * errors are reported too. Output must not overlap the blob.
 * Errors: AFX_E_INVALID_ARG, AFX_E_BUFFER_TOO_SMALL (out_bytes < 2n),
 * AFX_E_MISALIGNED, AFX_E_HIP. A device blob that differs from the validated
 * host copy decodes to wrong values but never reads or writes out of bounds. */
int afx_decode_tensor(const afx_info *info, const void *blob_dev, void *out_dev, size_t out_bytes,
                      void *stream);

/* afx_decode_layer_async: restore a batch of tensors (e.g. the 11 tensors of
 * one decoder layer, the unit that page's section "Loading during
 * computation" prefetches) with one launch per AFX_MAX_JOBS_PER_LAUNCH jobs,
 * enqueued on stream; returns without waiting. Completion is observed through
 * the stream or events recorded on it. All jobs are checked before anything
 * is enqueued. Errors: as afx_decode_tensor, but only enqueue-time HIP errors
 * are reported; AFX_E_HOST_MEMORY when the host memory for the overlap check
 * of a batch of more than 1024 jobs cannot be had (up to 1024 it allocates
 * nothing). */
int afx_decode_layer_async(const afx_job *jobs, size_t n_jobs, void *stream);

/* afx_decode_layer_grid_async: afx_decode_layer_async on at most
 * max_workgroups workgroups per launch (one workgroup per CU at most, so
 * this many CUs at most; a larger value is the whole device, as in
 * afx_decode_layer_async). For a caller that restores the next unit while
 * its computation runs on the same GPU ("Why Weight Offloading Slows
 * Inference", section "Loading during computation"): the restore then
 * leaves the other CUs to that computation. Outputs are the same bits for
 * every max_workgroups. Errors: as afx_decode_layer_async;
 * AFX_E_INVALID_ARG when max_workgroups is 0. */
int afx_decode_layer_grid_async(const afx_job *jobs, size_t n_jobs, uint32_t max_workgroups, void *stream);

/* afx_status_str: a static description of a status code. */
const char *afx_status_str(int status);

/* ---- Encoder (host). Produces format-1 blobs; the code lengths are an
 * optimal prefix code limited to 12 bits over the tensor's exponent values. */

/* afx_encode_plan: histogram the exponents of x (n BF16 bit patterns), pick
 * the code lengths, and report the stream length and the blob size.
 * threads <= 0 picks the hardware thread count. Errors: AFX_E_INVALID_ARG
 * (NULL pointer), AFX_E_UNSUPPORTED (n above 2^40), AFX_E_HOST_MEMORY. */
int afx_encode_plan(const uint16_t *x, uint64_t n, int threads, uint8_t code_len[256],
                    uint64_t *total_bits, uint64_t *blob_bytes);

/* afx_encode: write the blob for x with the lengths and stream length from
 * afx_encode_plan into blob (host memory, blob_bytes >= the planned size).
 * shape has ndim entries (ndim 1..4, product == n). Errors: AFX_E_INVALID_ARG
 * (NULL pointer, ndim out of range, shape product != n, code_len not a
 * complete prefix code of lengths <= 12 -- Kraft sum 1, or one symbol of
 * length 1 --, an exponent of x without a code, total_bits not the stream
 * length those lengths give x), AFX_E_UNSUPPORTED (n above 2^40),
 * AFX_E_BUFFER_TOO_SMALL (blob_bytes below the blob size),
 * AFX_E_HOST_MEMORY. On an error the blob's contents are unspecified. */
int afx_encode(const uint16_t *x, uint64_t n, uint32_t ndim, const uint64_t *shape,
               const uint8_t code_len[256], uint64_t total_bits, void *blob, size_t blob_bytes,
               int threads);

/* ---- The restore fused into its consumer. "Why Weight Offloading Slows
 * Inference" (section "Lossless compression") reconstructs a weight's bits
 * ahead of the computation that uses it; when that computation is a product
 * on the GPU, the reconstructed matrix need not reach HBM at all. */

/* afx_restore_gemv_async: y += W x, where W is the tensor of the device blob
 * (info from afx_query on a host copy), taken as row-major [rows, cols]
 * (rows * cols == n_elems), x is BF16 [m, cols] and y FP32 [m, rows], both
 * row-major in device memory; m is 1, 2 or 4. W is restored chunk by chunk
 * in registers and LDS and never written out. Products of two BF16 values
 * are exact in FP32; the sums are FP32 and added into y with atomic adds,
 * so their order (and the last bits) may differ between calls. The caller
 * owns y and its initial contents. Enqueued on stream; returns without
 * waiting. Errors: as afx_decode_layer_async; AFX_E_INVALID_ARG (rows *
 * cols != n_elems, NULL pointer, y sharing a byte with the blob or x),
 * AFX_E_UNSUPPORTED (cols not a multiple of
 * 8 or 2^31 or more; m not 1, 2 or 4), AFX_E_MISALIGNED (blob or x not
 * 16-byte aligned, y not 4-byte aligned). */
int afx_restore_gemv_async(const afx_info *info, const void *blob_dev, uint64_t rows, uint64_t cols,
                           const uint16_t *x_dev, uint32_t m, float *y_dev, void *stream);

#define AFX_MAX_GEMV_JOBS_PER_LAUNCH 16u

/* One matrix of a batch of products (e.g. the seven of a decoder layer). */
typedef struct afx_gemv_job {
    const afx_info *info;  /* filled by afx_query from a host copy of the blob */
    const void *blob_dev;  /* device copy of the same blob, 16-byte aligned */
    uint64_t rows, cols;   /* W is row-major [rows, cols], rows * cols == n_elems */
    const uint16_t *x_dev; /* BF16 [m, cols], 16-byte aligned */
    float *y_dev;          /* FP32 [m, rows], added into, 4-byte aligned */
} afx_gemv_job;

/* afx_restore_gemv_batch_async: afx_restore_gemv_async for every job (all
 * with the same m), one launch per AFX_MAX_GEMV_JOBS_PER_LAUNCH jobs; all
 * jobs are checked before anything is enqueued. Jobs may share x and may
 * add into the same y; no job's y may share a byte with any job's blob or
 * x (AFX_E_INVALID_ARG). Errors otherwise as afx_restore_gemv_async. */
int afx_restore_gemv_batch_async(const afx_gemv_job *jobs, size_t n_jobs, uint32_t m, void *stream);

/* ---- The restore fused into a product over many tokens (prefill). The
 * same restore as above, but tiles of W go from LDS straight into the
 * matrix cores instead of to HBM. */

/* afx_restore_gemm_async: y += x W^T, where W is the tensor of the device
 * blob (info from afx_query on a host copy), taken as row-major
 * [rows, cols] (rows * cols == n_elems), x is BF16 [m, cols] and y FP32
 * [m, rows], both row-major in device memory; any m >= 1. 64-row tiles of W
 * are restored into LDS 256 columns at a time and multiplied there with
 * BF16 matrix instructions (FP32 accumulation); for m = 1, 2 or 4 the call
 * runs afx_restore_gemv_async's kernel instead, which is faster for so few
 * tokens (the same y within the same bound). Tiles over different column
 * ranges of the same rows add their partial sums into y with atomic adds,
 * so their order (and the last bits) may differ between calls. The caller
 * owns y and its initial contents. Enqueued on stream; returns without
 * waiting. Errors: as afx_decode_layer_async; AFX_E_INVALID_ARG (rows *
 * cols != n_elems, a zero size, NULL pointer, y sharing a byte with the
 * blob or x), AFX_E_UNSUPPORTED (rows not
 * a multiple of 64, cols not a multiple of 256, either >= 2^31, m == 0 or
 * m > 8388480), AFX_E_MISALIGNED (blob or x not 16-byte aligned, y not
 * 4-byte aligned). */
int afx_restore_gemm_async(const afx_info *info, const void *blob_dev, uint64_t rows, uint64_t cols,
                           const uint16_t *x_dev, uint32_t m, float *y_dev, void *stream);

/* afx_restore_gemm_batch_async: afx_restore_gemm_async for every job (all
 * with the same m), one launch per AFX_MAX_GEMV_JOBS_PER_LAUNCH jobs; all
 * jobs are checked before anything is enqueued. Jobs may share x and may
 * add into the same y; no job's y may share a byte with any job's blob or
 * x (AFX_E_INVALID_ARG). Errors otherwise as afx_restore_gemm_async. */
int afx_restore_gemm_batch_async(const afx_gemv_job *jobs, size_t n_jobs, uint32_t m, void *stream);

/* ---- The feed-forward half of a layer around those products, over coded
 * weights ("Why Weight Offloading Slows Inference", section "Lossless
 * compression": the bits are reconstructed before the computation that uses
 * them). A coded weight is a constant: gradients are formed for activations,
 * and for the norms' own (uncoded) weights and gates. All buffers are device
 * memory owned by the caller; a workspace holds nothing between calls, and
 * calls that may run at the same time (two streams, two captured graphs)
 * each need their own. Strides count elements between rows (tokens). Buffers
 * that may not share a byte may be column ranges of one wider matrix (rows
 * the same number of bytes apart); of buffers with other row distances whole
 * extents are compared, from the first byte to the last. */

typedef enum afx_act {
    AFX_ACT_SILU = 0,      /* g / (1 + e^-g) */
    AFX_ACT_GELU_TANH = 1, /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
    AFX_ACT_GELU = 2       /* 0.5 g (1 + erf(g / sqrt(2))) */
} afx_act;

/* The two projections of a gated feed-forward block: the tensors of two
 * blobs, both taken as row-major [rows, cols] (rows * cols == n_elems). */
typedef struct afx_gated {
    const afx_info *gate_info;  /* filled by afx_query from host copies */
    const void *gate_blob_dev;  /* device copies of the blobs, 16-byte aligned */
    const afx_info *up_info;
    const void *up_blob_dev;
    uint64_t rows, cols;
    uint32_t act; /* an afx_act */
} afx_gated;

/* afx_restore_gated_workspace: bytes of device workspace that
 * afx_restore_gated_async (backward == 0) or
 * afx_restore_gated_backward_async (backward != 0) needs for m tokens. Host
 * only. Errors: AFX_E_INVALID_ARG (NULL, a zero size), AFX_E_UNSUPPORTED
 * (cols not a multiple of 8, rows >= 2^21, cols >= 2^22, m > 2^23). */
int afx_restore_gated_workspace(uint64_t rows, uint64_t cols, uint32_t m, int backward, size_t *bytes);

/* afx_restore_gated_async: h = act(x Wg^T) * (x Wu^T) for m tokens, x BF16
 * [m, cols], h BF16 [m, rows]; any m (0 does nothing), any rows, cols a
 * multiple of 8. The sums g = x Wg^T and u = x Wu^T, the activation and the
 * product are FP32; h is rounded to BF16 once. With g_dev and u_dev (both
 * or neither) g and u are written too, rounded to BF16, for the backward
 * pass. Results are the same bits on every run. Enqueued on stream; returns
 * without waiting. No output or workspace may share a byte with an input or
 * with another output. Errors: as afx_decode_layer_async; AFX_E_INVALID_ARG
 * (NULL pointer, rows * cols != n_elems, one of g_dev and u_dev, a stride
 * shorter than its row, unknown act, buffers sharing bytes),
 * AFX_E_UNSUPPORTED (sizes as above, x_stride not a multiple of 8, a stride
 * >= 2^22), AFX_E_MISALIGNED (blobs, x or workspace not 16-byte aligned),
 * AFX_E_BUFFER_TOO_SMALL (workspace). */
int afx_restore_gated_async(const afx_gated *w, uint32_t m, const uint16_t *x_dev, uint64_t x_stride, uint16_t *h_dev,
                            uint64_t h_stride, uint16_t *g_dev, uint16_t *u_dev, uint64_t gu_stride, void *ws_dev,
                            size_t ws_bytes, void *stream);

/* afx_restore_gated_backward_async: the gradients of afx_restore_gated_async
 * for dh FP32 [m, rows] (as afx_restore_gemm_t_async writes it), from the g
 * and u it kept: dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu, dx
 * BF16 [m, cols]. dg and du are rounded to BF16 (the matrix cores' operand
 * type) and dx is their FP32 sum, rounded to BF16 once. With dg_dev and
 * du_dev (both or neither, rows gu_stride apart like g and u) they are
 * written too: the gradient of a weight matrix, where a program keeps one,
 * is dg^T x or du^T x. dg_dev may be g_dev and du_dev may be u_dev (in
 * place); otherwise nothing may overlap. Same bits on every run. Errors: as
 * afx_restore_gated_async (dh 4-byte aligned). */
int afx_restore_gated_backward_async(const afx_gated *w, uint32_t m, const float *dh_dev, uint64_t dh_stride,
                                     const uint16_t *g_dev, const uint16_t *u_dev, uint64_t gu_stride,
                                     uint16_t *dx_dev, uint64_t dx_stride, uint16_t *dg_dev, uint16_t *du_dev,
                                     void *ws_dev, size_t ws_bytes, void *stream);

/* afx_restore_gemm_t_workspace: bytes of device workspace that
 * afx_restore_gemm_t_async needs for m tokens. Host only. Errors:
 * AFX_E_INVALID_ARG (NULL, a zero size), AFX_E_UNSUPPORTED (rows or cols not
 * a multiple of 8, rows >= 2^21, cols >= 2^22, m > 2^23). */
int afx_restore_gemm_t_workspace(uint64_t rows, uint64_t cols, uint32_t m, size_t *bytes);

/* afx_restore_gemm_t_async: y = d W (add == 0) or y += d W (add != 0), where
 * W is the tensor of the device blob taken as row-major [rows, cols], d is
 * BF16 [m, rows] and y FP32 [m, cols], both row-major without gaps: the
 * input gradient of afx_restore_gemm_async's product y = x W^T. Any m (0
 * does nothing). Sums are FP32, in an order that depends on the sizes only:
 * the same bits on every run. Enqueued on stream; returns without waiting.
 * y and the workspace may not share a byte with the blob, d or each other.
 * Errors: as afx_decode_layer_async; AFX_E_INVALID_ARG (NULL pointer, rows *
 * cols != n_elems, buffers sharing bytes), AFX_E_UNSUPPORTED (sizes as
 * above), AFX_E_MISALIGNED (blob, d or workspace not 16-byte aligned, y not
 * 4-byte aligned), AFX_E_BUFFER_TOO_SMALL (workspace). */
int afx_restore_gemm_t_async(const afx_info *info, const void *blob_dev, uint64_t rows, uint64_t cols,
                             const uint16_t *d_dev, uint32_t m, float *y_dev, int add, void *ws_dev, size_t ws_bytes,
                             void *stream);

#define AFX_MAX_NORM_WIDTH 32768u

typedef enum afx_type { AFX_TYPE_BF16 = 0, AFX_TYPE_FP32 = 1 } afx_type;

/* What stands between two blocks of a layer: a norm after the first, its
 * gate and residual scale, the residual add, and the norm before the second.
 *   bh = b * rsqrt(mean(b^2) + eps) * w_post   (w_post NULL: bh = b)
 *   r' = r + scale * gate * bh                 (gate NULL: 1)
 *   xn = r' * rsqrt(mean(r'^2) + eps) * w_pre
 * means over the d values of a row. The residual stream r, r' (and its
 * gradients) has type r_type; b is FP32 (a product's y), xn BF16 (a
 * product's x). */
typedef struct afx_block_norm {
    uint64_t d;             /* width, 1..AFX_MAX_NORM_WIDTH */
    float eps;              /* > 0 */
    float scale;            /* a constant of the block: it has no gradient here */
    uint32_t r_type;        /* an afx_type */
    const uint16_t *w_post; /* device, BF16 [d], or NULL */
    const uint16_t *gate;   /* device, BF16 [d] (gate_stride 0) or [m, d], or NULL */
    uint64_t gate_stride;   /* 0: one gate for all rows; else elements between rows, >= d */
    const uint16_t *w_pre;  /* device, BF16 [d], or NULL (no xn) */
} afx_block_norm;

/* afx_block_norm_async: r' and xn of m rows. b_dev NULL: r' = r (only the
 * norm before a block; w_post and gate are not read). r_out_dev (r') may be
 * r_dev itself with the same stride, or NULL when b_dev is NULL; xn_dev may
 * be NULL exactly when w_pre is. xn is computed from r' before r' is rounded
 * to r_type. All arithmetic is FP32 and each output is rounded once. Any m
 * (0 does nothing), any width up to AFX_MAX_NORM_WIDTH; fastest when d and
 * the strides are multiples of 8 and the buffers 16-byte aligned. Squares
 * are FP32: a value above about 1e19 overflows its row's mean to infinity.
 * Enqueued on stream; returns without waiting. Errors: AFX_E_INVALID_ARG
 * (NULL pointer, d 0, eps not > 0, scale not finite, unknown r_type, a
 * stride shorter than d, nothing to write, outputs sharing bytes with each
 * other or an input), AFX_E_UNSUPPORTED (d above AFX_MAX_NORM_WIDTH,
 * a stride of 2^28 or more), AFX_E_MISALIGNED (a pointer not aligned to its element), AFX_E_HIP. */
int afx_block_norm_async(const afx_block_norm *p, uint32_t m, const float *b_dev, uint64_t b_stride, const void *r_dev,
                         uint64_t r_stride, void *r_out_dev, uint64_t r_out_stride, uint16_t *xn_dev,
                         uint64_t xn_stride, void *stream);

/* afx_block_norm_workspace: bytes of device workspace that
 * afx_block_norm_backward_async needs for m rows. Host only. Errors:
 * AFX_E_INVALID_ARG, AFX_E_UNSUPPORTED as above. */
int afx_block_norm_workspace(const afx_block_norm *p, uint32_t m, size_t *bytes);

/* afx_block_norm_backward_async: the gradients of afx_block_norm_async from
 * b and r' (r_out, as it was written) and the gradients dxn (BF16) and
 * dr_out (r_type) of its outputs, either of which may be NULL (zero; dxn
 * must be NULL when w_pre is):
 *   dr  = dr_out + the gradient of xn through r'     [m, d] of r_type
 *   db  = the gradient of r' through b               [m, d] BF16 (a product's d)
 *   dw_pre = sum over rows of dxn r' rsqrt(..)       FP32 [d]
 *   dw_post, and dgate: FP32 [d], or dgate FP32 [m, d] when gate_stride != 0
 * Each output may be NULL (not computed). dr_dev may be dr_out_dev itself
 * with the same stride. dr is used unrounded in the others. b_dev NULL: only
 * dr and dw_pre. The sums over rows are FP32 and their order depends on the
 * sizes only (that of the sums within a row, here and in the forward call,
 * also on whether d, strides and alignment allow 8 values at a time): the
 * same bits on every run; with m == 0 they are written as zeros. Errors: as afx_block_norm_async (asking for dw_pre without w_pre,
 * dw_post without w_post, dgate without gate, or db, dw_post or dgate
 * without b is AFX_E_INVALID_ARG); AFX_E_BUFFER_TOO_SMALL (workspace),
 * AFX_E_MISALIGNED also for a workspace not 16-byte aligned. */
int afx_block_norm_backward_async(const afx_block_norm *p, uint32_t m, const float *b_dev, uint64_t b_stride,
                                  const void *r_out_dev, uint64_t r_out_stride, const uint16_t *dxn_dev,
                                  uint64_t dxn_stride, const void *dr_out_dev, uint64_t dr_out_stride, void *dr_dev,
                                  uint64_t dr_stride, uint16_t *db_dev, uint64_t db_stride, float *dw_pre_dev,
                                  float *dw_post_dev, float *dgate_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* ---- The attention half of a layer around the products: what stands between
 * the q, k and v products and the attention, the attention of new tokens
 * over a paged cache, and the cache's pages. Conventions (buffers, strides,
 * workspaces) are those of the feed-forward half above. Page ids, lengths,
 * slots and row starts are device memory that the host never reads: a value
 * outside its range is treated as its call says and never reaches memory out
 * of bounds. */

#define AFX_MAX_HEAD_DIM 256u

/* Keys and values of one layer, in pages of page_tokens tokens each:
 *   k_dev: BF16 [n_pages][kv_heads][head_dim / 8][page_tokens][8]
 *   v_dev: BF16 [n_pages][kv_heads][page_tokens / 8][head_dim][8]
 * (the order in which the matrix cores take them: 8 consecutive dimensions of
 * a key, 8 consecutive tokens of a value). A slot, page * page_tokens + its
 * place in the page, names a token's place. */
typedef struct afx_kv_pages {
    uint16_t *k_dev, *v_dev; /* 16-byte aligned */
    uint32_t n_pages;        /* n_pages * page_tokens < 2^31 */
    uint32_t page_tokens;    /* 16, 32, 64, 128 or 256 */
    uint32_t kv_heads;       /* 1..1024 */
    uint32_t head_dim;       /* a multiple of 8 up to AFX_MAX_HEAD_DIM */
} afx_kv_pages;

/* Which two values of a head turn together. */
typedef enum afx_pairing {
    AFX_ROPE_HALVES = 0,    /* i and i + rot_dim / 2 */
    AFX_ROPE_NEIGHBOURS = 1 /* 2 i and 2 i + 1 */
} afx_pairing;

/* Norm and rotary positions of the query and key heads:
 *   n = x * rsqrt(mean(x^2) + eps) * w   over a head's values (w NULL: n = x)
 *   a' = n_a cos t - n_b sin t, b' = n_b cos t + n_a sin t for every pair
 *   (a, b) of the first rot_dim values, t = position[axis[i]] * freq[i] of
 *   its pair i; the other values stay n.
 * Positions may have several axes (time, height and width of images and
 * video), each pair turning with one of them. */
typedef struct afx_heads {
    uint32_t q_heads, kv_heads; /* 1..1024 */
    uint32_t head_dim;          /* a multiple of 8 up to AFX_MAX_HEAD_DIM */
    uint32_t rot_dim;           /* even, 0..head_dim */
    uint32_t pairing;           /* an afx_pairing */
    uint32_t n_axes;            /* 1..4 */
    float eps;                  /* > 0 (not used without w_q and w_k) */
    const uint16_t *w_q, *w_k;  /* device, BF16 [head_dim], or NULL */
    const float *freq;          /* device, FP32 [rot_dim / 2]: radians per position */
    const uint8_t *axis;        /* device [rot_dim / 2], each below n_axes (larger: the last); NULL: all 0 */
} afx_heads;

/* afx_heads_async: norm and positions of m tokens' query and key heads, and
 * the write of keys and values to the cache. q, k and v are FP32 rows (the
 * products' y) of q_heads or kv_heads heads; pos is int32 [n_axes] rows of m,
 * pos_stride apart (not read when rot_dim is 0; negative positions turn
 * back). q NULL: no query heads; k NULL: no keys; v NULL: no values. q_out
 * and k_out are BF16 rows; k_out may be NULL when kv is given. With kv, token
 * i's key and value go to slot slots[i]; a slot outside the cache (such as
 * -1) writes none. Slots inside it have to be distinct. Sums and rotations
 * are FP32 (a value above about 1e19 overflows its head's mean to infinity),
 * angles FP64, and each output is rounded once. Any m (0 does
 * nothing). Enqueued on stream; returns without waiting. Fastest when rot_dim
 * and the strides are multiples of 8 and the buffers 16-byte aligned. Errors:
 * AFX_E_INVALID_ARG (NULL pointer, nothing to do, a count out of its range,
 * kv of other heads, v or slots without kv, q without q_out or the other way
 * round, a stride shorter than its row, outputs sharing bytes with each other
 * or an input), AFX_E_UNSUPPORTED (head_dim, page_tokens or the cache's size
 * as above, a stride of 2^28 or more, m above 2^23), AFX_E_MISALIGNED,
 * AFX_E_HIP. */
int afx_heads_async(const afx_heads *p, uint32_t m, const int32_t *pos_dev, uint64_t pos_stride, const float *q_dev,
                    uint64_t q_stride, const float *k_dev, uint64_t k_stride, const float *v_dev, uint64_t v_stride,
                    uint16_t *q_out_dev, uint64_t q_out_stride, uint16_t *k_out_dev, uint64_t k_out_stride,
                    const afx_kv_pages *kv, const int32_t *slots_dev, void *stream);

/* afx_heads_workspace: bytes of device workspace that
 * afx_heads_backward_async needs for m tokens. Host only. */
int afx_heads_workspace(const afx_heads *p, uint32_t m, size_t *bytes);

/* afx_heads_backward_async: the gradients of afx_heads_async from its inputs
 * q and k and the gradients dq and dk (BF16) of q_out and k_out: dq_in and
 * dk_in BF16 (afx_restore_gemm_t_async's d), dw_q and dw_k FP32 [head_dim],
 * summed over tokens and heads in an order that depends on the sizes only
 * (the same bits on every run; zeros with m == 0). dq NULL: nothing of the
 * query heads, dk NULL: nothing of the keys. dq_in may be dq itself with the
 * same stride, dk_in dk. q (k) is only read where w_q (w_k) is given and may
 * else be NULL. dq_in, dk_in, dw_q and dw_k may each be NULL (not computed).
 * Errors: as afx_heads_async; AFX_E_INVALID_ARG for dw_q without w_q or dq
 * (dw_k likewise) where m is not 0, AFX_E_BUFFER_TOO_SMALL (workspace, only
 * needed for dw_q and dw_k). */
int afx_heads_backward_async(const afx_heads *p, uint32_t m, const int32_t *pos_dev, uint64_t pos_stride,
                             const float *q_dev, uint64_t q_stride, const float *k_dev, uint64_t k_stride,
                             const uint16_t *dq_dev, uint64_t dq_stride, const uint16_t *dk_dev, uint64_t dk_stride,
                             uint16_t *dq_in_dev, uint64_t dq_in_stride, uint16_t *dk_in_dev, uint64_t dk_in_stride,
                             float *dw_q_dev, float *dw_k_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* Which pages hold the tokens of n_seqs sequences: token j of sequence s is at
 * place j % page_tokens of page table[s][j / page_tokens]. Entries behind a
 * sequence's last page are -1. refs counts how many sequences hold a page; 0
 * is a free one. All three are changed by the afx_pages calls only. */
typedef struct afx_page_table {
    int32_t *table_dev;    /* [n_seqs] rows of max_pages, table_stride apart */
    uint64_t table_stride; /* elements */
    int32_t *len_dev;      /* [n_seqs]: tokens */
    int32_t *refs_dev;     /* [n_pages] (afx_attend_async does not read it: may be NULL there) */
    uint32_t n_seqs, max_pages, n_pages, page_tokens;
} afx_page_table;

/* Attention of new tokens. */
typedef struct afx_attend {
    uint32_t q_heads;  /* a multiple of the cache's kv_heads; q_heads / kv_heads <= 256 */
    float scale;       /* finite */
    uint32_t causal;   /* 0: every token sees its sequence's whole cache */
    uint32_t window;   /* 0: none; else a token sees itself and the window - 1 tokens before it (and, not causal,
                          those after it) */
    uint32_t max_new;  /* the most new tokens of a sequence and the most tokens of one, by which the */
    uint32_t max_len;  /* work is divided: larger ones come out right too, but take longer */
} afx_attend;

/* afx_attend_workspace: bytes of device workspace that afx_attend_async needs
 * for n_rows sequences with m new tokens in all. Host only. */
int afx_attend_workspace(const afx_attend *p, const afx_kv_pages *kv, uint32_t n_rows, uint32_t m, size_t *bytes);

/* afx_attend_async: out = softmax(scale q k^T) v for the new tokens of n_rows
 * sequences over the cache, which already holds them. Row r's new tokens are
 * rows starts[r] .. starts[r + 1] - 1 of q and out (starts: device, n_rows + 1
 * values from 0 to m, not decreasing; a row may have none), and belong to
 * sequence seqs[r] (seqs NULL: r). With len tokens in the sequence and n new
 * ones, new token i stands at position len - n + i and sees the positions up
 * to its own (causal), within its window. Query head h reads key and value
 * head h / (q_heads / kv_heads). q and out are BF16 rows of q_heads heads;
 * lse, if not NULL, is FP32 [m][q_heads]: the natural logarithm of the sum of
 * e^score. A query that sees nothing (or only scores of minus infinity) gets
 * zeros and an lse of minus infinity. Rows of q behind the last start are not
 * read, and those of out and lse are left as they were. What a query does not
 * see never changes its result, infinities and NaN in it included; an
 * infinite or NaN value that it sees, however little it weighs, makes its
 * output infinite or NaN. Tokens of a page whose id is outside the cache are
 * seen by none, rows whose sequence is outside the table have no tokens,
 * lengths are capped at max_pages pages, and starts at m. Scores and sums are FP32; the weights of the values are
 * rounded to BF16 (the matrix cores' operand), as is out. The same bits on
 * every run. Enqueued on stream; returns without waiting. Errors:
 * AFX_E_INVALID_ARG (NULL pointer, a count out of its range, a table of other
 * pages, a stride shorter than its row, outputs sharing bytes with each other
 * or an input), AFX_E_UNSUPPORTED (the cache's sizes as above, max_pages *
 * page_tokens above 2^31 - 1024, m above 2^23, n_rows above 2^16, a stride
 * of 2^28 or more, more work than one launch takes: kv_heads times the rows'
 * parts or query rows of 2^24 or more, or kv_heads times the parts of all
 * tiles of 256 query rows of 2^23 or more (above 128 dimensions: of 128 rows,
 * 2^24)), AFX_E_MISALIGNED (q, out or the workspace not
 * 16-byte aligned, strides not multiples of 8, or lse, starts, seqs, len or
 * the table not 4-byte aligned), AFX_E_BUFFER_TOO_SMALL, AFX_E_HIP. */
int afx_attend_async(const afx_attend *p, const afx_kv_pages *kv, const afx_page_table *t, uint32_t n_rows,
                     const int32_t *seqs_dev, const int32_t *starts_dev, uint32_t m, const uint16_t *q_dev,
                     uint64_t q_stride, uint16_t *out_dev, uint64_t out_stride, float *lse_dev, void *ws_dev,
                     size_t ws_bytes, void *stream);

/* ---- The cache's pages. These calls change tables, lengths and counts on the
 * GPU, without waiting and without the host seeing them, so that steps of
 * generation may be captured in a HIP graph. Each gives one result, whatever
 * runs at the same time inside it: that of taking its rows in their order.
 * Calls that share a table have to follow one another on a stream. Lists hold
 * at most AFX_MAX_PAGE_ROWS rows (AFX_E_UNSUPPORTED). Errors of all:
 * AFX_E_INVALID_ARG (NULL pointer, a zero size, table_stride below max_pages,
 * buffers sharing bytes), AFX_E_UNSUPPORTED (page_tokens not a power of two
 * from 16 to 256, n_pages * page_tokens or max_pages * page_tokens of 2^31 or
 * more, n_seqs above 2^20, table_stride of 2^28 or more), AFX_E_MISALIGNED,
 * AFX_E_BUFFER_TOO_SMALL (workspace), AFX_E_HIP. */

#define AFX_MAX_PAGE_ROWS 1024u

/* What the pages hold: n_planes arrays of n_pages pages (keys and values of
 * every layer), each page page_bytes long (a multiple of 16). */
typedef struct afx_page_data {
    void *data_dev;        /* 16-byte aligned */
    uint64_t page_bytes;   /* a multiple of 16, up to 2^30 */
    uint64_t plane_stride; /* bytes between planes: a multiple of 16, at least n_pages * page_bytes */
    uint32_t n_planes;     /* 1..65535 */
} afx_page_data;

/* afx_pages_fork_async: sequence dst[r] becomes a copy of src[r] that shares
 * all of its pages (their counts rise by one); no page is copied until one of
 * the holders grows into it. A row is refused, and changes nothing, if either
 * id is outside the table, dst[r] holds tokens, dst[r] is the dst of an
 * earlier row, or src[r] is the dst of any row. granted (int32 [n], may be
 * NULL) tells 1 or 0 for each row. */
int afx_pages_fork_async(const afx_page_table *t, uint32_t n, const int32_t *src_dev, const int32_t *dst_dev,
                         int32_t *granted_dev, void *stream);

/* afx_pages_trim_async: sequence seqs[r] keeps its first lens[r] tokens (lens
 * NULL: none: it is freed); pages behind them are given up (their counts fall
 * by one). A length of 0 or less frees, one above the sequence's changes
 * nothing. Rows with ids outside the table, or named in an earlier row, are
 * passed over. */
int afx_pages_trim_async(const afx_page_table *t, uint32_t n, const int32_t *seqs_dev, const int32_t *lens_dev,
                         void *stream);

/* afx_pages_extend_workspace: bytes of device workspace that
 * afx_pages_extend_async needs for n rows. Host only. */
int afx_pages_extend_workspace(const afx_page_table *t, uint32_t n, size_t *bytes);

/* afx_pages_extend_async: sequence seqs[r] grows by the starts[r + 1] -
 * starts[r] tokens of row r (as in afx_attend_async, m in all). It gets the
 * pages that it needs, the free ones of the lowest ids, rows in their order;
 * if its last page is partly filled and held by others too, it first gets a
 * copy of its own (of rows that share such a page, the last holder keeps it).
 * A row for which too few pages are left is refused with all rows after it; a
 * row is also refused if its id is outside the table or named in an earlier
 * row, or if the sequence would exceed max_pages pages. granted[r] (may be
 * NULL) is the number of tokens by which it grew. slots[i] is the slot of
 * token i (-1 for tokens of refused rows and those behind the last start),
 * pos[i] (may be NULL) its position in the sequence (0 there). The new slots'
 * contents are what they were. */
int afx_pages_extend_async(const afx_page_table *t, const afx_page_data *d, uint32_t n, const int32_t *seqs_dev,
                           const int32_t *starts_dev, uint32_t m, int32_t *slots_dev, int32_t *pos_dev,
                           int32_t *granted_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* afx_pages_compact_workspace: bytes of device workspace of
 * afx_pages_compact_async. Host only. */
int afx_pages_compact_workspace(const afx_page_table *t, size_t *bytes);

/* afx_pages_compact_async: the live pages (count above 0) move to the lowest
 * ids: with `live` of them, the k-th one at an id of `live` or more moves to
 * the k-th free id below it, the others stay. Tables and counts follow. map
 * (int32 [n_pages]) is each page's new id, -1 for free ones; live (int32 [1],
 * may be NULL) the number of live pages: what stays behind them is free. */
int afx_pages_compact_async(const afx_page_table *t, const afx_page_data *d, int32_t *map_dev, int32_t *live_dev,
                            void *ws_dev, size_t ws_bytes, void *stream);

/* afx_pages_copy_async: in every plane, page dst[i] becomes a copy of page
 * src[i], for n pairs (any n; 0 does nothing). Pairs with an id outside the
 * n_pages pages are passed over. No dst may be named twice or be a src. */
int afx_pages_copy_async(const afx_page_data *d, uint32_t n_pages, uint32_t n, const int32_t *src_dev,
                         const int32_t *dst_dev, void *stream);

/* ---- Unpack on the host. "Why Weight Offloading Slows Inference" (section
 * "The path from storage to the GPU", Figure 1) unpacks a compressed weight
 * in RAM between the read and the copy to the GPU, and section "Lossless
 * compression" finds that placement too slow for compression to pay
 * (Eq. (2)). The GPU entry points above never call this; it exists to
 * measure that placement beside the GPU restore. */

/* afx_decode_host: validate a host blob as afx_query does, then restore its
 * n_elems BF16 bit patterns into out (host memory, out_bytes >= 2 n), with
 * `threads` workers over chunks (<= 0: hardware thread count).
 * Errors: as afx_query; AFX_E_INVALID_ARG (NULL out with n > 0),
 * AFX_E_BUFFER_TOO_SMALL (out_bytes < 2 n), AFX_E_HOST_MEMORY. */
int afx_decode_host(const void *blob_host, size_t blob_bytes, uint16_t *out, size_t out_bytes, int threads);

/* ---- Storage (host). "Why Weight Offloading Slows Inference" (section
 * "The path from storage to the GPU", Figure 1, and Eq. (1)) reads a stored
 * weight from the SSD into RAM before unpacking it and copying it to the GPU;
 * the page measures that read with the page cache cleared. */

#define AFX_READ_DIRECT 1u /* open with O_DIRECT: bypass the page cache */

/* afx_file_read: read bytes [offset, offset + bytes) of the file at path into
 * dst (host memory owned by the caller, any alignment; pinned memory lets a
 * following copy to the GPU start from it), with `threads` workers (<= 0:
 * the hardware thread count) each issuing 4 MiB preads. With
 * AFX_READ_DIRECT each worker reads the enclosing 4096-aligned range into
 * its own page-aligned 4 MiB buffer and copies the requested part to dst
 * (the kernel refuses direct transfers into GPU-pinned host memory). On
 * error dst may be partly written.
 * Errors: AFX_E_INVALID_ARG (NULL path or dst, unknown flag, offset +
 * bytes above 2^63 - 1), AFX_E_UNSUPPORTED (the file system refuses
 * O_DIRECT), AFX_E_IO (open or read failed, or the file ends inside the
 * range), AFX_E_HOST_MEMORY (no bounce buffer for a direct read). */
int afx_file_read(const char *path, uint64_t offset, uint64_t bytes, void *dst, int threads, unsigned flags);

#ifdef __cplusplus
}
#endif

#endif /* AFX_H */
