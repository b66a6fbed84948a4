// afx_attend.hip -- attention of new tokens over a paged cache (gfx950).
//
//   o = sum_j e^(s_j - M) v_j / sum_j e^(s_j - M),  s_j = scale q k_j,
//   lse = M + ln sum_j e^(s_j - M)
// over the positions j that the query sees; M is the running maximum of one
// pass over them.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "afx_paged.h"

namespace afx {
namespace {

constexpr uint32_t kMaxRows = 1u << 16, kMaxGroup = 256;

struct AttendArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    const int32_t *table, *len, *seqs, *starts;
    uint64_t q_stride, out_stride, table_stride;
    uint32_t m, n_rows, n_seqs, max_pages, n_pages, page_shift, q_heads, kv_heads, group, d, causal, window;
    float scale;
};

__device__ inline float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// A batch row's sequence, its new tokens and its length.
struct Row {
    uint32_t seq, from, n, len;  // n == 0: nothing to do
    __device__ Row(const AttendArgs &a, uint32_t r) {
        seq = a.seqs ? (uint32_t)a.seqs[r] : r;
        from = (uint32_t)min(max(a.starts[r], 0), (int32_t)a.m);
        const uint32_t to = (uint32_t)min(max(a.starts[r + 1], 0), (int32_t)a.m);
        n = to > from ? to - from : 0;
        len = seq < a.n_seqs ? (uint32_t)min((int64_t)max(a.len[seq], 0), (int64_t)a.max_pages << a.page_shift) : 0;
    }
};

__global__ __launch_bounds__(64) void afx_attend_kernel(AttendArgs a) {
    __shared__ float q[AFX_MAX_HEAD_DIM], p[64];
    __shared__ int32_t ids[64];
    const uint32_t t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, size = 1u << a.page_shift;
    uint32_t lo = 0, hi = a.n_rows;  // the last row that starts at t or before
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.starts[mid] <= (int32_t)t) lo = mid; else hi = mid;
    }
    const Row row(a, lo);
    if (t < row.from || t >= row.from + row.n) return;
    const int64_t at = (int64_t)row.len - row.n + (t - row.from);
    const int64_t end = a.causal ? min(at + 1, (int64_t)row.len) : (int64_t)row.len;
    const int64_t begin = a.window ? max(at - (int64_t)a.window + 1, (int64_t)0) : 0;
    for (uint32_t i = lane; i < a.d; i += 64) q[i] = from_bf16(a.q[t * a.q_stride + h * a.d + i]) * a.scale;
    __syncthreads();
    const uint64_t head = (uint64_t)(h / a.group) * size * a.d, page_elems = (uint64_t)size * a.kv_heads * a.d;
    const int32_t *table = a.table + row.seq * a.table_stride;
    float top = -INFINITY, sum = 0.f, o[4] = {};
    for (int64_t j0 = begin; j0 < end; j0 += 64) {
        const uint32_t j = (uint32_t)j0 + lane;
        const uint32_t id = j < end ? (uint32_t)table[j / size] : ~0u;
        const bool seen = id < a.n_pages;
        float s = -INFINITY;
        if (seen) {
            s = 0.f;
            const uint16_t *k = a.k + id * page_elems + head + j % size * 8;
            for (uint32_t c = 0; c < a.d; ++c) s += q[c] * from_bf16(k[c / 8 * size * 8 + c % 8]);
        }
        float best = s;
        for (int x = 1; x < 64; x *= 2) best = fmaxf(best, __shfl_xor(best, x));
        const float now = fmaxf(top, best), base = now == -INFINITY ? 0.f : now;
        const float old = __expf(top - base);
        __syncthreads();
        p[lane] = seen ? __expf(s - base) : 0.f;
        ids[lane] = seen ? (int32_t)id : -1;
        float part = p[lane];
        for (int x = 1; x < 64; x *= 2) part += __shfl_xor(part, x);
        sum = sum * old + part;
        top = now;
        __syncthreads();
        for (int e = 0; e < 4; ++e) {
            const uint32_t c = lane + 64 * e;
            if (c >= a.d) break;
            o[e] *= old;
            for (uint32_t i = 0; i < 64; ++i) {
                if (ids[i] < 0) continue;
                const uint32_t off = ((uint32_t)j0 + i) % size;
                o[e] += p[i] * from_bf16(a.v[(uint32_t)ids[i] * page_elems + head + ((off & ~7u) * a.d) + c * 8 + off % 8]);
            }
        }
    }
    for (int e = 0; e < 4; ++e) {
        const uint32_t c = lane + 64 * e;
        if (c < a.d)
            a.out[t * a.out_stride + h * a.d + c] = __builtin_bit_cast(uint16_t, (__bf16)(sum == 0.f ? 0.f : o[e] / sum));
    }
    if (a.lse && lane == 0) a.lse[(uint64_t)t * a.q_heads + h] = sum == 0.f ? -INFINITY : top + __logf(sum);
}

int check_attend(const afx_attend *p, const afx_kv_pages *kv, uint32_t n_rows, uint32_t m) {
    const int rc = check_kv(kv);
    if (rc != AFX_OK) return rc;
    if (!p || p->q_heads == 0 || p->q_heads % kv->kv_heads || p->q_heads / kv->kv_heads > kMaxGroup ||
        !std::isfinite(p->scale))
        return AFX_E_INVALID_ARG;
    return n_rows > kMaxRows || m > kMaxTokens ? AFX_E_UNSUPPORTED : AFX_OK;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_attend_workspace(const afx_attend *p, const afx_kv_pages *kv, uint32_t n_rows, uint32_t m, size_t *bytes) {
    const int rc = check_attend(p, kv, n_rows, m);
    if (rc != AFX_OK) return rc;
    if (!bytes) return AFX_E_INVALID_ARG;
    *bytes = 0;
    return AFX_OK;
}

int afx_attend_async(const afx_attend *p, const afx_kv_pages *kv, const afx_page_table *t, uint32_t n_rows,
                     const int32_t *seqs_dev, const int32_t *starts_dev, uint32_t m, const uint16_t *q_dev,
                     uint64_t q_stride, uint16_t *out_dev, uint64_t out_stride, float *lse_dev, void *ws_dev,
                     size_t ws_bytes, void *stream) {
    int rc = check_attend(p, kv, n_rows, m);
    if (rc == AFX_OK) rc = check_table(t, false);
    if (rc != AFX_OK) return rc;
    if (t->n_pages != kv->n_pages || t->page_tokens != kv->page_tokens) return AFX_E_INVALID_ARG;
    if (m == 0 || n_rows == 0) return AFX_OK;
    const uint64_t width = (uint64_t)p->q_heads * kv->head_dim;
    if (!starts_dev || !q_dev || !out_dev || q_stride < width || out_stride < width || (!seqs_dev && n_rows > t->n_seqs))
        return AFX_E_INVALID_ARG;
    if (q_stride >= kMaxRowStride || out_stride >= kMaxRowStride) return AFX_E_UNSUPPORTED;
    if (q_stride % 8 || out_stride % 8 || !aligned({q_dev, out_dev}, 16) || !aligned({seqs_dev, starts_dev, lse_dev}, 4))
        return AFX_E_MISALIGNED;
    const RowSpan s[] = {RowSpan{out_dev, m, 2 * width, 2 * out_stride},
                         flat(lse_dev, 4ull * m * p->q_heads),
                         RowSpan{q_dev, m, 2 * width, 2 * q_stride},
                         flat(kv->k_dev, kv_bytes(kv)),
                         flat(kv->v_dev, kv_bytes(kv)),
                         table_span(t),
                         flat(t->len_dev, 4ull * t->n_seqs),
                         flat(seqs_dev, 4ull * n_rows),
                         flat(starts_dev, 4ull * n_rows + 4)};
    if (outputs_overlap(s, 2, 9)) return AFX_E_INVALID_ARG;
    AttendArgs a{};
    a.q = q_dev;
    a.k = kv->k_dev;
    a.v = kv->v_dev;
    a.out = out_dev;
    a.lse = lse_dev;
    a.table = t->table_dev;
    a.len = t->len_dev;
    a.seqs = seqs_dev;
    a.starts = starts_dev;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.table_stride = t->table_stride;
    a.m = m;
    a.n_rows = n_rows;
    a.n_seqs = t->n_seqs;
    a.max_pages = t->max_pages;
    a.n_pages = t->n_pages;
    a.page_shift = (uint32_t)__builtin_ctz(t->page_tokens);
    a.q_heads = p->q_heads;
    a.kv_heads = kv->kv_heads;
    a.group = p->q_heads / kv->kv_heads;
    a.d = kv->head_dim;
    a.causal = p->causal;
    a.window = p->window;
    a.scale = p->scale;
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_attend_kernel), dim3(m, p->q_heads), dim3(64), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

}  // extern "C"
