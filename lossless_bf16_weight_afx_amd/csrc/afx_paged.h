// afx_paged.h -- checks and device helpers shared by the calls on a paged
// cache (afx_heads.hip, afx_attend.hip, afx_pages.hip).
#pragma once

#include <initializer_list>

#include "afx_internal.h"

namespace afx {

constexpr uint64_t kMaxRowStride = 1ull << 28;  // (2^23 rows of them stay far below 2^64 bytes)
constexpr uint32_t kMaxTokens = 1u << 23;       // new tokens of one call
constexpr uint32_t kMaxHeads = 1024;

inline bool page_size_ok(uint32_t n) { return n >= 16 && n <= 256 && (n & (n - 1)) == 0; }

inline bool aligned(std::initializer_list<const void *> ps, uintptr_t to) {
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
    return true;
}

inline int check_kv(const afx_kv_pages *kv) {
    if (!kv || !kv->k_dev || !kv->v_dev || kv->n_pages == 0 || kv->kv_heads == 0 || kv->kv_heads > kMaxHeads ||
        kv->head_dim == 0)
        return AFX_E_INVALID_ARG;
    if (kv->head_dim % 8 || kv->head_dim > AFX_MAX_HEAD_DIM || !page_size_ok(kv->page_tokens) ||
        (uint64_t)kv->n_pages * kv->page_tokens >= 1ull << 31)
        return AFX_E_UNSUPPORTED;
    return aligned({kv->k_dev, kv->v_dev}, 16) ? AFX_OK : AFX_E_MISALIGNED;
}
inline uint64_t kv_bytes(const afx_kv_pages *kv) {  // of the keys, and of the values
    return 2ull * kv->n_pages * kv->page_tokens * kv->kv_heads * kv->head_dim;
}

inline int check_table(const afx_page_table *t, bool refs) {
    if (!t || !t->table_dev || !t->len_dev || (refs && !t->refs_dev) || t->n_seqs == 0 || t->max_pages == 0 ||
        t->n_pages == 0 || t->table_stride < t->max_pages)
        return AFX_E_INVALID_ARG;
    if (!page_size_ok(t->page_tokens) || (uint64_t)t->n_pages * t->page_tokens >= 1ull << 31 ||
        (uint64_t)t->max_pages * t->page_tokens >= 1ull << 31 || t->n_seqs > 1u << 20 ||
        t->table_stride >= kMaxRowStride)
        return AFX_E_UNSUPPORTED;
    return aligned({t->table_dev, t->len_dev, t->refs_dev}, 4) ? AFX_OK : AFX_E_MISALIGNED;
}
inline RowSpan table_span(const afx_page_table *t) {
    return RowSpan{t->table_dev, t->n_seqs, 4ull * t->max_pages, 4ull * t->table_stride};
}
inline RowSpan flat(const void *p, uint64_t bytes) { return RowSpan{bytes ? p : nullptr, 1, bytes, bytes}; }

// Whether an output (the first n_out spans) shares a byte with any other.
inline bool outputs_overlap(const RowSpan *s, size_t n_out, size_t n) {
    for (size_t i = 0; i < n_out; ++i)
        for (size_t k = 0; k < n; ++k)
            if (i != k && s[i].p && s[k].p && rows_overlap(s[i], s[k])) return true;
    return false;
}

}  // namespace afx
