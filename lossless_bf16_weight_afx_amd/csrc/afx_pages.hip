// afx_pages.hip -- the pages of a paged cache (gfx950): sequences forked,
// trimmed and grown, live pages compacted, pages copied.
//
// The state (page tables, lengths, counts of holders) is the caller's and
// lives on the GPU; no call reads it on the host. What decides ids and grants
// is a matter of prefix sums over at most 1024 rows and over the counts of all
// pages, which one workgroup forms in fixed order, so that every run gives the
// same ids. Latency bounds it: one workgroup reads 16 KB of counts at a time
// with the next 16 KB on their way. The bytes of pages that have to be copied
// are moved by a second launch over all CUs, 16 bytes a lane and four loads in
// flight; memory bounds that (the live half of 80 planes moved to the front:
// 154 us, 5.0 TB/s read and written; the plan before it 5).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "afx_paged.h"

namespace afx {
namespace {

constexpr uint32_t kRowThreads = 256;    // threads that fork or trim a sequence
constexpr uint32_t kPlanThreads = 1024;  // threads of the workgroup that deals out pages
constexpr uint32_t kCopyThreads = 256;
constexpr uint32_t kCopyBlocks = 4096;  // workgroups of a launch that copies pages

// Device view of an afx_page_table.
struct Table {
    int32_t *table, *len, *refs;
    uint64_t stride;
    uint32_t n_seqs, max_pages, n_pages, shift;  // tokens of a page: 1 << shift

    __device__ uint32_t tokens(uint32_t s) const {  // a sequence's length, within what its pages could hold
        const int64_t most = (int64_t)max_pages << shift;
        return (uint32_t)min(max((int64_t)len[s], (int64_t)0), most);
    }
    __device__ uint32_t pages(uint32_t tokens) const { return (tokens + (1u << shift) - 1) >> shift; }
    __device__ bool holds(int32_t page) const { return (uint32_t)page < n_pages; }
};

// Device view of an afx_page_data, cut into units of a page's kUnit bytes.
struct Data {
    uint8_t *p;
    uint64_t page_bytes, plane_stride;
    uint32_t n_planes, units;  // units of a page
};
constexpr uint32_t kUnit = 16 * 1024;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// One unit of one plane's page, by the whole workgroup.
__device__ inline void copy_unit(const Data &d, uint32_t plane, uint32_t unit, uint32_t from, uint32_t to) {
    uint8_t *base = d.p + plane * d.plane_stride + (uint64_t)unit * kUnit;
    const u32x4 *src = reinterpret_cast<const u32x4 *>(base + from * d.page_bytes);
    u32x4 *dst = reinterpret_cast<u32x4 *>(base + to * d.page_bytes);
    const uint32_t n = (uint32_t)min((uint64_t)kUnit, d.page_bytes - (uint64_t)unit * kUnit) / 16;
    constexpr int kDeep = kUnit / 16 / kCopyThreads;
    u32x4 v[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
        if (threadIdx.x + i * kCopyThreads < n) v[i] = __builtin_nontemporal_load(src + threadIdx.x + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
        if (threadIdx.x + i * kCopyThreads < n)
            __builtin_nontemporal_store(v[i], dst + threadIdx.x + i * kCopyThreads);
}

__global__ __launch_bounds__(kRowThreads) void afx_pages_fork_kernel(Table t, uint32_t n, const int32_t *src,
                                                                     const int32_t *dst, int32_t *granted) {
    const uint32_t r = blockIdx.x;
    const uint32_t s = (uint32_t)src[r], d = (uint32_t)dst[r];
    bool bad = s >= t.n_seqs || d >= t.n_seqs;
    for (uint32_t i = threadIdx.x; i < n; i += kRowThreads) {
        const uint32_t to = (uint32_t)dst[i];
        bad |= to == s || (i < r && to == d);
    }
    if (!bad) bad = t.len[d] != 0;
    bad = __syncthreads_or(bad);
    if (granted && threadIdx.x == 0) granted[r] = !bad;
    if (bad) return;
    const uint32_t tokens = t.tokens(s), pages = t.pages(tokens);
    const int32_t *from = t.table + s * t.stride;
    int32_t *to = t.table + d * t.stride;
    for (uint32_t i = threadIdx.x; i < pages; i += kRowThreads) {
        const int32_t page = from[i];
        to[i] = page;
        if (t.holds(page)) atomicAdd(t.refs + page, 1);
    }
    if (threadIdx.x == 0) t.len[d] = (int32_t)tokens;
}

__global__ __launch_bounds__(kRowThreads) void afx_pages_trim_kernel(Table t, const int32_t *seqs,
                                                                     const int32_t *lens) {
    const uint32_t r = blockIdx.x, s = (uint32_t)seqs[r];
    bool skip = s >= t.n_seqs;
    for (uint32_t i = threadIdx.x; i < r; i += kRowThreads) skip |= (uint32_t)seqs[i] == s;
    skip = __syncthreads_or(skip);
    if (skip) return;
    const uint32_t had = t.tokens(s), keep = lens ? (uint32_t)max(lens[r], 0) : 0;
    __syncthreads();  // every thread has read the length
    if (keep >= had) return;
    int32_t *row = t.table + s * t.stride;
    for (uint32_t i = t.pages(keep) + threadIdx.x; i < t.pages(had); i += kRowThreads) {
        const int32_t page = row[i];
        row[i] = -1;
        if (t.holds(page)) atomicSub(t.refs + page, 1);
    }
    if (threadIdx.x == 0) t.len[s] = (int32_t)keep;
}

// Sum over the threads before this one (of their v), and over all in total.
template <class T>
__device__ inline T block_scan(T v, T &total) {
    __shared__ T waves[kPlanThreads / 64];
    const uint32_t lane = threadIdx.x % 64, w = threadIdx.x / 64;
    T sum = v;
#pragma unroll
    for (uint32_t o = 1; o < 64; o *= 2) {
        const T left = __shfl_up(sum, o);
        if (lane >= o) sum += left;
    }
    __syncthreads();  // (the last scan's sums have been read)
    if (lane == 63) waves[w] = sum;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (uint32_t i = 0; i < kPlanThreads / 64; ++i) {
        before += i < w ? waves[i] : 0;
        total += waves[i];
    }
    return before + sum - v;
}

// The counts of pages 4 tid .. 4 tid + 3 of the block of 4096 pages at `at`;
// those that are not there count as `rest`.
constexpr uint32_t kPlanPages = 4 * kPlanThreads;
struct Counts {
    int32_t c[4];
    __device__ void load(const Table &t, uint32_t at, uint32_t end, int32_t rest) {
        const uint32_t i = at + 4 * threadIdx.x;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) c[k] = i + k < end && i + k >= at ? t.refs[i + k] : rest;
    }
};

// What extend decides for a row.
struct Grant {
    int32_t had;    // tokens before
    int32_t grow;   // tokens granted, -1 for a refused row
    int32_t first;  // of its new pages in the list of ids
    int32_t copied; // page whose copy is the first of them, or -1
};

__global__ __launch_bounds__(kPlanThreads) void afx_pages_deal_kernel(Table t, uint32_t n, const int32_t *seqs,
                                                                      const int32_t *starts, uint32_t m,
                                                                      int32_t *granted, Grant *grants, int32_t *ids) {
    __shared__ int32_t seq[kPlanThreads], last[kPlanThreads];
    const uint32_t r = threadIdx.x, size = 1u << t.shift;
    const uint32_t s = r < n ? (uint32_t)seqs[r] : ~0u;
    uint32_t had = 0, grow = 0;
    bool ok = s < t.n_seqs;
    if (ok) {
        const uint32_t a = (uint32_t)min(max(starts[r], 0), (int32_t)m);
        const uint32_t b = (uint32_t)min(max(starts[r + 1], 0), (int32_t)m);
        grow = b > a ? b - a : 0;
        had = t.tokens(s);
        ok = (uint64_t)had + grow <= (uint64_t)t.max_pages << t.shift;
    }
    seq[r] = r < n ? (int32_t)s : -1;
    __syncthreads();
    for (uint32_t i = 0; i < n; ++i) ok &= !(i < r && seq[i] == (int32_t)s);
    int32_t page = -1, holders = 0;  // the partly filled last page
    if (ok && grow && had % size) {
        page = t.table[s * t.stride + had / size];
        if (t.holds(page))
            holders = t.refs[page];
        else
            page = -1;
    }
    last[r] = page;
    __syncthreads();
    if (page >= 0)
        for (uint32_t i = 0; i < r; ++i) holders -= last[i] == page;
    const bool copy = holders > 1;
    const uint32_t need = ok ? t.pages(had + grow) - t.pages(had) + copy : 0;
    uint64_t total;
    const uint64_t before = block_scan<uint64_t>(need, total);
    // the ids of the first `total` free pages
    uint32_t found = 0;
    Counts now, next;
    now.load(t, 0, t.n_pages, 1);
    for (uint64_t at = 0; at < t.n_pages && found < total; at += kPlanPages) {
        if (at + kPlanPages < t.n_pages) next.load(t, (uint32_t)at + kPlanPages, t.n_pages, 1);
        uint32_t mine = 0, all;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mine += now.c[k] == 0;
        uint32_t to = found + block_scan<uint32_t>(mine, all);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
            if (now.c[k] == 0) ids[to++] = (int32_t)(at + 4 * threadIdx.x + k);
        found += all;
        now = next;
    }
    __syncthreads();  // the counts have been read
    if (r >= n) return;
    ok &= before + need <= found;
    grants[r] = Grant{(int32_t)had, ok ? (int32_t)grow : -1, (int32_t)(ok ? before : 0), ok && copy ? page : -1};
    if (granted) granted[r] = ok ? (int32_t)grow : 0;
    if (ok) {
        t.len[s] = (int32_t)(had + grow);
        if (copy) atomicSub(t.refs + page, 1);
    }
}

// Workgroup (r, 0) writes row r's new pages and its tokens' slots, the others
// of row r copy its page.
__global__ __launch_bounds__(kCopyThreads) void afx_pages_grow_kernel(Table t, Data d, uint32_t n,
                                                                      const int32_t *seqs, const int32_t *starts,
                                                                      uint32_t m, int32_t *slots, int32_t *pos,
                                                                      const Grant *grants, const int32_t *ids) {
    const uint32_t r = blockIdx.x, size = 1u << t.shift;
    const Grant g = grants[r];
    if (blockIdx.y) {
        if (g.copied < 0) return;
        const uint32_t to = (uint32_t)ids[g.first];
        const uint64_t all = (uint64_t)d.n_planes * d.units;
        for (uint64_t u = blockIdx.y - 1; u < all; u += gridDim.y - 1)
            copy_unit(d, (uint32_t)(u / d.units), (uint32_t)(u % d.units), (uint32_t)g.copied, to);
        return;
    }
    const uint32_t a = (uint32_t)min(max(starts[r], 0), (int32_t)m);
    const uint32_t b = (uint32_t)min(max(starts[r + 1], 0), (int32_t)m);
    auto none = [&](uint32_t from, uint32_t to) {
        for (uint32_t i = from + threadIdx.x; i < to; i += kCopyThreads) {
            slots[i] = -1;
            if (pos) pos[i] = 0;
        }
    };
    if (r == 0) {  // tokens of no row
        none(0, a);
        none((uint32_t)min(max(starts[n], 0), (int32_t)m), m);
    }
    if (g.grow < 0) {
        none(a, b);
        return;
    }
    int32_t *row = t.table + (uint64_t)(uint32_t)seqs[r] * t.stride;
    const uint32_t had = (uint32_t)g.had, first = t.pages(had) - (g.copied >= 0), end = t.pages(had + g.grow);
    const int32_t kept = had % size && g.copied < 0 ? row[had / size] : -1;
    for (uint32_t i = first + threadIdx.x; i < end; i += kCopyThreads) {
        const int32_t id = ids[g.first + i - first];
        row[i] = id;
        t.refs[id] = 1;
    }
    for (uint32_t i = threadIdx.x; i < (uint32_t)g.grow; i += kCopyThreads) {
        const uint32_t at = had + i, page = at / size;
        const int32_t id = page >= first ? ids[g.first + page - first] : kept;
        slots[a + i] = t.holds(id) ? (int32_t)(id * size + at % size) : -1;
        if (pos) pos[a + i] = (int32_t)at;
    }
}

// Pages above the live ones' number move down: map, counts and the list of
// moves (moves[0]: how many, then from and to of each).
__global__ __launch_bounds__(kPlanThreads) void afx_pages_plan_kernel(Table t, int32_t *map, int32_t *live,
                                                                      int32_t *moves) {
    uint32_t n_live = 0, all;
    Counts now;
    for (uint64_t at = 0; at < t.n_pages; at += kPlanPages) {
        now.load(t, (uint32_t)at, t.n_pages, 0);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) n_live += now.c[k] > 0;
    }
    block_scan<uint32_t>(n_live, all);
    n_live = all;
    int32_t *pairs = moves + 2;
    uint32_t found = 0;
    for (uint64_t at = 0; at < n_live; at += kPlanPages) {
        now.load(t, (uint32_t)at, n_live, 1);
        uint32_t mine = 0;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mine += now.c[k] <= 0;
        uint32_t to = found + block_scan<uint32_t>(mine, all);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t i = (uint32_t)at + 4 * threadIdx.x + k;
            if (i >= n_live) break;
            map[i] = now.c[k] > 0 ? (int32_t)i : -1;
            if (now.c[k] <= 0) pairs[2 * to++ + 1] = (int32_t)i;
        }
        found += all;
    }
    __syncthreads();  // the list of free pages is whole
    found = 0;
    for (uint64_t at = n_live; at < t.n_pages; at += kPlanPages) {
        now.load(t, (uint32_t)at, t.n_pages, 0);
        uint32_t mine = 0;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mine += now.c[k] > 0;
        uint32_t from = found + block_scan<uint32_t>(mine, all);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint64_t i = at + 4 * threadIdx.x + k;
            if (i >= t.n_pages) break;
            int32_t to = -1;
            if (now.c[k] > 0) {
                to = pairs[2 * from + 1];
                pairs[2 * from++] = (int32_t)i;
                t.refs[to] = now.c[k];
                t.refs[i] = 0;
            }
            map[i] = to;
        }
        found += all;
    }
    if (threadIdx.x == 0) {
        moves[0] = (int32_t)found;
        if (live) *live = (int32_t)n_live;
    }
}

// Copies every moved page, and follows the map in the tables.
__global__ __launch_bounds__(kCopyThreads) void afx_pages_move_kernel(Table t, Data d, const int32_t *map,
                                                                      const int32_t *moves) {
    const uint64_t each = (uint64_t)d.n_planes * d.units, all = each * (uint32_t)moves[0];
    for (uint64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const uint64_t i = u / each, part = u % each;
        copy_unit(d, (uint32_t)(part / d.units), (uint32_t)(part % d.units), (uint32_t)moves[2 + 2 * i],
                  (uint32_t)moves[3 + 2 * i]);
    }
    const uint64_t entries = (uint64_t)t.n_seqs * t.max_pages;
    for (uint64_t i = (uint64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < entries;
         i += (uint64_t)gridDim.x * kCopyThreads) {
        int32_t *e = t.table + i / t.max_pages * t.stride + i % t.max_pages;
        if (t.holds(*e)) *e = map[*e];
    }
}

__global__ __launch_bounds__(kCopyThreads) void afx_pages_copy_kernel(Data d, uint32_t n_pages, uint32_t n,
                                                                      const int32_t *src, const int32_t *dst) {
    const uint64_t each = (uint64_t)d.n_planes * d.units, all = each * n;
    for (uint64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const uint64_t i = u / each, part = u % each;
        const uint32_t from = (uint32_t)src[i], to = (uint32_t)dst[i];
        if (from < n_pages && to < n_pages && from != to)
            copy_unit(d, (uint32_t)(part / d.units), (uint32_t)(part % d.units), from, to);
    }
}

// ---- argument checks ---------------------------------------------------------
Table view(const afx_page_table *t) {
    return Table{t->table_dev, t->len_dev,   t->refs_dev, t->table_stride,
                 t->n_seqs,    t->max_pages, t->n_pages,  (uint32_t)__builtin_ctz(t->page_tokens)};
}
Data view(const afx_page_data *d) {
    return Data{static_cast<uint8_t *>(d->data_dev), d->page_bytes, d->plane_stride, d->n_planes,
                (uint32_t)((d->page_bytes + kUnit - 1) / kUnit)};
}

int check_data(const afx_page_data *d, uint64_t n_pages) {
    if (!d || !d->data_dev || d->page_bytes == 0 || d->n_planes == 0 || n_pages == 0) return AFX_E_INVALID_ARG;
    if (d->page_bytes > 1ull << 30 || d->n_planes > 65535 || d->page_bytes % 16 || d->plane_stride % 16 ||
        d->plane_stride >= 1ull << 46)
        return AFX_E_UNSUPPORTED;
    if (d->plane_stride < n_pages * d->page_bytes) return AFX_E_INVALID_ARG;
    return aligned({d->data_dev}, 16) ? AFX_OK : AFX_E_MISALIGNED;
}
RowSpan data_span(const afx_page_data *d, uint64_t n_pages) {
    return RowSpan{d->data_dev, d->n_planes, n_pages * d->page_bytes, d->plane_stride};
}

// Workgroups that copy `pages` pages' units.
uint32_t copy_blocks(const Data &d, uint64_t pages) {
    return (uint32_t)std::min<uint64_t>(pages * d.n_planes * d.units, kCopyBlocks);
}

template <class... A>
int launch(const void *fn, dim3 grid, uint32_t threads, void *stream, A... a) {
    void *args[] = {&a...};
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, static_cast<hipStream_t>(stream)) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}
template <class F>
const void *kernel(F *f) {
    return reinterpret_cast<const void *>(f);
}

uint64_t extend_space(const afx_page_table *t, uint32_t n) { return (uint64_t)n * sizeof(Grant) + 4ull * t->n_pages; }
uint64_t compact_space(const afx_page_table *t) { return 4 * (2ull + 2ull * t->n_pages); }

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_pages_fork_async(const afx_page_table *t, uint32_t n, const int32_t *src_dev, const int32_t *dst_dev,
                         int32_t *granted_dev, void *stream) {
    const int rc = check_table(t, true);
    if (rc != AFX_OK) return rc;
    if (n > AFX_MAX_PAGE_ROWS) return AFX_E_UNSUPPORTED;
    if (n == 0) return AFX_OK;
    if (!src_dev || !dst_dev) return AFX_E_INVALID_ARG;
    if (!aligned({src_dev, dst_dev, granted_dev}, 4)) return AFX_E_MISALIGNED;
    const RowSpan s[] = {table_span(t),           flat(t->len_dev, 4ull * t->n_seqs), flat(t->refs_dev, 4ull * t->n_pages),
                         flat(granted_dev, 4ull * n), flat(src_dev, 4ull * n),            flat(dst_dev, 4ull * n)};
    if (outputs_overlap(s, 4, 6)) return AFX_E_INVALID_ARG;
    return launch(kernel(&afx_pages_fork_kernel), dim3(n), kRowThreads, stream, view(t), n, src_dev, dst_dev,
                  granted_dev);
}

int afx_pages_trim_async(const afx_page_table *t, uint32_t n, const int32_t *seqs_dev, const int32_t *lens_dev,
                         void *stream) {
    const int rc = check_table(t, true);
    if (rc != AFX_OK) return rc;
    if (n > AFX_MAX_PAGE_ROWS) return AFX_E_UNSUPPORTED;
    if (n == 0) return AFX_OK;
    if (!seqs_dev) return AFX_E_INVALID_ARG;
    if (!aligned({seqs_dev, lens_dev}, 4)) return AFX_E_MISALIGNED;
    const RowSpan s[] = {table_span(t), flat(t->len_dev, 4ull * t->n_seqs), flat(t->refs_dev, 4ull * t->n_pages),
                         flat(seqs_dev, 4ull * n), flat(lens_dev, 4ull * n)};
    if (outputs_overlap(s, 3, 5)) return AFX_E_INVALID_ARG;
    return launch(kernel(&afx_pages_trim_kernel), dim3(n), kRowThreads, stream, view(t), seqs_dev, lens_dev);
}

int afx_pages_extend_workspace(const afx_page_table *t, uint32_t n, size_t *bytes) {
    const int rc = check_table(t, true);
    if (rc != AFX_OK) return rc;
    if (!bytes) return AFX_E_INVALID_ARG;
    if (n > AFX_MAX_PAGE_ROWS) return AFX_E_UNSUPPORTED;
    *bytes = extend_space(t, n);
    return AFX_OK;
}

int afx_pages_extend_async(const afx_page_table *t, const afx_page_data *d, uint32_t n, const int32_t *seqs_dev,
                           const int32_t *starts_dev, uint32_t m, int32_t *slots_dev, int32_t *pos_dev,
                           int32_t *granted_dev, void *ws_dev, size_t ws_bytes, void *stream) {
    int rc = check_table(t, true);
    if (rc == AFX_OK) rc = check_data(d, t->n_pages);
    if (rc != AFX_OK) return rc;
    if (n > AFX_MAX_PAGE_ROWS || m > kMaxTokens) return AFX_E_UNSUPPORTED;
    if (n == 0) return m ? AFX_E_INVALID_ARG : AFX_OK;
    if (!seqs_dev || !starts_dev || (m && !slots_dev) || !ws_dev) return AFX_E_INVALID_ARG;
    if (!aligned({seqs_dev, starts_dev, slots_dev, pos_dev, granted_dev}, 4) || !aligned({ws_dev}, 16))
        return AFX_E_MISALIGNED;
    const uint64_t need = extend_space(t, n);
    const RowSpan s[] = {table_span(t),
                         flat(t->len_dev, 4ull * t->n_seqs),
                         flat(t->refs_dev, 4ull * t->n_pages),
                         data_span(d, t->n_pages),
                         flat(slots_dev, 4ull * m),
                         flat(pos_dev, 4ull * m),
                         flat(granted_dev, 4ull * n),
                         flat(ws_dev, need),
                         flat(seqs_dev, 4ull * n),
                         flat(starts_dev, 4ull * n + 4)};
    if (outputs_overlap(s, 8, 10)) return AFX_E_INVALID_ARG;
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
    Grant *grants = static_cast<Grant *>(ws_dev);
    int32_t *ids = reinterpret_cast<int32_t *>(grants + n);
    rc = launch(kernel(&afx_pages_deal_kernel), dim3(1), kPlanThreads, stream, view(t), n, seqs_dev, starts_dev, m,
                granted_dev, grants, ids);
    if (rc != AFX_OK) return rc;
    const Data data = view(d);
    const uint32_t each = std::max(1u, (copy_blocks(data, n) + n - 1) / n);
    return launch(kernel(&afx_pages_grow_kernel), dim3(n, 1 + each), kCopyThreads, stream, view(t), data, n, seqs_dev,
                  starts_dev, m, slots_dev, pos_dev, (const Grant *)grants, (const int32_t *)ids);
}

int afx_pages_compact_workspace(const afx_page_table *t, size_t *bytes) {
    const int rc = check_table(t, true);
    if (rc != AFX_OK) return rc;
    if (!bytes) return AFX_E_INVALID_ARG;
    *bytes = compact_space(t);
    return AFX_OK;
}

int afx_pages_compact_async(const afx_page_table *t, const afx_page_data *d, int32_t *map_dev, int32_t *live_dev,
                            void *ws_dev, size_t ws_bytes, void *stream) {
    int rc = check_table(t, true);
    if (rc == AFX_OK) rc = check_data(d, t->n_pages);
    if (rc != AFX_OK) return rc;
    if (!map_dev || !ws_dev) return AFX_E_INVALID_ARG;
    if (!aligned({map_dev, live_dev}, 4) || !aligned({ws_dev}, 16)) return AFX_E_MISALIGNED;
    const uint64_t need = compact_space(t);
    const RowSpan s[] = {table_span(t),
                         flat(t->len_dev, 4ull * t->n_seqs),
                         flat(t->refs_dev, 4ull * t->n_pages),
                         data_span(d, t->n_pages),
                         flat(map_dev, 4ull * t->n_pages),
                         flat(live_dev, 4),
                         flat(ws_dev, need)};
    if (outputs_overlap(s, 7, 7)) return AFX_E_INVALID_ARG;
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
    int32_t *moves = static_cast<int32_t *>(ws_dev);
    rc = launch(kernel(&afx_pages_plan_kernel), dim3(1), kPlanThreads, stream, view(t), map_dev, live_dev, moves);
    if (rc != AFX_OK) return rc;
    const Data data = view(d);
    return launch(kernel(&afx_pages_move_kernel), dim3(copy_blocks(data, t->n_pages)), kCopyThreads, stream, view(t),
                  data, (const int32_t *)map_dev, (const int32_t *)moves);
}

int afx_pages_copy_async(const afx_page_data *d, uint32_t n_pages, uint32_t n, const int32_t *src_dev,
                         const int32_t *dst_dev, void *stream) {
    const int rc = check_data(d, n_pages);
    if (rc != AFX_OK) return rc;
    if (n == 0) return AFX_OK;
    if (!src_dev || !dst_dev) return AFX_E_INVALID_ARG;
    if (!aligned({src_dev, dst_dev}, 4)) return AFX_E_MISALIGNED;
    const RowSpan s[] = {data_span(d, n_pages), flat(src_dev, 4ull * n), flat(dst_dev, 4ull * n)};
    if (outputs_overlap(s, 1, 3)) return AFX_E_INVALID_ARG;
    const Data data = view(d);
    return launch(kernel(&afx_pages_copy_kernel), dim3(copy_blocks(data, n)), kCopyThreads, stream, data, n_pages, n,
                  src_dev, dst_dev);
}

}  // extern "C"
