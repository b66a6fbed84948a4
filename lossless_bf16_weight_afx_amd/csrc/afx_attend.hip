// afx_attend.hip -- attention of new tokens over a paged cache (gfx950): entry
// points, the division of the work, and the join of parts.
//
//   o = sum_j e^(s_j - M) v_j / sum_j e^(s_j - M),  s_j = scale q k_j,
//   lse = M + ln sum_j e^(s_j - M)
// over the positions j that the query sees; M is the running maximum of one
// pass over them. Batch rows of a few query rows a head go to
// afx_attend_few.hip, which memory bounds, the others to
// afx_attend_many.hip, which the matrix cores bound. Where there are too few
// workgroups to fill the card, tokens are cut into parts, whose sums (FP32) a
// last launch joins: with M the largest of the parts' M_i,
//   o = sum_i 2^(M_i - M) o_i / sum_i 2^(M_i - M) l_i.
// A part whose factor has become 0 is added too: an infinity or NaN in it that
// the query sees shows (0 times it is NaN), as it does beside the largest
// score in one part.
#include <algorithm>
#include <cmath>

#include "afx_attend.h"

namespace afx {
namespace {

constexpr uint32_t kMaxRows = 1u << 16, kMaxGroup = 256;
constexpr uint32_t kJoinThreads = 256;
constexpr uint32_t kTeamParts = 16;  // parts that a team of d / 4 lanes joins by itself
constexpr float kLog2e = 1.4426950408889634f;

// The parts of one query row of a batch row that the kernel for few rows took,
// by a workgroup: teams of d / 4 lanes add up every n-th part, then the teams.
__global__ __launch_bounds__(kJoinThreads) void afx_attend_join_few_kernel(AttendArgs a) {
    __shared__ float weight[kMaxSplits];
    __shared__ f32x4 sums[kJoinThreads];
    __shared__ float tops[kJoinThreads / 64], totals[kJoinThreads / 64];
    const uint32_t rr = blockIdx.x % a.few_rows, kvh = blockIdx.x / a.few_rows % a.kv_heads;
    const uint32_t r = blockIdx.x / a.few_rows / a.kv_heads;
    const BatchRow row(a, r);
    if (rr >= row.n * a.group || row.n * a.group > a.few_rows) return;
    const uint32_t n = FewRange(a, row).splits;
    if (n == 1) return;
    const uint64_t p = (uint64_t)blockIdx.x * a.few_splits;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const float2 ml = threadIdx.x < n ? a.few_ml[p + threadIdx.x] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
    weight[threadIdx.x] = f;
    float sum = f * ml.y;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) sum += __shfl_xor(sum, o);
    if (lane == 0) totals[wave] = sum;
    __syncthreads();
    sum = (totals[0] + totals[1]) + (totals[2] + totals[3]);
    const uint32_t quads = a.d / 4, teams = kJoinThreads / quads, team = threadIdx.x / quads, quad = threadIdx.x % quads;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if (team < teams) {
#pragma unroll 4
        for (uint32_t i = team; i < n; i += teams) {
            const float w = weight[i];
            o += w * *reinterpret_cast<const f32x4 *>(a.few_o + (p + i) * a.d + 4 * quad);
        }
    }
    sums[threadIdx.x] = o;
    __syncthreads();
    if (team) return;
    for (uint32_t i = 1; i < teams; ++i) o += sums[i * quads + quad];
    const float k = sum == 0.f ? 0.f : 1.f / sum;
    if (sum == 0.f) o = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint64_t t = row.from + rr / a.group;
    const uint32_t h = kvh * a.group + rr % a.group;
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + h * a.d + 4 * quad) =
        make_uint2(pack2(o[0] * k, o[1] * k), pack2(o[2] * k, o[3] * k));
    if (a.lse && quad == 0) a.lse[t * a.q_heads + h] = lse_of(top, sum);
}

// One query row's parts p .. p + n - 1, by a team of d / 4 lanes that hold 4
// values each: one pass, 8 parts' loads at a time in flight.
__device__ inline void join_row(const AttendArgs &a, const float *po, const float2 *pml, uint64_t p, uint32_t n,
                                uint32_t quad, uint64_t t, uint32_t h) {
    constexpr uint32_t kAtOnce = 8;
    float top = -INFINITY, sum = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t i0 = 0; i0 < n; i0 += kAtOnce) {
        float2 ml[kAtOnce];
        f32x4 v[kAtOnce];
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) {
            const uint64_t at = p + min(i0 + i, n - 1);
            ml[i] = pml[at];
            v[i] = *reinterpret_cast<const f32x4 *>(po + at * a.d + 4 * quad);
        }
        float now = top;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) now = fmaxf(now, ml[i].x);
        const float base = now == -INFINITY ? 0.f : now, old = exp2_fast(top - base);
        top = now;
        sum *= old;
        o *= old;
#pragma unroll
        for (uint32_t i = 0; i < kAtOnce; ++i) {
            const bool once = i0 + i < n;  // (behind the last part it is loaded again)
            const float w = once && ml[i].x != -INFINITY ? exp2_fast(ml[i].x - base) : 0.f;
            sum += w * (once ? ml[i].y : 0.f);
            o += w * (once ? v[i] : f32x4{0.f, 0.f, 0.f, 0.f});
        }
    }
    const float k = sum == 0.f ? 0.f : 1.f / sum;
    if (sum == 0.f) o = f32x4{0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + h * a.d + 4 * quad) =
        make_uint2(pack2(o[0] * k, o[1] * k), pack2(o[2] * k, o[3] * k));
    if (a.lse && quad == 0) a.lse[t * a.q_heads + h] = lse_of(top, sum);
}

// Up to kTeamParts parts of the query rows that the kernel for few rows took, a team a row.
__global__ __launch_bounds__(kJoinThreads) void afx_attend_join_teams_kernel(AttendArgs a) {
    const uint32_t quads = a.d / 4, teams = kJoinThreads / quads;
    const uint32_t team = threadIdx.x / quads, quad = threadIdx.x % quads;
    const uint64_t at = (uint64_t)blockIdx.x * teams + team;
    if (team >= teams || at >= (uint64_t)a.n_rows * a.kv_heads * a.few_rows) return;
    const uint32_t rr = (uint32_t)(at % a.few_rows), kvh = (uint32_t)(at / a.few_rows % a.kv_heads);
    const BatchRow row(a, (uint32_t)(at / a.few_rows / a.kv_heads));
    if (rr >= row.n * a.group || row.n * a.group > a.few_rows) return;
    const uint32_t n = FewRange(a, row).splits;
    if (n > 1) join_row(a, a.few_o, a.few_ml, at * a.few_splits, n, quad, row.from + rr / a.group, kvh * a.group + rr % a.group);
}

// The parts of query rows that the kernel for many rows took, a team per token and head.
__global__ __launch_bounds__(kJoinThreads) void afx_attend_join_many_kernel(AttendArgs a) {
    const uint32_t quads = a.d / 4, teams = kJoinThreads / quads;
    const uint32_t team = threadIdx.x / quads, quad = threadIdx.x % quads;
    const uint64_t at = (uint64_t)blockIdx.x * teams + team;
    if (team >= teams || at >= (uint64_t)a.m * a.q_heads) return;
    const uint32_t t = (uint32_t)(at / a.q_heads), h = (uint32_t)(at % a.q_heads);
    uint32_t lo = 0, hi = a.n_rows;  // the last batch row that starts at t or before
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.starts[mid] <= (int32_t)t) lo = mid; else hi = mid;
    }
    const BatchRow row(a, lo);
    if (t < row.from || t >= row.from + row.n || row.n * a.group <= a.few_rows) return;
    join_row(a, a.many_o, a.many_ml, at * a.many_splits, a.many_splits, quad, t, h);
}

// ---- the division of the work --------------------------------------------------
uint64_t up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

struct Plan {
    uint32_t few_rows, few_part, few_splits, many_tiles, many_splits;
    uint64_t few_sums, many_sums;  // rows of sums of parts
    uint64_t bytes(uint32_t d) const { return (few_sums + many_sums) * 4ull * (d + 2); }
};

// Depends on the parameters and sizes only, as the order of the sums does.
Plan plan(const afx_attend *p, const afx_kv_pages *kv, uint32_t n_rows, uint32_t m) {
    Plan s{};
    const uint32_t group = p->q_heads / kv->kv_heads;
    const uint64_t most = std::max<uint64_t>(1, std::min(p->max_new, m));  // new tokens of a sequence
    uint64_t tokens = std::min(std::max<uint64_t>(1, p->max_len), kMaxPositions);  // that its queries see
    if (p->window) tokens = std::min<uint64_t>(tokens, (p->causal ? 0 : tokens) + p->window + most);
    const bool few = most * group <= 32, many = !few;
    s.few_rows = few ? (uint32_t)(most * group) : n_rows > 1 ? 32 : 0;
    s.few_part = 1u << 30;
    s.few_splits = 1;
    s.many_splits = 1;
    if (s.few_rows) {
        // Parts of 256 tokens at least. A part's start and end cost about as much as 128 tokens, a join as 490, and
        // two workgroups of a CU share its reads: the cheapest number for rows of equal lengths and rows of any
        // (0.55 of the longest, the last part alone) together. Times by tokens of a part, 40 query and 8 key-value
        // heads of 128:
        //   64 rows of 8192 tokens       1024: 354 us  2048: 337  8192: 319
        //   64 rows of up to 8192        1024: 188 us  2048: 192  8192: 226
        //   16 rows of up to 4000         512: 36 us   1024: 38   4096: 58
        //   1 row of 16000                256: 20 us    512: 19   1024: 24  8192: 105
        // The estimate knows no head size. With heads of 64 and 256, what it takes is within 10% of the best of up to
        // six numbers tried: 1 row of 16000 (13 and 23 us), 16 rows of 4000 (28 and 50), 64 rows of 4096 (48 and 178).
        double best = 1e30;
        for (uint64_t n = 1; n <= kMaxSplits && (n == 1 || tokens > (n / 2) * 256); n *= 2) {
            const uint64_t part = up(up(tokens, n), 128) * 128;
            const double each = ((double)part + 128) / 2, units = (double)(n * kv->kv_heads * n_rows) / 256;
            const double cost = (std::ceil(units) + (n_rows > 1 ? 0.55 * units + 1 : 0)) * each + (n > 1 ? 490 : 0);
            if (cost < best) best = cost, s.few_part = (uint32_t)part, s.few_splits = (uint32_t)up(tokens, part);
        }
        if (s.few_splits > 1) s.few_sums = (uint64_t)n_rows * kv->kv_heads * s.few_rows * s.few_splits;
    }
    if (many) {
        const uint64_t rows = 32 * many_waves((int)up(kv->head_dim, 32)), tiles = up((uint64_t)m * group, rows);
        s.many_tiles = (uint32_t)((uint64_t)m * group / rows + n_rows);
        // Parts of 256 tokens at least, of the number that costs least by an estimate in us: a workgroup's token costs
        // 0.022 of its round and 0.012 more as far as every CU has one, its start and end 12, a join 10 and 8 more per
        // 81920 rows of a part. Measured, with 40 query and 8 key-value heads of 128 (tokens over tokens):
        //   parts              1       2       3       4
        //   2048 over 2048    79 us  111     112     131
        //   2048 over 4096   177     198     195     211
        //   2048 over 8192   413     379     361     375
        //   2048 over 16384  885     745     698     692
        //   512 over 8192    232     139     108     149
        //   64 over 16384    443     235     164     127   (16: 53)
        // With heads of 64 and 256 what it takes is within 1% of the best of those tried for 2048 over 8192 (131 and 502
        // us), 512 over 8192 (78 and 150) and 64 over 16384 (38 and 69), and with 20 query and 4 key-value heads of 64
        // or 128 one part for 2048 over 2048 where three are faster (53 and 71 us, 45 and 64).
        const uint64_t most_splits = std::min<uint64_t>(16, std::max<uint64_t>(1, tokens / 256));
        const double length = (double)tokens - (p->causal ? (double)std::min(most, tokens) / 2 : 0);
        double best = 1e30;
        for (uint64_t n = 1; n <= most_splits; ++n) {
            const double units = (double)(tiles * kv->kv_heads * n) / 256, rounds = std::ceil(units);
            const double join = n > 1 ? 10 + 8 * (double)n * (double)((uint64_t)m * p->q_heads) / 81920 : 0;
            const double cost = length / (double)n * (0.022 * rounds + 0.012 * units) + 12 * rounds + join;
            if (cost < best) best = cost, s.many_splits = (uint32_t)n;
        }
        if (s.many_splits > 1) s.many_sums = (uint64_t)m * p->q_heads * s.many_splits;
    }
    return s;
}

int check_attend(const afx_attend *p, const afx_kv_pages *kv, uint32_t n_rows, uint32_t m) {
    const int rc = check_kv(kv);
    if (rc != AFX_OK) return rc;
    if (!p || p->q_heads == 0 || p->q_heads % kv->kv_heads || p->q_heads / kv->kv_heads > kMaxGroup ||
        !std::isfinite(p->scale * kLog2e))
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
    *bytes = plan(p, kv, n_rows, m).bytes(kv->head_dim);
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
    if ((uint64_t)t->max_pages * t->page_tokens > kMaxPositions) return AFX_E_UNSUPPORTED;
    if (m == 0 || n_rows == 0) return AFX_OK;
    const uint64_t width = (uint64_t)p->q_heads * kv->head_dim;
    if (!starts_dev || !q_dev || !out_dev || q_stride < width || out_stride < width || (!seqs_dev && n_rows > t->n_seqs))
        return AFX_E_INVALID_ARG;
    if (q_stride >= kMaxRowStride || out_stride >= kMaxRowStride) return AFX_E_UNSUPPORTED;
    if (q_stride % 8 || out_stride % 8 || !aligned({q_dev, out_dev}, 16) || !aligned({seqs_dev, starts_dev, lse_dev}, 4))
        return AFX_E_MISALIGNED;
    const Plan w = plan(p, kv, n_rows, m);
    const uint64_t need = w.bytes(kv->head_dim);
    // a launch takes fewer than 2^32 threads
    const uint64_t few_blocks = (uint64_t)kv->kv_heads * n_rows * std::max(w.few_rows, w.few_splits);
    const uint64_t many_blocks = (uint64_t)kv->kv_heads * w.many_tiles * w.many_splits;
    const uint64_t joins = w.many_sums ? up((uint64_t)m * p->q_heads, kJoinThreads / (kv->head_dim / 4)) : 0;
    if (std::max(few_blocks, joins) * kJoinThreads >= 1ull << 32 ||
        many_blocks * 64 * many_waves((int)up(kv->head_dim, 32)) >= 1ull << 32)
        return AFX_E_UNSUPPORTED;
    if (need && !ws_dev) return AFX_E_INVALID_ARG;
    if (need && !aligned({ws_dev}, 16)) return AFX_E_MISALIGNED;
    const RowSpan s[] = {RowSpan{out_dev, m, 2 * width, 2 * out_stride},
                         flat(lse_dev, 4ull * m * p->q_heads),
                         flat(ws_dev, need),
                         RowSpan{q_dev, m, 2 * width, 2 * q_stride},
                         flat(kv->k_dev, kv_bytes(kv)),
                         flat(kv->v_dev, kv_bytes(kv)),
                         table_span(t),
                         flat(t->len_dev, 4ull * t->n_seqs),
                         flat(seqs_dev, 4ull * n_rows),
                         flat(starts_dev, 4ull * n_rows + 4)};
    if (outputs_overlap(s, 3, 10)) return AFX_E_INVALID_ARG;
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
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
    a.scale2 = p->scale == 0.f ? 1.f : std::fabs(p->scale) * kLog2e;
    a.q_and = p->scale == 0.f ? 0 : ~0u;
    a.q_xor = p->scale < 0.f ? 0x80008000u : 0;
    a.few_rows = w.few_rows;
    a.few_part = w.few_part;
    a.few_splits = w.few_splits;
    a.many_tiles = w.many_tiles;
    a.many_splits = w.many_splits;
    a.few_o = static_cast<float *>(ws_dev);
    a.many_o = a.few_o + w.few_sums * a.d;
    a.few_ml = reinterpret_cast<float2 *>(a.many_o + w.many_sums * a.d);
    a.many_ml = a.few_ml + w.few_sums;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (w.many_tiles) rc = launch_attend_many(a, st);
    if (rc == AFX_OK && w.few_rows) rc = launch_attend_few(a, st);
    void *args[] = {&a};
    auto join = [&](const void *fn, uint64_t blocks) {
        return hipLaunchKernel(fn, dim3((uint32_t)blocks), dim3(kJoinThreads), args, 0, st) == hipSuccess ? AFX_OK
                                                                                                       : AFX_E_HIP;
    };
    const uint32_t teams = kJoinThreads / (a.d / 4);
    if (rc == AFX_OK && w.few_sums && w.few_splits <= kTeamParts)
        rc = join(reinterpret_cast<const void *>(&afx_attend_join_teams_kernel),
                  up((uint64_t)n_rows * a.kv_heads * a.few_rows, teams));
    else if (rc == AFX_OK && w.few_sums)
        rc = join(reinterpret_cast<const void *>(&afx_attend_join_few_kernel), (uint64_t)n_rows * a.kv_heads * a.few_rows);
    if (rc == AFX_OK && w.many_sums)
        rc = join(reinterpret_cast<const void *>(&afx_attend_join_many_kernel),
                  up((uint64_t)m * a.q_heads, teams));
    return rc;
}

}  // extern "C"
