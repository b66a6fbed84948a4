// afx_attend_few.hip -- attention of few query rows (one or a few new tokens
// a sequence) over a paged cache: generation (gfx950).
//
// Reading the cache once bounds it. A workgroup of 4 waves takes one
// key-value head of a batch row, or one part of its tokens; each wave takes
// every fourth tile of 32 tokens on its own, and the waves' sums meet in LDS
// at the end. Keys and values go from memory to the matrix cores' operand
// registers as they lie in the pages, 16 bytes a lane, no LDS in between:
//   S^T = K Q^T    v_mfma_f32_16x16x32_bf16, K rows (tokens) as A, query rows
//                  as B: a lane holds 4 tokens' scores of one query row;
//   O^T += V^T P^T V^T rows (dimensions) as A, the weights as B.
// Two score tiles of 16 tokens take their rows from tokens 8 (i / 4) + i mod 4
// and 4 more, so that lane group g (lanes 16 g ..) ends up with the scores of
// tokens 8 g .. 8 g + 7, which is what it has to feed as B: the weights never
// leave their lane.
//
// The next tile's keys are requested when this tile's scores are done with
// them, its values after the second product: one of both is always on its
// way. A row's running maximum moves only when one of its scores exceeds it by
// 8 (a factor 2^8): most tiles exchange nothing between lanes. Weights then lie in 0..2^8
// and lose nothing, as their rounding to BF16 is relative.
//
// With 40 query and 8 key-value heads of 128: one token of each of 64
// sequences of up to 8192 tokens takes 189 us, and 5 for the join (1.08 GB of
// cache, 5.7 TB/s); one token over 131072 80 us (537 MB, 6.7 TB/s), and 5.
// Heads of 200 to 248 dimensions reload up to 16 values a lane from scratch
// memory in the loop: 64 x 1 over 4096 tokens of 4 heads of 232 take 225 us,
// where those of 256, 10% more bytes, take 178.
#include <type_traits>

#include "afx_attend.h"

namespace afx {
namespace {

constexpr uint32_t kWaves = 4, kThreads = 64 * kWaves;
constexpr float kSlack = 8.f;

// One wave's state: for each of RG groups of 16 query rows, the lane's row is
// lane mod 16 of it.
template <int KC, int RG>
struct Wave {
    static constexpr int kDT = 2 * KC;  // tiles of 16 dimensions
    bf16x8 q[RG][KC];
    f32x4 o[RG][kDT];
    float top[RG], sum[RG];
};

struct Where {
    const int32_t *table;
    const uint16_t *k, *v;  // of page 0's head
    uint32_t page_elems, size, shift, d;
    int32_t lo, hi;      // positions that all rows see
    int32_t first, last; // and any
    // In LDS: begin and end of what each of the wave's rows sees. (Only partial tiles need them; at 256 dimensions the
    // hot loop has no registers left.)
    int2 *range;
};

// 8 tokens' worth of a value fragment without the tokens that ok leaves out.
__device__ inline u32x4 only(u32x4 v, uint32_t ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] &= ((ok >> (2 * i)) & 1 ? 0xFFFFu : 0u) | ((ok >> (2 * i + 1)) & 1 ? 0xFFFF0000u : 0u);
    return v;
}

__device__ inline u32x4 once(const uint16_t *p) {  // (read by this wave only)
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}

// A wave's reads of a tile of 32 tokens. kFull: a head has 32 KC dimensions,
// none of a fragment lies behind them.
template <int KC, bool kFull>
struct Reads {
    static constexpr int kDT = 2 * KC;
    const AttendArgs &a;
    const Where &w;
    uint32_t c, g;

    // The page ids of the lane's key tokens (8 (c / 4) ..) and value tokens (8 g ..).
    __device__ uint32_t page(int32_t at) const { return (uint32_t)w.table[min((uint32_t)at >> w.shift, a.max_pages - 1)]; }
    __device__ uint32_t k_page(int32_t j) const { return page(j + 8 * (int32_t)(c >> 2)); }
    __device__ uint32_t v_page(int32_t j) const { return page(j + 8 * (int32_t)g); }

    __device__ void keys(int32_t j, uint32_t id, u32x4 (&f)[2][KC]) const {
        const uint32_t tok = ((uint32_t)j + 8 * (c >> 2) + (c & 3)) & (w.size - 1), last = w.d / 8 - 1;
        const uint16_t *p = w.k + (uint64_t)(id < a.n_pages ? id : 0) * w.page_elems + tok * 8;
        if (kFull) p += g * w.size * 8;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
            const uint16_t *pc = p + (kFull ? 4 * kc : min(4 * kc + g, last)) * w.size * 8;
            f[0][kc] = once(pc);
            f[1][kc] = once(pc + 32);
        }
    }
    __device__ void values(int32_t j, uint32_t id, u32x4 (&f)[kDT]) const {
        const uint32_t tok = ((uint32_t)j + 8 * g) & (w.size - 1);
        const uint16_t *p = w.v + (uint64_t)(id < a.n_pages ? id : 0) * w.page_elems + tok * w.d + (kFull ? c * 8 : 0);
#pragma unroll
        for (int t = 0; t < kDT; ++t)
            f[t] = once(p + (kFull ? 16 * t : min(16 * t + c, w.d - 1)) * 8);
    }
};

// The scores of a tile: sc[x][y][e] is that of query row c of group x and token 8 g + 4 y + e.
template <int KC, int RG, bool kFull>
__device__ __forceinline__ void scores(const Where &w, const Wave<KC, RG> &s, const u32x4 (&kf)[2][KC], uint32_t g,
                                       f32x4 (&sc)[RG][2]) {
#pragma unroll
    for (int x = 0; x < RG; ++x) sc[x][0] = sc[x][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kc = 0; kc < KC; ++kc)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            u32x4 f = kf[y][kc];
            if (!kFull && kc >= KC - 2 && 4 * kc + g >= w.d / 8) f = u32x4{0, 0, 0, 0};  // behind the head's dimensions
#pragma unroll
            for (int x = 0; x < RG; ++x)
                sc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), s.q[x][kc], sc[x][y], 0,
                                                                   0, 0);
        }
}

// Their weights, with the running maximum and sum.
template <int KC, int RG>
__device__ __forceinline__ void weights(const AttendArgs &a, Wave<KC, RG> &s, const f32x4 (&sc)[RG][2], bf16x8 (&p)[RG]) {
#pragma unroll
    for (int x = 0; x < RG; ++x) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = sc[x][e / 4][e % 4];
        float best = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
        best *= a.scale2;
        if (__any(best > s.top[x] + kSlack)) {
            best = fmaxf(best, __shfl_xor(best, 16));
            best = fmaxf(best, __shfl_xor(best, 32));
            // (not with another row's: what this row does not see would change its bits)
            const bool moves = best > s.top[x] + kSlack;
            const float f = moves ? exp2_fast(s.top[x] - best) : 1.f;
            s.top[x] = moves ? best : s.top[x];
            s.sum[x] *= f;
#pragma unroll
            for (int t = 0; t < 2 * KC; ++t) s.o[x][t] *= f;
        }
        const float base = s.top[x] == -INFINITY ? 0.f : s.top[x];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = exp2_fast(__builtin_fmaf(v[e], a.scale2, -base));
        s.sum[x] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
#pragma unroll
        for (int e = 0; e < 8; ++e) p[x][e] = (__bf16)v[e];
    }
}

template <int KC, int RG>
__device__ __forceinline__ void add_values(Wave<KC, RG> &s, const u32x4 (&vf)[2 * KC], const bf16x8 (&p)[RG]) {
#pragma unroll
    for (int t = 0; t < 2 * KC; ++t)
#pragma unroll
        for (int x = 0; x < RG; ++x)
            s.o[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vf[t]), p[x], s.o[x][t], 0, 0, 0);
}

// The tile at j, of which some rows see only a part, or not all pages are in
// the cache. Returns whether there are infinities or NaN among its values
// that some row sees, which have been left out.
template <int KC, int RG, bool kFull>
__device__ __forceinline__ bool partial_tile(const AttendArgs &a, const Where &w, Wave<KC, RG> &s, int32_t j,
                                             uint32_t lane) {
    lane = opaque(lane);
    const uint32_t c = lane & 15, g = lane >> 4;
    const Reads<KC, kFull> reads{a, w, c, g};
    const uint32_t id = reads.v_page(j);
    u32x4 kf[2][KC], vf[2 * KC];
    reads.keys(j, reads.k_page(j), kf);
    reads.values(j, id, vf);
    f32x4 sc[RG][2];
    scores<KC, RG, kFull>(w, s, kf, g, sc);
    uint32_t any = 0;  // of the lane's 8 tokens, those that some row sees
    int2 see[RG];
#pragma unroll
    for (int x = 0; x < RG; ++x) see[x] = w.range[16 * x + c];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int32_t at = j + 8 * (int32_t)g + e;
        const bool there = id < a.n_pages;
        any |= there && at >= w.first && at < w.last ? 1u << e : 0u;
#pragma unroll
        for (int x = 0; x < RG; ++x)
            if (!there || at < see[x].x || at >= see[x].y) sc[x][e / 4][e % 4] = -INFINITY;
    }
    bf16x8 p[RG];
    weights<KC, RG>(a, s, sc, p);
    uint32_t strange = 0;
#pragma unroll
    for (int t = 0; t < 2 * KC; ++t) {
        vf[t] = only(vf[t], any);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = finite2(vf[t][i]);
            strange |= v ^ vf[t][i];
            vf[t][i] = v;
        }
    }
    add_values<KC, RG>(s, vf, p);
    return __any(strange != 0);
}

// The last place of a whole tile before j1.
__device__ inline int32_t whole_end(const Where &w, int32_t j1) { return min(w.hi - (int32_t)kFewTokens, j1 - 1); }

// The infinities and NaN that partial_tile left out of the wave's tiles from
// j0 to j1 are added to the outputs of a row that sees begin .. end - 1, if it
// sees them: to the lane's four of every 16, row[dim].
__device__ __forceinline__ void add_strange(const AttendArgs &a, const Where &w, int32_t begin, int32_t end, int32_t j0,
                                            int32_t j1, uint32_t g, float *row) {
    auto page = [&](int32_t at) { return (uint32_t)w.table[min((uint32_t)at >> w.shift, a.max_pages - 1)]; };
#pragma unroll 1
    for (int32_t j = j0; j < j1; j += (int32_t)(kWaves * kFewTokens)) {
        if (j >= w.lo && j <= whole_end(w, j1) && page(j) < a.n_pages && page(j + 16) < a.n_pages) continue;
#pragma unroll 1
        for (int32_t at = j; at < j + (int32_t)kFewTokens; ++at) {
            const uint32_t id = page(at);
            if (id >= a.n_pages || at < begin || at >= end) continue;
            const uint16_t *v = w.v + (uint64_t)id * w.page_elems + ((uint32_t)at & (w.size - 1) & ~7u) * w.d + at % 8;
#pragma unroll 1
            for (uint32_t dim = 4 * g; dim < w.d; dim += 16)
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x) {
                    const uint16_t value = v[(dim + x) * 8];
                    if (odd(value)) row[dim + x] += from_bf16(value);
                }
        }
    }
}

// One pass over the wave's tiles from j0 to j1; whether partial_tile left out
// values of one.
template <int KC, int RG, bool kFull>
__device__ __forceinline__ bool run(const AttendArgs &a, const Where &w, Wave<KC, RG> &s, int32_t j0, int32_t j1,
                                    uint32_t wave, uint32_t lane) {
#pragma unroll
    for (int x = 0; x < RG; ++x) {
        s.top[x] = -INFINITY;
        s.sum[x] = 0.f;
#pragma unroll
        for (int t = 0; t < 2 * KC; ++t) s.o[x][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    constexpr int32_t kStep = kWaves * kFewTokens;
    const uint32_t g = lane >> 4;
    const Reads<KC, kFull> reads{a, w, lane & 15, g};
    int32_t j = j0 + (int32_t)(wave * kFewTokens);
    const int32_t end = whole_end(w, j1);
    bool strange = false;
    while (j < j1) {
        if (j >= w.lo && j <= end) {
            uint32_t id = reads.v_page(j), kid2 = reads.k_page(j + kStep), vid2 = reads.v_page(j + kStep);
            u32x4 kf[2][KC], vf[2 * KC];
            reads.keys(j, reads.k_page(j), kf);
            reads.values(j, id, vf);
            while (__all(id < a.n_pages)) {
                f32x4 sc[RG][2];
                scores<KC, RG, kFull>(w, s, kf, g, sc);
                const uint32_t kid3 = reads.k_page(j + 2 * kStep), vid3 = reads.v_page(j + 2 * kStep);
                const bool more = j + kStep <= end;
                if (more) reads.keys(j + kStep, kid2, kf);
                bf16x8 p[RG];
                weights<KC, RG>(a, s, sc, p);
                add_values<KC, RG>(s, vf, p);
                j += kStep;
                if (!more) break;
                reads.values(j, vid2, vf);
                id = vid2;
                kid2 = kid3;
                vid2 = vid3;
            }
            if (j > end) continue;
        }
        if (j < j1) strange |= partial_tile<KC, RG, kFull>(a, w, s, j, lane);
        j += kStep;
    }
    return strange;
}

template <int KC>
struct Lds {
    float o[kWaves][16][32 * KC + 4];
    float2 ml[kWaves][16];
    int2 range[kWaves][32];
};

// What a workgroup works on: a key-value head of batch row r, or one part of
// its tokens, j0 .. j1 - 1.
struct Part {
    BatchRow row;
    uint32_t r, kvh, part, splits;
    int32_t j0, j1;
};

// The query rows from r0 on.
template <int KC, int RG, bool kFull>
__device__ __forceinline__ void unit(const AttendArgs &a, const Part &t, uint32_t r0, Lds<KC> &lds) {
    constexpr int kDT = 2 * KC;
    const BatchRow &row = t.row;
    const int32_t j0 = t.j0, j1 = t.j1;
    const uint32_t r = t.r, kvh = t.kvh, part = t.part;
    const uint32_t lane = opaque(threadIdx.x) % 64, c = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);  // (a scalar: so are the places of its tiles)
    const uint32_t rows = row.n * a.group;
    Where w;
    w.table = a.table + (row.seq < a.n_seqs ? row.seq : 0) * a.table_stride;
    w.size = 1u << a.page_shift;
    w.shift = a.page_shift;
    w.d = a.d;
    w.page_elems = w.size * a.kv_heads * a.d;
    w.k = a.k + (uint64_t)kvh * w.size * a.d;
    w.v = a.v + (uint64_t)kvh * w.size * a.d;
    const uint32_t last = min(r0 + 16 * RG, rows) - 1;
    w.first = row.begin(a, r0 / a.group);
    w.last = row.end(a, last / a.group);
    w.lo = row.begin(a, last / a.group);
    w.hi = row.end(a, r0 / a.group);
    w.range = lds.range[wave];
    Wave<KC, RG> s;
#pragma unroll
    for (int x = 0; x < RG; ++x) {
        const uint32_t rr = min(r0 + 16 * x + c, last), t = rr / a.group;
        w.range[16 * x + c] = make_int2(row.begin(a, t), row.end(a, t));  // (read by this wave)
        const uint16_t *q = a.q + (row.from + t) * a.q_stride + (kvh * a.group + rr % a.group) * a.d;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) s.q[x][kc] = load_q(a, q, 32 * kc + 8 * g);
    }
    const bool strange = run<KC, RG, kFull>(a, w, s, j0, j1, wave, lane);
    // the waves' sums, 16 rows at a time
#pragma unroll
    for (int x = 0; x < RG; ++x) {
        const uint32_t tid = opaque(threadIdx.x), c = tid & 15, g = tid % 64 >> 4;  // (formed again: run has no room)
        s.sum[x] += __shfl_xor(s.sum[x], 16);
        s.sum[x] += __shfl_xor(s.sum[x], 32);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kDT; ++t) *reinterpret_cast<f32x4 *>(&lds.o[wave][c][16 * t + 4 * g]) = s.o[x][t];
        if (g == 0) lds.ml[wave][c] = make_float2(s.top[x], s.sum[x]);
        if (strange) {
            const int2 see = lds.range[wave][16 * x + c];
            add_strange(a, w, see.x, see.y, j0 + (int32_t)(wave * kFewTokens), j1, g, lds.o[wave][c]);
        }
        __syncthreads();
        const uint32_t quads = a.d / 4;
        for (uint32_t i = tid; i < 16 * quads; i += kThreads) {
            const uint32_t at = i / quads, quad = i % quads, rr = r0 + 16 * x + at;
            if (rr >= rows) break;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (uint32_t v = 0; v < kWaves; ++v) top = fmaxf(top, lds.ml[v][at].x);
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t v = 0; v < kWaves; ++v) {
                const float2 ml = lds.ml[v][at];
                const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - top);
                sum += f * ml.y;
                // (also where f has become 0: an infinity or NaN that a row sees shows, wherever the tokens are cut)
                o += f * *reinterpret_cast<const f32x4 *>(&lds.o[v][at][4 * quad]);
            }
            const uint32_t tok = row.from + rr / a.group, h = kvh * a.group + rr % a.group;
            if (t.splits == 1) {
                const float k = sum == 0.f ? 0.f : 1.f / sum;
                if (sum == 0.f) o = f32x4{0.f, 0.f, 0.f, 0.f};
                *reinterpret_cast<uint2 *>(a.out + tok * a.out_stride + h * a.d + 4 * quad) =
                    make_uint2(pack2(o[0] * k, o[1] * k), pack2(o[2] * k, o[3] * k));
                if (a.lse && quad == 0) a.lse[(uint64_t)tok * a.q_heads + h] = lse_of(top, sum);
            } else {
                const uint64_t p = (((uint64_t)r * a.kv_heads + kvh) * a.few_rows + rr) * a.few_splits + part;
                *reinterpret_cast<f32x4 *>(a.few_o + p * a.d + 4 * quad) = o;
                if (quad == 0) a.few_ml[p] = make_float2(top, sum);
            }
        }
    }
}

template <int KC, int RG, bool kFull>
__global__ __launch_bounds__(kThreads, KC * RG <= 8 ? 2 : 1) void afx_attend_few_kernel(AttendArgs a) {
    __shared__ Lds<KC> lds;
    Part t;
    t.kvh = blockIdx.x % a.kv_heads, t.r = blockIdx.x / a.kv_heads, t.part = blockIdx.y;
    t.row = BatchRow(a, t.r);
    const uint32_t rows = t.row.n * a.group;
    if (rows == 0 || (a.many_tiles && rows > a.few_rows)) return;
    const FewRange range(a, t.row);
    t.splits = range.splits;
    if (t.part >= t.splits) return;
    t.j0 = range.base + (int32_t)(t.part * range.part);
    t.j1 = t.part + 1 == t.splits ? range.end : t.j0 + (int32_t)range.part;
    for (uint32_t r0 = 0; r0 < rows; r0 += 16 * RG)
        unit<KC, RG, kFull>(a, t, r0, lds);
}

}  // namespace

int launch_attend_few(const AttendArgs &a, hipStream_t stream) {
    AttendArgs args = a;
    void *p[] = {&args};
    auto go = [&](auto kc) {
        constexpr int KC = decltype(kc)::value;
        auto pick = [](auto *f) { return reinterpret_cast<const void *>(f); };
        const bool one = a.few_rows <= 16;
        const void *fn = a.d == 32 * KC ? one ? pick(&afx_attend_few_kernel<KC, 1, true>) : pick(&afx_attend_few_kernel<KC, 2, true>)
                         : one          ? pick(&afx_attend_few_kernel<KC, 1, false>)
                                        : pick(&afx_attend_few_kernel<KC, 2, false>);
        return hipLaunchKernel(fn, dim3(a.kv_heads * a.n_rows, a.few_splits), dim3(kThreads), p, 0, stream) == hipSuccess
                   ? AFX_OK
                   : AFX_E_HIP;
    };
    if (a.d <= 64) return go(std::integral_constant<int, 2>{});
    if (a.d <= 96) return go(std::integral_constant<int, 3>{});
    if (a.d <= 128) return go(std::integral_constant<int, 4>{});
    if (a.d <= 192) return go(std::integral_constant<int, 6>{});
    return go(std::integral_constant<int, 8>{});
}

}  // namespace afx
