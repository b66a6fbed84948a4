// afx_attend_many.hip -- attention of many query rows (chunks of prompts) over
// a paged cache (gfx950).
//
// The matrix cores bound it, with the vector unit close behind: 32 tokens of a
// wave's 32 rows are 16 matrix instructions of 32 cycles and 16 exponentials
// of 16. A workgroup of 8 waves takes 256 query rows of one key-value head, 32
// a wave, and its keys and values in tiles of 64 tokens (heads of more than
// 128 dimensions: 4 waves, tiles of 32), which go from the pages to LDS without
// passing through registers. The pages' order is that of the operands, so that
// every LDS read is 16 bytes a lane, 512 in a row.
//   S^T = K Q^T    v_mfma_f32_32x32x16_bf16, K rows (tokens) as A, query rows
//                  as B: a lane holds 16 of 32 tokens' scores of one query row;
//   O^T += V^T P^T V^T rows (dimensions) as A, the weights as B.
// Rows 4 .. 7 and 8 .. 11 of every 16 score rows take each other's tokens, so
// that a half wave ends up with the scores of tokens 8 h .. 8 h + 7 of every
// 16, which is what it has to feed as B.
//
// A wave runs one step of 32 tokens ahead of itself: while the vector unit
// forms one step's weights, the matrix cores multiply the next step's keys,
// and its largest score is found while they multiply the first step's values.
// Its keys thus belong to the next tile at a tile's last step, where the
// barrier stands; three tiles of LDS let the tile after that be requested
// there, with a tile's time to arrive. A row's running maximum moves only when
// one of its scores exceeds it by 8 (a factor 2^8), as in afx_attend_few.hip.
//
// 2048 tokens over 16384, 40 query and 8 key-value heads of 128: 660-740 us
// as the clock allows (0.87-0.97 PFLOP/s), and 30 for the join of 4 parts. Of
// the kernel's cycles the matrix cores work in 43%, vector instructions take
// 57% to issue (an exponential 16 cycles, others 4) and LDS works in 22%: the
// first two hardly overlap. 64 rows a
// wave, one wave a SIMD, with half the reads of LDS and every exponential
// between matrix instructions, took as long.
#include <type_traits>

#include "afx_attend.h"

namespace afx {
namespace {

constexpr float kSlack = 8.f;

template <int KC>
struct Shape {
    static constexpr uint32_t kWaves = many_waves(KC), kThreads = 64 * kWaves, kRows = 32 * kWaves;
    static constexpr uint32_t kT = KC <= 4 ? 64 : 32;  // tokens of a tile
    static constexpr int kSteps = kT / 32;
    static constexpr uint32_t kDims = 32 * KC;
    static constexpr uint32_t kBytes = kT * kDims * 2;  // of a key tile, [dim / 8][token] of 16, or value tile, [token / 8][dim]
    static constexpr uint32_t kPieces = kBytes / 1024;  // a wave's load fills 1 KB
    static constexpr int kEach = (kPieces + kWaves - 1) / kWaves;
};

// 16 bytes a lane from p into LDS at `to` (wave-uniform) + 16 lane.
__device__ inline void load_to_lds(const uint16_t *p, uint8_t *to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)p,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// What a workgroup works on.
struct Tile {
    BatchRow row;
    uint32_t r0, rows, kvh, part;  // first query row, all query rows of the batch row
};

// Tile number u, counted over the batch rows that this kernel takes, the last
// tiles of a row (the longest) first. False behind the last.
__device__ inline bool find_tile(const AttendArgs &a, uint32_t u, uint32_t rows, Tile &t) {
    const uint32_t lane = threadIdx.x % 64;
    uint32_t before = 0;
    for (uint32_t r0 = 0; r0 < a.n_rows; r0 += 64) {
        const uint32_t r = r0 + lane;
        uint32_t n = 0;
        if (r < a.n_rows) {
            const uint32_t from = (uint32_t)min(max(a.starts[r], 0), (int32_t)a.m);
            const uint32_t to = (uint32_t)min(max(a.starts[r + 1], 0), (int32_t)a.m);
            n = to > from ? (to - from) * a.group : 0;
        }
        const uint32_t tiles = n > a.few_rows ? (n + rows - 1) / rows : 0;
        uint32_t sum = tiles;
#pragma unroll
        for (uint32_t o = 1; o < 64; o *= 2) {
            const uint32_t left = __shfl_up(sum, o);
            if (lane >= o) sum += left;
        }
        const uint64_t at = __ballot(u < before + sum);
        if (at) {
            const uint32_t l = (uint32_t)__ffsll((unsigned long long)at) - 1;
            t.row = BatchRow(a, __builtin_amdgcn_readfirstlane(r0 + l));
            t.rows = t.row.n * a.group;
            const uint32_t end = before + __builtin_amdgcn_readlane(sum, l);
            t.r0 = (end - 1 - u) * rows;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

template <int KC>
struct Wave {
    bf16x8 q[2 * KC];
    f32x16 o[KC], sc;  // outputs; the scores of the next step
    float top, sum;
    int32_t begin, end;  // positions that the lane's row sees
};

struct Where {
    const int32_t *table;
    const uint16_t *k, *v;  // of page 0's head
    uint32_t page_elems, size;
    int32_t lo, hi;              // positions that all rows of the wave see
    int32_t first, last;         // and any
    int32_t wg_lo, wg_hi;        // the same for the rows of the workgroup
    int32_t wg_first, wg_last;
};

// The largest of the lane's scores.
__device__ inline float largest(const f32x16 &s) {
    float best = fmaxf(s[0], s[1]);
#pragma unroll
    for (int e = 2; e < 16; e += 2) best = fmaxf(best, fmaxf(s[e], s[e + 1]));
    return best;
}

// Moves the rows' running maxima to their scores of the next step, where one exceeds its row's by kSlack.
template <int KC>
__device__ __forceinline__ void follow(Wave<KC> &s, float best) {
    if (!__any(best > s.top + kSlack)) return;
    best = fmaxf(best, __shfl_xor(best, 32));
    // (not with another row's: what this row does not see would change its bits)
    const bool moves = best > s.top + kSlack;
    const float f = moves ? exp2_fast(s.top - best) : 1.f;
    s.top = moves ? best : s.top;
    s.sum *= f;
#pragma unroll
    for (int t = 0; t < KC; ++t) s.o[t] *= f;
}

// Without the scores of what the lane's row does not see; j: the step's first
// position, there: which of its 32 tokens have pages in the cache.
template <int KC>
__device__ __forceinline__ void hide(Wave<KC> &s, int32_t j, uint32_t there, uint32_t lane) {
    // the lane's tokens of e: 8 h + t, t = 16 (e / 8) + e mod 8
    const uint32_t h8 = opaque(lane) >> 5 << 3;
    const int32_t own = j + (int32_t)h8;
    const uint32_t from = (uint32_t)max(s.begin - own, 0), n = (uint32_t)max(s.end - own - (int32_t)from, 0);
    const uint32_t pages = there >> h8;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint32_t t = 16 * (e / 8) + e % 8;
        if (t - from >= n || !(pages >> t & 1)) s.sc[e] = -INFINITY;
    }
}

// Values of the tile at j that no row of the workgroup sees become 0, and so
// do infinities and NaN; whether there were such (in a scalar register: as a
// lane's flag it costs the loop 60 registers). there: which tokens have pages.
template <int KC>
__device__ __forceinline__ uint32_t clear_values(const Where &w, uint8_t *v_tile, int32_t j, uint64_t there) {
    using S = Shape<KC>;
    uint32_t strange = 0;
    for (uint32_t x = opaque(threadIdx.x); x < S::kBytes / 16; x += S::kThreads) {
        u32x4 *p = reinterpret_cast<u32x4 *>(v_tile + x * 16);
        u32x4 v = *p;
        const uint32_t t8 = x / S::kDims * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            auto seen = [&](uint32_t t) {
                const int32_t at = j + (int32_t)t;
                return (there >> t & 1) && at >= w.wg_first && at < w.wg_last;
            };
            const uint32_t u = v[e] & ((seen(t8 + 2 * e) ? 0xFFFFu : 0u) | (seen(t8 + 2 * e + 1) ? 0xFFFF0000u : 0u));
            v[e] = finite2(u);
            strange |= u ^ v[e];
        }
        *p = v;
    }
    return (uint32_t)__builtin_amdgcn_readfirstlane(__syncthreads_or(strange != 0));
}

// The infinities and NaN that clear_values took out of the tiles from j0 to j1
// are added to the row's outputs in memory, if it sees them: to those of the
// lane, put(dim, value).
template <int KC, class F>
__device__ __forceinline__ void add_strange(const AttendArgs &a, const Where &w, const Wave<KC> &s, int32_t j0,
                                            int32_t j1, uint32_t h, F put) {
    constexpr int32_t kT = Shape<KC>::kT;
    auto page = [&](int32_t at) { return (uint32_t)w.table[min((uint32_t)at >> a.page_shift, a.max_pages - 1)]; };
#pragma unroll 1
    for (int32_t j = j0; j < j1; j += kT) {
        bool cleared = j < w.wg_lo || j + kT > w.wg_hi;
        for (int32_t t = 0; t < kT; t += 16) cleared |= page(j + t) >= a.n_pages;
        if (!cleared) continue;
#pragma unroll 1
        for (int32_t at = j; at < j + kT; ++at) {
            const uint32_t id = page(at);
            if (id >= a.n_pages || at < s.begin || at >= s.end) continue;
            const uint16_t *v = w.v + (uint64_t)id * w.page_elems + ((uint32_t)at & (w.size - 1) & ~7u) * a.d + at % 8;
#pragma unroll 1
            for (uint32_t dim = 4 * h; dim < a.d; dim += 8)
#pragma unroll
                for (uint32_t x = 0; x < 4; ++x) {
                    const uint16_t value = v[(dim + x) * 8];
                    if (odd(value)) put(dim + x, from_bf16(value));
                }
        }
    }
}

// The keys of step n of a tile: s.sc.
template <int KC>
__device__ __forceinline__ void multiply_keys(Wave<KC> &s, const uint8_t *k_tile, int n, uint32_t lane) {
    using S = Shape<KC>;
    const uint32_t i = lane & 31, h = lane >> 5;
    // a score row's token: rows 4 .. 7 and 8 .. 11 of 16 change places
    const uint32_t tok = (i & 16) | (i & 3) | ((i & 4) << 1) | ((i & 8) >> 1);
    const uint8_t *base = k_tile + (h * S::kT + tok) * 16;
#pragma unroll
    for (int e = 0; e < 16; ++e) s.sc[e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 2 * KC; ++ks)
        s.sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8 *>(base + (2 * ks * S::kT + 32 * n) * 16), s.q[ks], s.sc, 0, 0, 0);
}

// One step: the weights of s.sc, which are of step n of the tile at j, times
// the step's values, and the scores of the next step (step m of `next`).
template <int KC>
__device__ __forceinline__ void step(const AttendArgs &a, const Where &w, Wave<KC> &s, const uint8_t *v_tile, int n,
                                     const uint8_t *next, int m, bool more, int32_t j_next, uint32_t there_next,
                                     uint32_t lane) {
    using S = Shape<KC>;
    const uint32_t i = lane & 31, h = lane >> 5;
    const float base = s.top == -INFINITY ? 0.f : s.top;
    bf16x8 p[2];
    auto weigh = [&](const f32x16 &was) __attribute__((always_inline)) {
        float part[4] = {};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float v = exp2_fast(__builtin_fmaf(was[e], a.scale2, -base));
            part[e % 4] += v;
            p[e / 8][e % 8] = (__bf16)v;
        }
        s.sum += (part[0] + part[1]) + (part[2] + part[3]);
    };
    const f32x16 was = s.sc;
    const uint8_t *v_base = v_tile + ((4 * n + h) * S::kDims + i) * 16;
    bf16x8 v[2 * KC];
    // the next step's keys beside this one's weights
    multiply_keys<KC>(s, next, m, lane);
    weigh(was);
#pragma unroll
    for (int x = 0; x < 2 * KC; ++x)
        v[x] = *reinterpret_cast<const bf16x8 *>(v_base + (x / KC * 2 * S::kDims + 32 * (x % KC)) * 16);
    // and its largest score beside this one's values
#pragma unroll
    for (int x = 0; x < 2 * KC; ++x)
        s.o[x % KC] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[x], p[x / KC], s.o[x % KC], 0, 0, 0);
    float best = largest(s.sc);
    if (there_next != ~0u || j_next < w.lo || j_next + 32 > w.hi) {
        hide<KC>(s, j_next, there_next, lane);
        best = largest(s.sc);
    }
    follow<KC>(s, more ? best * a.scale2 : -INFINITY);
}

// All tiles from j0 to j1; whether clear_values took infinities or NaN out of
// one. The buffers are objects of their own: of one array the compiler would
// have every read wait for all loads into it.
template <int KC>
__device__ __forceinline__ uint32_t run(const AttendArgs &a, const Where &w, Wave<KC> &s, uint8_t *k0, uint8_t *v0,
                                    uint8_t *k1, uint8_t *v1, uint8_t *k2, uint8_t *v2, int32_t j0, int32_t j1,
                                    uint32_t wave, uint32_t lane) {
    using S = Shape<KC>;
    constexpr int32_t kT = S::kT;
    const uint32_t chunks = a.d / 8;
    s.top = -INFINITY;
    s.sum = 0.f;
#pragma unroll
    for (int t = 0; t < KC; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) s.o[t][e] = 0.f;
    if (j0 >= j1) return 0;
    auto page_of = [&](int32_t at) __attribute__((always_inline)) {  // of the lane's token of the tile at `at`
        return (uint32_t)w.table[min(((uint32_t)at + lane % kT) >> a.page_shift, a.max_pages - 1)];
    };
    auto tokens_there = [&](uint32_t id) __attribute__((always_inline)) {
        const uint64_t there = __ballot(id < a.n_pages);
        return kT == 64 ? there : there | ~0ull << 32;
    };
    // Wave w takes 1 KB pieces w, w + kWaves, .. of both tiles: 64 / kT groups of 8 dimensions of kT keys, 64
    // dimensions of 8 values (of 96 dimensions, two such groups where they end inside a piece). Values behind the
    // head's dimensions repeat its last.
    auto request = [&](int32_t at, uint32_t id, uint8_t *k_tile, uint8_t *v_tile) __attribute__((always_inline)) {
        const uint32_t safe = id < a.n_pages ? id : 0, mask = w.size - 1;
        const uint16_t *pk = w.k + (uint64_t)safe * w.page_elems + (((uint32_t)at + lane % kT) & mask) * 8;
#pragma unroll
        for (int x = 0; x < S::kEach; ++x) {
            const uint32_t piece = wave + S::kWaves * x;
            if (S::kPieces % S::kWaves && piece >= S::kPieces) continue;
            if constexpr (kT == 64) {
                if (piece < chunks) load_to_lds(pk + piece * w.size * 8, k_tile + piece * 1024);
            } else {
                const uint32_t chunk = 2 * piece + lane / 32;  // (behind the head's last one the zeros stay)
                if (chunk < chunks) load_to_lds(pk + chunk * w.size * 8, k_tile + piece * 1024);
            }
        }
#pragma unroll
        for (int x = 0; x < S::kEach; ++x) {
            const uint32_t piece = wave + S::kWaves * x;
            if (S::kPieces % S::kWaves && piece >= S::kPieces) continue;
            uint32_t tok, dim, page;
            if constexpr (S::kDims % 64 == 0) {  // one group of 8 values: its page is the same for all lanes
                tok = piece / (S::kDims / 64) * 8;
                dim = piece % (S::kDims / 64) * 64 + lane;
                page = __builtin_amdgcn_readlane(safe, tok);
            } else {
                const uint32_t entry = piece * 64 + lane;
                tok = entry / S::kDims * 8;
                dim = entry % S::kDims;
                page = __shfl(safe, tok);
            }
            load_to_lds(w.v + (uint64_t)page * w.page_elems + (((uint32_t)at + tok) & mask) * a.d + min(dim, a.d - 1) * 8,
                        v_tile + piece * 1024);
        }
    };
    auto whole = [&](int32_t j, uint64_t there) __attribute__((always_inline)) { return there == ~0ull && j >= w.wg_lo && j + kT <= w.wg_hi; };
    // ids of three tiles: this one's, whose keys and values have arrived, the next one's, which are on their way, and
    // the one after that
    uint32_t id = page_of(j0), id1 = page_of(j0 + kT), id2 = page_of(j0 + 2 * kT);
    __syncthreads();  // (the keys' zeros)
    request(j0, id, k0, v0);
    if (j0 + kT < j1) request(j0 + kT, id1, k1, v1);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
    uint64_t there = tokens_there(id);
    uint32_t strange = 0;
    if (!whole(j0, there)) strange = clear_values<KC>(w, v0, j0, there);
    multiply_keys<KC>(s, k0, 0, lane);
    if ((uint32_t)there != ~0u || j0 < w.lo || j0 + 32 > w.hi) hide<KC>(s, j0, (uint32_t)there, lane);
    follow<KC>(s, largest(s.sc) * a.scale2);
    auto tile = [&](int32_t j, uint8_t *k_tile, uint8_t *v_tile, uint8_t *k_next, uint8_t *v_next, uint8_t *k_after,
                    uint8_t *v_after) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n + 1 < S::kSteps; ++n)
            step<KC>(a, w, s, v_tile, n, k_tile, n + 1, true, j + 32 * (n + 1),
                     (uint32_t)(there >> 32 * (n + 1)), lane);
        // The last step multiplies the next tile's keys: it has to have arrived, in every wave. No wave is still in the
        // tile before this one, whose buffers take the tile after the next.
        const bool more = j + kT < j1;
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __syncthreads();
        const uint64_t there1 = tokens_there(id1);
        const uint32_t id3 = page_of(j + 3 * kT);
        if (j + 2 * kT < j1) request(j + 2 * kT, id2, k_after, v_after);
        if (more && !whole(j + kT, there1)) strange |= clear_values<KC>(w, v_next, j + kT, there1);
        constexpr int kLast = S::kSteps - 1;
        step<KC>(a, w, s, v_tile, kLast, k_next, 0, more, j + kT, (uint32_t)there1, lane);
        there = there1;
        id1 = id2;
        id2 = id3;
    };
    for (int32_t j = j0; j < j1; j += 3 * kT) {
        tile(j, k0, v0, k1, v1, k2, v2);
        if (j + kT >= j1) break;
        tile(j + kT, k1, v1, k2, v2, k0, v0);
        if (j + 2 * kT >= j1) break;
        tile(j + 2 * kT, k2, v2, k0, v0, k1, v1);
    }
    return strange;
}

template <int KC>
__global__ __launch_bounds__(Shape<KC>::kThreads, KC <= 4 ? 2 : 1) void afx_attend_many_kernel(AttendArgs a) {
    using S = Shape<KC>;
    constexpr uint32_t kT = S::kT;
    __shared__ __attribute__((aligned(16))) uint8_t k0[S::kBytes], k1[S::kBytes], k2[S::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t v0[S::kBytes], v1[S::kBytes], v2[S::kBytes];
    Tile t;
    const uint32_t u = blockIdx.x / a.kv_heads;
    t.kvh = blockIdx.x % a.kv_heads;  // (neighbouring workgroups, on different XCDs, read different heads)
    t.part = u % a.many_splits;
    if (!find_tile(a, u / a.many_splits, S::kRows, t)) return;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, i = lane & 31, h = lane >> 5;
    const BatchRow &row = t.row;
    const uint32_t wg_last = min(t.r0 + S::kRows, t.rows) - 1;
    const uint32_t w0 = min(t.r0 + 32 * wave, wg_last), w1 = min(t.r0 + 32 * wave + 31, wg_last);
    Where w;
    w.table = a.table + (row.seq < a.n_seqs ? row.seq : 0) * a.table_stride;
    w.size = 1u << a.page_shift;
    w.page_elems = w.size * a.kv_heads * a.d;
    w.k = a.k + (uint64_t)t.kvh * w.size * a.d;
    w.v = a.v + (uint64_t)t.kvh * w.size * a.d;
    w.wg_first = row.begin(a, t.r0 / a.group);
    w.wg_last = max(row.end(a, wg_last / a.group), w.wg_first);
    w.wg_lo = row.begin(a, wg_last / a.group);
    w.wg_hi = row.end(a, t.r0 / a.group);
    w.first = row.begin(a, w0 / a.group);
    w.last = row.end(a, w1 / a.group);
    w.lo = row.begin(a, w1 / a.group);
    w.hi = row.end(a, w0 / a.group);
    // this part's tiles
    const int32_t base = w.wg_first & ~(int32_t)(kT - 1);
    const uint32_t tiles = ((uint32_t)(w.wg_last - base) + kT - 1) / kT;
    const int32_t j0 = base + (int32_t)((uint64_t)tiles * t.part / a.many_splits * kT);
    const int32_t j1 = base + (int32_t)((uint64_t)tiles * (t.part + 1) / a.many_splits * kT);
    // keys' dimensions behind the head's: zeros
    for (uint32_t x = a.d / 8 * kT + threadIdx.x; x < S::kBytes / 16; x += S::kThreads)
        *reinterpret_cast<u32x4 *>(k0 + x * 16) = *reinterpret_cast<u32x4 *>(k1 + x * 16) =
            *reinterpret_cast<u32x4 *>(k2 + x * 16) = u32x4{0, 0, 0, 0};
    Wave<KC> s;
    const uint32_t rr = min(t.r0 + 32 * wave + i, wg_last), tok = rr / a.group, head = t.kvh * a.group + rr % a.group;
    s.begin = row.begin(a, tok);
    s.end = row.end(a, tok);
    const uint16_t *q = a.q + (row.from + tok) * a.q_stride + head * a.d;
#pragma unroll
    for (int ks = 0; ks < 2 * KC; ++ks) s.q[ks] = load_q(a, q, 16 * ks + 8 * h);
    const uint32_t strange = run<KC>(a, w, s, k0, v0, k1, v1, k2, v2, j0, j1, wave, lane);
    s.sum += __shfl_xor(s.sum, 32);
    if (t.r0 + 32 * wave + i > wg_last) return;
    const uint64_t at = row.from + tok;
    if (a.many_splits == 1) {
        const float k = s.sum == 0.f ? 0.f : 1.f / s.sum;
        uint16_t *out = a.out + at * a.out_stride + head * a.d;
#pragma unroll
        for (int d = 0; d < KC; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const uint32_t dim = 32 * d + 2 * e + 4 * h;
                if (dim >= a.d) continue;
                float v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = s.sum == 0.f ? 0.f : s.o[d][e + x] * k;
                *reinterpret_cast<uint2 *>(out + dim) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
            }
        if (a.lse && h == 0) a.lse[at * a.q_heads + head] = lse_of(s.top, s.sum);
        if (strange && s.sum != 0.f)
            add_strange<KC>(a, w, s, j0, j1, h, [&](uint32_t dim, float v) { out[dim] = to_bf16(from_bf16(out[dim]) + v); });
    } else {
        const uint64_t p = (at * a.q_heads + head) * a.many_splits + t.part;
#pragma unroll
        for (int d = 0; d < KC; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const uint32_t dim = 32 * d + 2 * e + 4 * h;
                if (dim >= a.d) continue;
                *reinterpret_cast<f32x4 *>(a.many_o + p * a.d + dim) =
                    f32x4{s.o[d][e], s.o[d][e + 1], s.o[d][e + 2], s.o[d][e + 3]};
            }
        if (h == 0) a.many_ml[p] = make_float2(s.top, s.sum);
        if (strange) add_strange<KC>(a, w, s, j0, j1, h, [&](uint32_t dim, float v) { a.many_o[p * a.d + dim] += v; });
    }
}

}  // namespace

int launch_attend_many(const AttendArgs &a, hipStream_t stream) {
    AttendArgs args = a;
    void *p[] = {&args};
    auto go = [&](auto kc) {
        constexpr int KC = decltype(kc)::value;
        return hipLaunchKernel(reinterpret_cast<const void *>(&afx_attend_many_kernel<KC>),
                               dim3(a.kv_heads * a.many_tiles * a.many_splits), dim3(Shape<KC>::kThreads), p, 0,
                               stream) == hipSuccess
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
