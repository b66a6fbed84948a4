// afx_attend_many.hip -- attention of many query rows (chunks of prompts) over
// a paged cache (gfx950).
//
// The matrix cores bound it. A workgroup of 4 waves takes 128 query rows of
// one key-value head, 32 a wave, and its keys and values in tiles of 64
// tokens, which go from the pages to LDS without passing through registers
// and are double-buffered: the next tile is requested right after the barrier
// that frees its buffer. The pages' order is that of the operands, so that
// every LDS read is 16 bytes a lane, 512 in a row.
//   S^T = K Q^T    v_mfma_f32_32x32x16_bf16, K rows (tokens) as A, query rows
//                  as B: a lane holds 32 tokens' scores of one query row;
//   O^T += V^T P^T V^T rows (dimensions) as A, the weights as B.
// Rows 4 .. 7 and 8 .. 11 of every 16 score rows take each other's tokens, so
// that a half wave ends up with the scores of tokens 8 h .. 8 h + 7 of every
// 16, which is what it has to feed as B. The running maximum moves only when a
// score exceeds it by 8 (a factor 2^8), as in afx_attend_few.hip.
#include <type_traits>

#include "afx_attend.h"

namespace afx {
namespace {

constexpr uint32_t kWaves = 4, kThreads = 64 * kWaves;
constexpr float kSlack = 8.f;
constexpr uint32_t kT = kManyTokens;

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
__device__ inline bool find_tile(const AttendArgs &a, uint32_t u, Tile &t) {
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
        const uint32_t tiles = n > a.few_rows ? (n + kManyRows - 1) / kManyRows : 0;
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
            t.r0 = (end - 1 - u) * kManyRows;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Bytes of a key tile, [dim / 8][token] of 16, and of a value tile, [token / 8][dim] of 16.
constexpr uint32_t tile_bytes(int KC) { return 32 * KC / 8 * kT * 16; }

template <int KC>
struct Wave {
    bf16x8 q[2 * KC];
    f32x16 o[KC];
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

// The tile at position j, which lies in k_tile and v_tile; there: its tokens
// whose pages are in the cache.
template <int KC>
__device__ __forceinline__ void use_tile(const AttendArgs &a, const Where &w, Wave<KC> &s, uint8_t *k_tile,
                                         uint8_t *v_tile, int32_t j, uint64_t there, uint32_t lane) {
    constexpr uint32_t kDims = 32 * KC;
    const uint32_t i = lane & 31, h = lane >> 5;
    // a score row's token: rows 4 .. 7 and 8 .. 11 of 16 change places
    const uint32_t tok = (i & 16) | (i & 3) | ((i & 4) << 1) | ((i & 8) >> 1);
    bool strange = false;
    if (there != ~0ull || j < w.wg_lo || j + (int32_t)kT > w.wg_hi) {
        // A tile that some rows see in part: values of tokens that none sees become 0, and infinities and NaN
        // among the others are looked for.
        for (uint32_t x = threadIdx.x; x < 8 * kDims; x += kThreads) {
            u32x4 *p = reinterpret_cast<u32x4 *>(v_tile + x * 16);
            u32x4 v = *p;
            const uint32_t t8 = x / kDims * 8;
            uint32_t odd = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                auto seen = [&](uint32_t t) {
                    const int32_t at = j + (int32_t)t;
                    return (there >> t & 1) && at >= w.wg_first && at < w.wg_last;
                };
                v[e] &= (seen(t8 + 2 * e) ? 0xFFFFu : 0u) | (seen(t8 + 2 * e + 1) ? 0xFFFF0000u : 0u);
                odd |= (v[e] & 0x7F807F80u) + 0x00800080u;  // (only all ones carry into bit 15)
            }
            strange |= (odd & 0x80008000u) != 0;
            *p = v;
        }
        strange = __syncthreads_or(strange);
    }
    if (j >= w.last || j + (int32_t)kT <= w.first) return;  // no row of this wave sees the tile
    f32x16 sc[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) sc[x][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 2 * KC; ++ks)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const bf16x8 f = *reinterpret_cast<const bf16x8 *>(k_tile + ((2 * ks + h) * kT + 32 * x + tok) * 16);
            sc[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, s.q[ks], sc[x], 0, 0, 0);
        }
    const bool clean = there == ~0ull && j >= w.lo && j + (int32_t)kT <= w.hi;
    if (!clean) {
        // the lane's tokens of x, e: 8 h + t, t = 32 x + 16 (e / 8) + e mod 8
        const int32_t own = j + 8 * (int32_t)h;
        const uint32_t from = (uint32_t)max(s.begin - own, 0), n = (uint32_t)max(s.end - own - (int32_t)from, 0);
        const uint64_t pages = there >> (8 * h);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t t = 32 * x + 16 * (e / 8) + e % 8;
                if (t - from >= n || !(pages >> t & 1)) sc[x][e] = -INFINITY;
            }
    }
    float best = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) best = fmaxf(best, fmaxf(sc[0][e], sc[1][e]));
    best *= a.scale2;
    if (__any(best > s.top + kSlack)) {
        best = fmaxf(best, __shfl_xor(best, 32));
        const float now = fmaxf(s.top, best);
        const float f = now == -INFINITY ? 1.f : exp2_fast(s.top - now);
        s.top = now;
        s.sum *= f;
#pragma unroll
        for (int t = 0; t < KC; ++t) s.o[t] *= f;
    }
    const float base = s.top == -INFINITY ? 0.f : s.top;
    bf16x8 p[4];
    float part[4] = {};
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float v = exp2_fast(__builtin_fmaf(sc[x][e], a.scale2, -base));
            part[e % 4] += v;
            p[2 * x + e / 8][e % 8] = (__bf16)v;
        }
    s.sum += (part[0] + part[1]) + (part[2] + part[3]);
    if (strange) {
        // value by value, so that an infinity or NaN reaches only the rows that see it
        const uint32_t own = opaque(4 * h);
#pragma unroll 1
        for (uint32_t t = 0; t < kT; ++t) {
            const u32x4 bits = t / 16 == 0   ? __builtin_bit_cast(u32x4, p[0])
                               : t / 16 == 1 ? __builtin_bit_cast(u32x4, p[1])
                               : t / 16 == 2 ? __builtin_bit_cast(u32x4, p[2])
                                             : __builtin_bit_cast(u32x4, p[3]);
            const uint32_t two = t / 2 % 4 == 0 ? bits[0] : t / 2 % 4 == 1 ? bits[1] : t / 2 % 4 == 2 ? bits[2] : bits[3];
            const uint32_t got = __shfl(two, i + 32 * (t / 8 % 2));
            const float weight = from_bf16((uint16_t)(t % 2 ? got >> 16 : got));
            const int32_t at = j + (int32_t)t;
            if (!(there >> t & 1) || at < s.begin || at >= s.end) continue;
            const uint16_t *values = reinterpret_cast<const uint16_t *>(v_tile) + t / 8 * kDims * 8 + t % 8;
#pragma unroll
            for (int d = 0; d < KC; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t dim = 32 * d + (e & 3) + 8 * (e >> 2) + own;
                    s.o[d][e] += weight * from_bf16(values[dim * 8]);
                }
        }
        return;
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int d = 0; d < KC; ++d) {
            const bf16x8 f = *reinterpret_cast<const bf16x8 *>(v_tile + ((2 * ks + h) * kDims + 32 * d + i) * 16);
            s.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, p[ks], s.o[d], 0, 0, 0);
        }
}

// All tiles from j0 to j1. The four buffers are objects of their own: of one
// array the compiler would have every read wait for all loads into it.
template <int KC>
__device__ __forceinline__ void run(const AttendArgs &a, const Where &w, Wave<KC> &s, uint8_t *k0, uint8_t *v0,
                                    uint8_t *k1, uint8_t *v1, int32_t j0, int32_t j1, uint32_t wave, uint32_t lane) {
    constexpr uint32_t kDims = 32 * KC;
    const uint32_t pieces = a.d / 8;
    s.top = -INFINITY;
    s.sum = 0.f;
#pragma unroll
    for (int t = 0; t < KC; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) s.o[t][e] = 0.f;
    auto page_of = [&](int32_t at) {  // of the lane's token of the tile at `at`
        return (uint32_t)w.table[min(((uint32_t)at + lane) >> a.page_shift, a.max_pages - 1)];
    };
    // Wave w takes 1 KB pieces w, w + 4, .. of both tiles: 8 dimensions of 64 keys, 64 dimensions of 8 values (two
    // groups of 8 where a head's dimensions end inside a piece). Values behind the head's dimensions repeat its last.
    auto request = [&](int32_t at, uint32_t id, uint8_t *k_tile, uint8_t *v_tile) {
        const uint32_t safe = id < a.n_pages ? id : 0;
        const uint16_t *pk = w.k + (uint64_t)safe * w.page_elems + (((uint32_t)at + lane) & (w.size - 1)) * 8;
#pragma unroll
        for (int x = 0; x < KC; ++x) {
            const uint32_t piece = wave + kWaves * x;
            if (piece < pieces) load_to_lds(pk + piece * w.size * 8, k_tile + piece * 1024);
        }
#pragma unroll
        for (int x = 0; x < KC; ++x) {
            const uint32_t entry = (wave + kWaves * x) * 64 + lane, tok = entry / kDims * 8;
            const uint32_t page = __shfl(safe, tok);
            load_to_lds(w.v + (uint64_t)page * w.page_elems +
                            ((((uint32_t)at + tok) & (w.size - 1)) * a.d + min(entry % kDims, a.d - 1) * 8),
                        v_tile + (wave + kWaves * x) * 1024);
        }
    };
    uint32_t id = page_of(j0), id2 = page_of(j0 + kT);
    __syncthreads();  // (the keys' zeros)
    if (j0 < j1) request(j0, id, k0, v0);
    auto step = [&](int32_t j, uint8_t *k_tile, uint8_t *v_tile, uint8_t *k_next, uint8_t *v_next) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's loads have landed; then every wave's
        __syncthreads();
        const uint32_t id3 = page_of(j + 2 * kT);
        if (j + (int32_t)kT < j1) request(j + kT, id2, k_next, v_next);
        const uint64_t there = __ballot(id < a.n_pages);
        id = id2;
        id2 = id3;
        use_tile<KC>(a, w, s, k_tile, v_tile, j, there, lane);
    };
    for (int32_t j = j0; j < j1; j += 2 * kT) {
        step(j, k0, v0, k1, v1);
        if (j + (int32_t)kT < j1) step(j + kT, k1, v1, k0, v0);
    }
}

template <int KC>
__global__ __launch_bounds__(kThreads, KC <= 4 ? 2 : 1) void afx_attend_many_kernel(AttendArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t k0[tile_bytes(KC)], k1[tile_bytes(KC)], v0[tile_bytes(KC)], v1[tile_bytes(KC)];
    Tile t;
    const uint32_t u = blockIdx.x / a.kv_heads;
    t.kvh = blockIdx.x % a.kv_heads;  // (neighbouring workgroups, on different XCDs, read different heads)
    t.part = u % a.many_splits;
    if (!find_tile(a, u / a.many_splits, t)) return;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, i = lane & 31, h = lane >> 5;
    const BatchRow &row = t.row;
    const uint32_t wg_last = min(t.r0 + kManyRows, t.rows) - 1;
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
    for (uint32_t x = a.d / 8 * kT + threadIdx.x; x < 4 * KC * kT; x += kThreads)
        *reinterpret_cast<u32x4 *>(k0 + x * 16) = *reinterpret_cast<u32x4 *>(k1 + x * 16) = u32x4{0, 0, 0, 0};
    Wave<KC> s;
    const uint32_t rr = min(t.r0 + 32 * wave + i, wg_last), tok = rr / a.group, head = t.kvh * a.group + rr % a.group;
    s.begin = row.begin(a, tok);
    s.end = row.end(a, tok);
    const uint16_t *q = a.q + (row.from + tok) * a.q_stride + head * a.d;
#pragma unroll
    for (int ks = 0; ks < 2 * KC; ++ks) s.q[ks] = load_q(a, q, 16 * ks + 8 * h);
    run<KC>(a, w, s, k0, v0, k1, v1, j0, j1, wave, lane);
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
    }
}

}  // namespace

int launch_attend_many(const AttendArgs &a, hipStream_t stream) {
    AttendArgs args = a;
    void *p[] = {&args};
    auto go = [&](auto kc) {
        constexpr int KC = decltype(kc)::value;
        return hipLaunchKernel(reinterpret_cast<const void *>(&afx_attend_many_kernel<KC>),
                               dim3(a.kv_heads * a.many_tiles * a.many_splits), dim3(kThreads), p, 0,
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
