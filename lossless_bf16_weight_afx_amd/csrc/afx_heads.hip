// afx_heads.hip -- what stands between the q, k and v products and the
// attention (gfx950): the heads' norms, rotary positions with one or more
// axes, the rounding to BF16 and the write of keys and values to the cache's
// pages, in one pass; and the gradients of norms and rotation in one.
//
//   n = x k w, k = 1 / sqrt(mean(x^2) + eps), over a head's values
//   a' = n_a cos t - n_b sin t,  b' = n_b cos t + n_a sin t
// A rotation's transpose is the rotation by -t, so from dy (the gradient of
// the rotated head): dm = R(-t) dy, and with nh = x k
//   dw = sum over tokens and heads of dm nh
//   dx = k (dm w - nh mean(dm w nh))
//
// Memory bounds both: every value is read once and stays in registers. A
// head's values are four pairs a lane, on teams of 8 (head_dim <= 64), 16 or
// 32 lanes; values behind rot_dim form pairs too, which do not turn (a
// rotation by 0 would bring one's infinity to the other as NaN). A
// workgroup takes 16 tokens and 8 heads; the 16 tokens' angles are computed
// once and read from LDS by all of its heads, while the next head is on its
// way. Neighbouring teams of a wave take neighbouring tokens, whose 16-byte
// pieces of a page lie side by side; a value's 2 bytes go one by one. 4096
// tokens of 40 query and 8 key-value heads of 128 take 42 us, of which 8 are
// the values' and 4 the keys' writes (176 MB, 4.2 TB/s; a copy of as many
// bytes 31); the gradients of 2048 tokens 22 us, the sum of dw 4.
//
// Angles: position times frequency in turns, in FP64, of which the fraction is
// kept: at position 2^24 an FP32 product is off by half a radian.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "afx_paged.h"

namespace afx {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kTokens = 16;       // tokens of a workgroup at a time
constexpr uint32_t kHeadBlock = 8;     // heads of a workgroup
constexpr uint32_t kGradBlocks = 1024; // workgroups of the gradients' launch, about

struct HeadsArgs {
    const float *q, *k, *v;
    const uint16_t *dq, *dk;        // backward
    uint16_t *q_out, *k_out;        // backward: dq_in, dk_in
    uint16_t *k_pages, *v_pages;
    const int32_t *pos, *slots;
    const uint16_t *w_q, *w_k;
    const float *freq;
    const uint8_t *axis;
    float *part;                    // backward: [workgroups][head_dim] partial sums of dw
    uint64_t q_stride, k_stride, v_stride, dq_stride, dk_stride, qo_stride, ko_stride, pos_stride;
    uint32_t m, q_heads, kv_heads, d, rot, axes;
    uint32_t n_slots, page_shift;   // slots of the cache; tokens of a page: 1 << page_shift
    uint32_t tokens, head_block;    // of a workgroup at a time
    uint32_t q_blocks, k_blocks;    // head blocks of q and k (then those of v)
    float eps, inv_d;
};

__device__ inline uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ inline float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline uint32_t pack(float lo, float hi) { return to_bf16(lo) | ((uint32_t)to_bf16(hi) << 16); }

// A lane's four pairs of a head: where they are, and their accesses. With
// kVec the four firsts are 4 consecutive values at a multiple of 4, and so are
// the seconds (halves), or all 8 are consecutive (neighbours).
template <bool kNeighbours, bool kVec>
struct Pairs {
    uint32_t p, d, r2;  // first pair; head_dim; pairs that turn
    __device__ Pairs(const HeadsArgs &a, uint32_t lane) : p(4 * lane), d(a.d), r2(a.rot / 2) {}
    __device__ bool any() const { return p < d / 2; }
    // Pair e's new value y if it turns, else x: bit by bit, as the compiler makes a branch of a choice of floats (the
    // gradients of 333 tokens then take 11.9 us instead of 9.8).
    __device__ float turned(uint32_t e, float x, float y) const {
        const int mask = (kVec ? p : p + e) < r2 ? -1 : 0;  // (kVec: r2 is a multiple of 4)
        const int u = __float_as_int(x);
        return __int_as_float(u ^ ((u ^ __float_as_int(y)) & mask));
    }
    __device__ uint32_t first(uint32_t i) const {
        return kNeighbours ? 2 * i : i < r2 ? i : r2 + i;  // (behind rot: rot + i - r2)
    }
    __device__ uint32_t second(uint32_t i) const {
        return kNeighbours ? 2 * i + 1 : i < r2 ? i + r2 : d / 2 + i;  // (rot + i - r2 + (d - rot) / 2)
    }
    // (FP32 rows are read once: not kept in the caches, 4096 tokens take 42 us instead of 47)
    __device__ void load(const float *x, float (&a)[4], float (&b)[4]) const {
        typedef float f32x4 __attribute__((ext_vector_type(4)));
        auto four = [&](uint32_t i) { return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(x + i)); };
        if constexpr (kVec && kNeighbours) {
            const f32x4 u = four(2 * p), w = four(2 * p + 4);
            a[0] = u[0], b[0] = u[1], a[1] = u[2], b[1] = u[3];
            a[2] = w[0], b[2] = w[1], a[3] = w[2], b[3] = w[3];
        } else if constexpr (kVec) {
            const f32x4 u = four(first(p)), w = four(second(p));
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = u[e], b[e] = w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = x[first(p + e)], b[e] = x[second(p + e)];
        }
    }
    __device__ void load(const uint16_t *x, float (&a)[4], float (&b)[4]) const {
        if constexpr (kVec) {
            uint2 u, w;
            if constexpr (kNeighbours) {
                const uint4 all = *reinterpret_cast<const uint4 *>(x + 2 * p);
                u = make_uint2(all.x, all.y), w = make_uint2(all.z, all.w);
            } else {
                u = *reinterpret_cast<const uint2 *>(x + first(p)), w = *reinterpret_cast<const uint2 *>(x + second(p));
            }
            const float c[8] = {from_bf16(u.x), __uint_as_float(u.x & 0xFFFF0000u), from_bf16(u.y),
                                __uint_as_float(u.y & 0xFFFF0000u), from_bf16(w.x), __uint_as_float(w.x & 0xFFFF0000u),
                                from_bf16(w.y), __uint_as_float(w.y & 0xFFFF0000u)};
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = c[kNeighbours ? 2 * e : e], b[e] = c[kNeighbours ? 2 * e + 1 : 4 + e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = from_bf16(x[first(p + e)]), b[e] = from_bf16(x[second(p + e)]);
        }
    }
    // To x: value i of the head at x[i] (stride 8), or, in pieces of 8 values, at x[i / 8 stride + i % 8].
    __device__ void store(uint16_t *x, const float (&a)[4], const float (&b)[4], uint64_t stride = 8) const {
        auto at = [&](uint32_t i) { return x + i / 8 * stride + i % 8; };
        if constexpr (kVec && kNeighbours) {
            *reinterpret_cast<uint4 *>(at(2 * p)) =
                make_uint4(pack(a[0], b[0]), pack(a[1], b[1]), pack(a[2], b[2]), pack(a[3], b[3]));
        } else if constexpr (kVec) {
            *reinterpret_cast<uint2 *>(at(first(p))) = make_uint2(pack(a[0], a[1]), pack(a[2], a[3]));
            *reinterpret_cast<uint2 *>(at(second(p))) = make_uint2(pack(b[0], b[1]), pack(b[2], b[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) *at(first(p + e)) = to_bf16(a[e]), *at(second(p + e)) = to_bf16(b[e]);
        }
    }
};

// Cosines and sines of n tokens' angles from token t0 on: turn[token][pair].
__device__ inline void turns(const HeadsArgs &a, uint32_t t0, uint32_t n, float2 *turn) {
    const uint32_t pairs = a.d / 2, r2 = a.rot / 2;
    for (uint32_t i = threadIdx.x; i < n * pairs; i += kThreads) {
        const uint32_t t = i / pairs, p = i % pairs;
        float2 cs = make_float2(1.f, 0.f);
        if (p < r2) {
            const uint32_t axis = a.axis ? min((uint32_t)a.axis[p], a.axes - 1) : 0;
            const double rev = (double)a.pos[axis * a.pos_stride + t0 + t] * ((double)a.freq[p] * 0.15915494309189535);
            sincospif(2.f * (float)(rev - rint(rev)), &cs.y, &cs.x);
        }
        turn[i] = cs;
    }
}

// Sum over the lanes of a team (of 8, 16 or 32), the same in all of them: of
// pairs, of quads, of a half row's two quads, of a row's two halves (each
// mirrored onto the other), of two rows.
template <uint32_t kTeam>
__device__ inline float team_sum(float v) {
    auto from = [&](auto ctrl) {
        const int i = __float_as_int(v);
        return __int_as_float(__builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xF, 0xF, true));
    };
    v += from(std::integral_constant<int, 0xB1>{});
    v += from(std::integral_constant<int, 0x4E>{});
    v += from(std::integral_constant<int, 0x141>{});
    if (kTeam >= 16) v += from(std::integral_constant<int, 0x140>{});
    if (kTeam >= 32) v += __shfl_xor(v, 16);
    return v;
}

// The items team, team + kTeams, .. of n tokens by nh heads, tokens first.
template <uint32_t kTeams>
struct Items {
    uint32_t n, t, h, dt, dh;
    __device__ Items(uint32_t n, uint32_t team) : n(n), t(team % n), h(team / n), dt(kTeams % n), dh(kTeams / n) {}
    __device__ void next() {
        t += dt;
        h += dh;
        if (t >= n) t -= n, ++h;
    }
};

__device__ inline float sum8(const float (&a)[4], const float (&b)[4]) {
    return ((a[0] * a[0] + a[1] * a[1]) + (a[2] * a[2] + a[3] * a[3])) +
           ((b[0] * b[0] + b[1] * b[1]) + (b[2] * b[2] + b[3] * b[3]));
}

template <uint32_t kTeam, bool kNeighbours, bool kVec>
__global__ __launch_bounds__(kThreads) void afx_heads_kernel(HeadsArgs a) {
    __shared__ float2 turn[kTokens * 4 * kTeam];
    const uint32_t t0 = blockIdx.x * a.tokens, n = min(a.tokens, a.m - t0);
    const Pairs<kNeighbours, kVec> P(a, threadIdx.x % kTeam);
    const uint32_t team = threadIdx.x / kTeam;
    constexpr uint32_t kTeams = kThreads / kTeam;
    const uint32_t kind = blockIdx.y < a.q_blocks ? 0 : blockIdx.y < a.q_blocks + a.k_blocks ? 1 : 2;
    const uint32_t heads = kind ? a.kv_heads : a.q_heads;
    const uint32_t h0 = (blockIdx.y - (kind == 0 ? 0 : kind == 1 ? a.q_blocks : a.q_blocks + a.k_blocks)) * a.head_block;
    const uint32_t nh = min(a.head_block, heads - h0);
    const uint32_t size = 1u << a.page_shift;
    if (kind == 2) {
        for (Items<kTeams> i(n, team); i.h < nh; i.next()) {
            const uint32_t t = t0 + i.t, h = h0 + i.h;
            const uint32_t slot = (uint32_t)a.slots[t];
            if (slot >= a.n_slots || !P.any()) continue;
            float x[4], y[4];
            P.load(a.v + t * a.v_stride + h * a.d, x, y);
            const uint32_t off = slot % size;
            uint16_t *to = a.v_pages + (((uint64_t)(slot >> a.page_shift) * a.kv_heads + h) * size + (off & ~7u)) * a.d + off % 8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                to[8 * P.first(P.p + e)] = to_bf16(x[e]);
                to[8 * P.second(P.p + e)] = to_bf16(y[e]);
            }
        }
        return;
    }
    // Each head is loaded while the one before it is computed, the first one while the angles are.
    float nx[4] = {}, ny[4] = {};
    const float *first = (kind ? a.k + t0 * a.k_stride : a.q + t0 * a.q_stride) + h0 * a.d;
    const uint64_t stride = kind ? a.k_stride : a.q_stride;
    Items<kTeams> next(n, team);
    if (P.any() && next.h < nh) P.load(first + next.t * stride + next.h * a.d, nx, ny);
    turns(a, t0, n, turn);
    const uint16_t *w = kind ? a.w_k : a.w_q;
    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
    if (w && P.any()) P.load(w, wa, wb);
    __syncthreads();
    // (every lane of a team takes part in its sums)
    while (next.h < nh) {
        const uint32_t t = next.t, h = h0 + next.h;
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = nx[e], y[e] = ny[e];
        next.next();
        if (P.any() && next.h < nh) P.load(first + next.t * stride + next.h * a.d, nx, ny);
        if (w) {
            const float k = rsqrtf(team_sum<kTeam>(sum8(x, y)) * a.inv_d + a.eps);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= k * wa[e], y[e] *= k * wb[e];
        }
        if (!P.any()) continue;
        const float2 *cs = turn + t * (a.d / 2) + P.p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = x[e], v = y[e];
            x[e] = P.turned(e, u, u * cs[e].x - v * cs[e].y);
            y[e] = P.turned(e, v, v * cs[e].x + u * cs[e].y);
        }
        if (kind == 0) {
            P.store(a.q_out + (t0 + t) * a.qo_stride + h * a.d, x, y);
            continue;
        }
        if (a.k_out) P.store(a.k_out + (t0 + t) * a.ko_stride + h * a.d, x, y);
        if (!a.k_pages) continue;
        const uint32_t slot = (uint32_t)a.slots[t0 + t];
        if (slot < a.n_slots)
            P.store(a.k_pages + ((uint64_t)(slot >> a.page_shift) * a.kv_heads + h) * size * a.d + slot % size * 8, x, y,
                    size * 8);
    }
}

// Workgroup (x, y) takes the token blocks x, x + gridDim.x, .. of head block y
// and adds up dw over them; a second launch adds the workgroups' sums.
template <uint32_t kTeam, bool kNeighbours, bool kVec>
__global__ __launch_bounds__(kThreads) void afx_heads_grad_kernel(HeadsArgs a) {
    __shared__ float2 turn[kTokens * 4 * kTeam];
    constexpr uint32_t kTeams = kThreads / kTeam;
    const Pairs<kNeighbours, kVec> P(a, threadIdx.x % kTeam);
    const uint32_t team = threadIdx.x / kTeam;
    const bool keys = blockIdx.y >= a.q_blocks;
    const uint32_t heads = keys ? a.kv_heads : a.q_heads;
    const uint32_t h0 = (blockIdx.y - (keys ? a.q_blocks : 0)) * a.head_block, nh = min(a.head_block, heads - h0);
    const uint16_t *w = keys ? a.w_k : a.w_q;
    uint16_t *out = keys ? a.k_out : a.q_out;
    float wa[4] = {}, wb[4] = {}, da[4] = {}, db[4] = {};
    if (w && P.any()) P.load(w, wa, wb);
    for (uint64_t t0 = (uint64_t)blockIdx.x * a.tokens; t0 < a.m; t0 += (uint64_t)gridDim.x * a.tokens) {
        const uint32_t n = (uint32_t)min((uint64_t)a.tokens, a.m - t0);
        __syncthreads();  // (the last block's angles have been read)
        turns(a, (uint32_t)t0, n, turn);
        __syncthreads();
        for (Items<kTeams> i(n, team); i.h < nh; i.next()) {
            const uint32_t t = i.t, h = h0 + i.h;
            float x[4] = {}, y[4] = {}, ga[4] = {}, gb[4] = {};
            if (P.any()) {
                P.load((keys ? a.dk + (t0 + t) * a.dk_stride : a.dq + (t0 + t) * a.dq_stride) + h * a.d, ga, gb);
                if (w) P.load((keys ? a.k + (t0 + t) * a.k_stride : a.q + (t0 + t) * a.q_stride) + h * a.d, x, y);
                const float2 *cs = turn + t * (a.d / 2) + P.p;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = ga[e], v = gb[e];
                    ga[e] = P.turned(e, u, u * cs[e].x + v * cs[e].y);
                    gb[e] = P.turned(e, v, v * cs[e].x - u * cs[e].y);
                }
            }
            if (w) {
                const float k = rsqrtf(team_sum<kTeam>(sum8(x, y)) * a.inv_d + a.eps);
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] *= k, y[e] *= k;
                    da[e] += ga[e] * x[e], db[e] += gb[e] * y[e];
                    ga[e] *= wa[e], gb[e] *= wb[e];
                    dot += ga[e] * x[e] + gb[e] * y[e];
                }
                dot = team_sum<kTeam>(dot) * a.inv_d;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ga[e] = (ga[e] - x[e] * dot) * k;
                    gb[e] = (gb[e] - y[e] * dot) * k;
                }
            }
            if (out && P.any())
                P.store(out + (t0 + t) * (keys ? a.ko_stride : a.qo_stride) + h * a.d, ga, gb);
        }
    }
    if (!a.part || !w) return;
    // the teams' sums, in their order
    __shared__ float all[kTeams][8 * kTeam];
    if (P.any()) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            all[team][P.first(P.p + e)] = da[e];
            all[team][P.second(P.p + e)] = db[e];
        }
    }
    __syncthreads();
    float *to = a.part + ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.d;
    for (uint32_t c = threadIdx.x; c < a.d; c += kThreads) {
        float s = 0.f;
        for (uint32_t i = 0; i < kTeams; ++i) s += all[i][c];
        to[c] = s;
    }
}

// dw = the sum of the workgroups' sums: 32 slices a column, slice y adds those
// of workgroups y, y + 32, .. and the slices are added in their order.
constexpr uint32_t kSumSlices = 32, kSumCols = 8;
__global__ __launch_bounds__(kSumSlices *kSumCols) void afx_heads_sum_kernel(const float *part, uint32_t d,
                                                                             uint32_t n_q, uint32_t n_k, float *dw_q,
                                                                             float *dw_k) {
    __shared__ float s[kSumSlices][kSumCols + 1];
    const uint32_t c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
    float *out = blockIdx.y ? dw_k : dw_q;
    if (!out) return;
    const uint32_t n = blockIdx.y ? n_k : n_q;
    const float *in = part + (blockIdx.y ? (uint64_t)n_q * d : 0) + min(c, d - 1);
    float t = 0.f;
#pragma unroll 8
    for (uint32_t g = y; g < n; g += kSumSlices) t += in[(uint64_t)g * d];
    s[y][threadIdx.x % kSumCols] = t;
    __syncthreads();
    if (y == 0 && c < d) {
        for (uint32_t k = 1; k < kSumSlices; ++k) t += s[k][threadIdx.x];
        out[c] = t;
    }
}

// ---- launches ----------------------------------------------------------------
template <bool kGrad, uint32_t kTeam>
const void *heads_kernel(bool neighbours, bool vec) {
    auto pick = [](auto *f) { return reinterpret_cast<const void *>(f); };
    if constexpr (kGrad) {
        if (neighbours)
            return vec ? pick(&afx_heads_grad_kernel<kTeam, true, true>) : pick(&afx_heads_grad_kernel<kTeam, true, false>);
        return vec ? pick(&afx_heads_grad_kernel<kTeam, false, true>) : pick(&afx_heads_grad_kernel<kTeam, false, false>);
    } else {
        if (neighbours)
            return vec ? pick(&afx_heads_kernel<kTeam, true, true>) : pick(&afx_heads_kernel<kTeam, true, false>);
        return vec ? pick(&afx_heads_kernel<kTeam, false, true>) : pick(&afx_heads_kernel<kTeam, false, false>);
    }
}
template <bool kGrad>
int launch_heads(const afx_heads *p, HeadsArgs &a, dim3 grid, bool vec, void *stream) {
    const bool nb = p->pairing == AFX_ROPE_NEIGHBOURS;
    const void *fn = p->head_dim <= 64    ? heads_kernel<kGrad, 8>(nb, vec)
                     : p->head_dim <= 128 ? heads_kernel<kGrad, 16>(nb, vec)
                                          : heads_kernel<kGrad, 32>(nb, vec);
    void *args[] = {&a};
    return hipLaunchKernel(fn, grid, dim3(kThreads), args, 0, static_cast<hipStream_t>(stream)) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

uint32_t blocks_of(uint32_t heads, uint32_t block) { return (heads + block - 1) / block; }

// Token blocks of the gradients' launch: about kGradBlocks workgroups in all.
uint32_t grad_columns(const afx_heads *p, uint32_t m) {
    const uint32_t rows = blocks_of(p->q_heads, kHeadBlock) + blocks_of(p->kv_heads, kHeadBlock);
    return std::max(1u, std::min(blocks_of(m, kTokens), kGradBlocks / rows));
}
uint64_t grad_space(const afx_heads *p, uint32_t m) {
    return 4ull * grad_columns(p, m) * (blocks_of(p->q_heads, kHeadBlock) + blocks_of(p->kv_heads, kHeadBlock)) *
           p->head_dim;
}

// ---- argument checks ---------------------------------------------------------
int check_heads(const afx_heads *p) {
    if (!p || p->q_heads == 0 || p->kv_heads == 0 || p->q_heads > kMaxHeads || p->kv_heads > kMaxHeads ||
        p->head_dim == 0 || p->rot_dim > p->head_dim || p->rot_dim % 2 || p->pairing > AFX_ROPE_NEIGHBOURS ||
        p->n_axes == 0 || p->n_axes > 4 || (p->rot_dim && !p->freq) ||
        ((p->w_q || p->w_k) && (!(p->eps > 0.f) || !std::isfinite(p->eps))))
        return AFX_E_INVALID_ARG;
    if (p->head_dim % 8 || p->head_dim > AFX_MAX_HEAD_DIM) return AFX_E_UNSUPPORTED;
    return aligned({p->w_q, p->w_k}, 2) && aligned({p->freq}, 4) ? AFX_OK : AFX_E_MISALIGNED;
}

// A strided buffer of m rows of `width` elements.
struct Rows {
    const void *p;
    uint64_t width, stride, elem;
    RowSpan span(uint32_t m) const { return RowSpan{p, m, width * elem, stride * elem}; }
};
int check_rows(const Rows *r, size_t n, bool *vec) {
    for (size_t i = 0; i < n; ++i) {
        if (!r[i].p) continue;
        if (r[i].stride < r[i].width) return AFX_E_INVALID_ARG;
        if (r[i].stride >= kMaxRowStride) return AFX_E_UNSUPPORTED;
        if (!aligned({r[i].p}, r[i].elem)) return AFX_E_MISALIGNED;
        *vec &= r[i].stride % 8 == 0 && aligned({r[i].p}, 16);
    }
    return AFX_OK;
}

void fill(HeadsArgs &a, const afx_heads *p, uint32_t m, const int32_t *pos, uint64_t pos_stride) {
    a.pos = pos;
    a.pos_stride = pos_stride;
    a.w_q = p->w_q;
    a.w_k = p->w_k;
    a.freq = p->freq;
    a.axis = p->axis;
    a.m = m;
    a.q_heads = p->q_heads;
    a.kv_heads = p->kv_heads;
    a.d = p->head_dim;
    a.rot = p->rot_dim;
    a.axes = p->n_axes;
    a.eps = p->eps;
    a.inv_d = 1.f / (float)p->head_dim;
}

// What both calls read beside their rows: the positions and the parameters.
constexpr size_t kShared = 5;
void shared_spans(RowSpan *s, const afx_heads *p, uint32_t m, const int32_t *pos, uint64_t pos_stride) {
    s[0] = p->rot_dim ? RowSpan{pos, p->n_axes, 4ull * m, 4 * pos_stride} : RowSpan{nullptr, 0, 0, 0};
    s[1] = flat(p->w_q, 2ull * p->head_dim);
    s[2] = flat(p->w_k, 2ull * p->head_dim);
    s[3] = flat(p->freq, 2ull * p->rot_dim);
    s[4] = flat(p->axis, p->rot_dim / 2);
}
int check_pos(const afx_heads *p, uint32_t m, const int32_t *pos, uint64_t pos_stride) {
    if (p->rot_dim == 0) return AFX_OK;
    if (!pos || (p->n_axes > 1 && pos_stride < m)) return AFX_E_INVALID_ARG;
    if (pos_stride >= kMaxRowStride) return AFX_E_UNSUPPORTED;
    return aligned({pos}, 4) ? AFX_OK : AFX_E_MISALIGNED;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_heads_async(const afx_heads *p, uint32_t m, const int32_t *pos_dev, uint64_t pos_stride, const float *q_dev,
                    uint64_t q_stride, const float *k_dev, uint64_t k_stride, const float *v_dev, uint64_t v_stride,
                    uint16_t *q_out_dev, uint64_t q_out_stride, uint16_t *k_out_dev, uint64_t k_out_stride,
                    const afx_kv_pages *kv, const int32_t *slots_dev, void *stream) {
    int rc = check_heads(p);
    if (rc == AFX_OK && kv) rc = check_kv(kv);
    if (rc != AFX_OK) return rc;
    if (kv && (kv->kv_heads != p->kv_heads || kv->head_dim != p->head_dim)) return AFX_E_INVALID_ARG;
    if (m > kMaxTokens) return AFX_E_UNSUPPORTED;
    if (m == 0) return AFX_OK;
    if ((!q_dev && !k_dev && !v_dev) || !q_dev != !q_out_dev || (k_dev && !k_out_dev && !kv) || (k_out_dev && !k_dev) ||
        (v_dev && !kv) || !kv != !slots_dev || (kv && !k_dev && !v_dev))
        return AFX_E_INVALID_ARG;
    if (q_dev || k_dev) rc = check_pos(p, m, pos_dev, pos_stride);
    if (rc != AFX_OK) return rc;
    if (!aligned({slots_dev}, 4)) return AFX_E_MISALIGNED;
    const uint64_t nq = (uint64_t)p->q_heads * p->head_dim, nk = (uint64_t)p->kv_heads * p->head_dim;
    const Rows rows[] = {{q_out_dev, nq, q_out_stride, 2}, {k_out_dev, nk, k_out_stride, 2}, {q_dev, nq, q_stride, 4},
                         {k_dev, nk, k_stride, 4},         {v_dev, nk, v_stride, 4}};
    bool vec = p->rot_dim % 8 == 0 && aligned({p->w_q, p->w_k}, 16);
    rc = check_rows(rows, 5, &vec);
    if (rc != AFX_OK) return rc;
    RowSpan s[4 + 4 + kShared] = {rows[0].span(m),
                                  rows[1].span(m),
                                  kv && k_dev ? flat(kv->k_dev, kv_bytes(kv)) : RowSpan{nullptr, 0, 0, 0},
                                  kv && v_dev ? flat(kv->v_dev, kv_bytes(kv)) : RowSpan{nullptr, 0, 0, 0},
                                  rows[2].span(m),
                                  rows[3].span(m),
                                  rows[4].span(m),
                                  flat(slots_dev, 4ull * m)};
    shared_spans(s + 8, p, m, q_dev || k_dev ? pos_dev : nullptr, pos_stride);
    if (outputs_overlap(s, 4, 8 + kShared)) return AFX_E_INVALID_ARG;
    HeadsArgs a{};
    fill(a, p, m, pos_dev, pos_stride);
    a.q = q_dev;
    a.k = k_dev;
    a.v = v_dev;
    a.q_out = q_out_dev;
    a.k_out = k_out_dev;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.ko_stride = k_out_stride;
    a.slots = slots_dev;
    if (kv) {
        a.k_pages = kv->k_dev;
        a.v_pages = kv->v_dev;
        a.n_slots = kv->n_pages * kv->page_tokens;
        a.page_shift = (uint32_t)__builtin_ctz(kv->page_tokens);
    }
    a.tokens = std::min(m, kTokens);
    a.head_block = std::max(kHeadBlock, 16 / a.tokens);
    a.q_blocks = q_dev ? blocks_of(p->q_heads, a.head_block) : 0;
    a.k_blocks = k_dev ? blocks_of(p->kv_heads, a.head_block) : 0;
    const uint32_t v_blocks = v_dev ? blocks_of(p->kv_heads, a.head_block) : 0;
    return launch_heads<false>(p, a, dim3(blocks_of(m, a.tokens), a.q_blocks + a.k_blocks + v_blocks), vec, stream);
}

int afx_heads_workspace(const afx_heads *p, uint32_t m, size_t *bytes) {
    const int rc = check_heads(p);
    if (rc != AFX_OK) return rc;
    if (!bytes) return AFX_E_INVALID_ARG;
    if (m > kMaxTokens) return AFX_E_UNSUPPORTED;
    *bytes = grad_space(p, m);
    return AFX_OK;
}

int afx_heads_backward_async(const afx_heads *p, uint32_t m, const int32_t *pos_dev, uint64_t pos_stride,
                             const float *q_dev, uint64_t q_stride, const float *k_dev, uint64_t k_stride,
                             const uint16_t *dq_dev, uint64_t dq_stride, const uint16_t *dk_dev, uint64_t dk_stride,
                             uint16_t *dq_in_dev, uint64_t dq_in_stride, uint16_t *dk_in_dev, uint64_t dk_in_stride,
                             float *dw_q_dev, float *dw_k_dev, void *ws_dev, size_t ws_bytes, void *stream) {
    int rc = check_heads(p);
    if (rc != AFX_OK) return rc;
    if (m > kMaxTokens) return AFX_E_UNSUPPORTED;
    if ((dw_q_dev && !p->w_q) || (dw_k_dev && !p->w_k) || (!dq_in_dev && !dk_in_dev && !dw_q_dev && !dw_k_dev))
        return AFX_E_INVALID_ARG;
    const uint64_t nq = (uint64_t)p->q_heads * p->head_dim, nk = (uint64_t)p->kv_heads * p->head_dim;
    const bool do_q = dq_in_dev || dw_q_dev, do_k = dk_in_dev || dw_k_dev, sums = dw_q_dev || dw_k_dev;
    const uint64_t need = m && sums ? grad_space(p, m) : 0;
    if (m) {
        if ((do_q && (!dq_dev || (p->w_q && !q_dev))) || (do_k && (!dk_dev || (p->w_k && !k_dev))) || (need && !ws_dev))
            return AFX_E_INVALID_ARG;
        rc = check_pos(p, m, pos_dev, pos_stride);
        if (rc != AFX_OK) return rc;
    }
    if (!aligned({dw_q_dev, dw_k_dev}, 4) || (need && !aligned({ws_dev}, 16))) return AFX_E_MISALIGNED;
    const Rows rows[] = {{dq_in_dev, nq, dq_in_stride, 2},
                         {dk_in_dev, nk, dk_in_stride, 2},
                         {do_q ? dq_dev : nullptr, nq, dq_stride, 2},
                         {do_k ? dk_dev : nullptr, nk, dk_stride, 2},
                         {do_q && p->w_q ? q_dev : nullptr, nq, q_stride, 4},
                         {do_k && p->w_k ? k_dev : nullptr, nk, k_stride, 4}};
    bool vec = p->rot_dim % 8 == 0 && aligned({p->w_q, p->w_k}, 16);
    if (m) {
        rc = check_rows(rows, 6, &vec);
        if (rc != AFX_OK) return rc;
        // a gradient may be formed in place: then its input is no other buffer
        const bool q_in_place = dq_in_dev && dq_in_dev == rows[2].p && dq_in_stride == dq_stride;
        const bool k_in_place = dk_in_dev && dk_in_dev == rows[3].p && dk_in_stride == dk_stride;
        const RowSpan none{nullptr, 0, 0, 0};
        RowSpan s[5 + 4 + kShared] = {rows[0].span(m),
                                      rows[1].span(m),
                                      flat(dw_q_dev, 4ull * p->head_dim),
                                      flat(dw_k_dev, 4ull * p->head_dim),
                                      flat(ws_dev, need),
                                      q_in_place ? none : rows[2].span(m),
                                      k_in_place ? none : rows[3].span(m),
                                      rows[4].span(m),
                                      rows[5].span(m)};
        shared_spans(s + 9, p, m, pos_dev, pos_stride);
        if (outputs_overlap(s, 5, 9 + kShared)) return AFX_E_INVALID_ARG;
    } else {
        const RowSpan s[] = {flat(dw_q_dev, 4ull * p->head_dim), flat(dw_k_dev, 4ull * p->head_dim)};
        if (outputs_overlap(s, 2, 2)) return AFX_E_INVALID_ARG;
    }
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
    HeadsArgs a{};
    fill(a, p, m, pos_dev, pos_stride);
    a.q = q_dev;
    a.k = k_dev;
    a.dq = dq_dev;
    a.dk = dk_dev;
    a.q_out = dq_in_dev;
    a.k_out = dk_in_dev;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.qo_stride = dq_in_stride;
    a.ko_stride = dk_in_stride;
    a.part = need ? static_cast<float *>(ws_dev) : nullptr;
    a.tokens = std::min(m, kTokens);
    a.head_block = kHeadBlock;
    a.q_blocks = do_q ? blocks_of(p->q_heads, kHeadBlock) : 0;
    a.k_blocks = do_k ? blocks_of(p->kv_heads, kHeadBlock) : 0;
    const uint32_t cols = m ? grad_columns(p, m) : 0;
    if (m) {
        rc = launch_heads<true>(p, a, dim3(cols, a.q_blocks + a.k_blocks), vec, stream);
        if (rc != AFX_OK) return rc;
    }
    if (!sums) return AFX_OK;
    uint32_t n_q = cols * a.q_blocks, n_k = cols * a.k_blocks;
    void *args[] = {&a.part, &a.d, &n_q, &n_k, &dw_q_dev, &dw_k_dev};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_heads_sum_kernel),
                           dim3((a.d + kSumCols - 1) / kSumCols, 2), dim3(kSumSlices * kSumCols), args, 0,
                           static_cast<hipStream_t>(stream)) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

}  // extern "C"
