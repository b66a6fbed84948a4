// afx_norm.hip -- what stands between two blocks of a layer (gfx950): the
// norm after the first block, its gate and residual scale, the residual add,
// and the norm before the second, in one pass; and its gradients in one.
//
//   bh = b k w_post,  k = 1 / sqrt(mean(b^2) + eps)
//   r' = r + s gate bh
//   xn = r' k' w_pre, k' = 1 / sqrt(mean(r'^2) + eps)
//
// With n = v k, the gradient of v through n, given dn, is k (dn - n mean(dn
// n)). So, from dxn and dr_out (the gradients of xn and r'):
//   dr      = dr_out + k' (dxn w_pre - n' mean(dxn w_pre n')),  n' = r' k'
//   dw_pre  = sum over rows of dxn n'
//   dbh     = s gate dr,   dgate = s bh dr (summed over rows for a shared gate)
//   dw_post = sum over rows of dbh n,  n = b k
//   db      = k (dbh w_post - n mean(dbh w_post n))
//
// Memory bounds both: every value is read once and held in registers (FP32)
// between the sums and the outputs. A team of 16 lanes (d <= 128), a wave
// (d <= 512) or a workgroup of up to 16 waves takes a row; each lane holds 8
// values, 16 for d > 8192, 32 for d > 16384. (The gradients keep nine values
// for each; 32 of them do not fit the registers: 1024 x 16384, BF16, 342 us
// with 32, 124 with 16; 1024 x 32768, where they must, 622.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "afx_internal.h"

namespace afx {
namespace {

constexpr uint32_t kTeamThreads = 256;  // threads of a workgroup of small teams
constexpr uint32_t kMaxTeamWaves = 16;

struct NormArgs {
    const float *b;
    const void *r;           // forward: r; backward: r'
    void *r_out;             // forward
    uint16_t *xn;            // forward
    const uint16_t *dxn;     // backward
    const void *dr_out;      // backward
    void *dr;                // backward
    uint16_t *db;            // backward
    float *part;             // backward: [workgroups][3][d] partial sums, or NULL
    float *dgate_rows;       // backward: FP32 [m, d] of a gate per row
    const uint16_t *w_post, *gate, *w_pre;
    uint64_t b_stride, r_stride, ro_stride, xn_stride, dxn_stride, dro_stride, dr_stride, db_stride, gate_stride;
    uint32_t m, d;
    float eps, scale, inv_d;
};

__device__ inline float bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ inline uint32_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// The lane's 8 I values of a row: with kVec, I chunks of 8 consecutive ones,
// else single ones a team apart. Values past the row are 0 and not stored.
template <uint32_t kTeam, bool kVec, int I>
struct Lanes {
    uint32_t lane, team, d;
    __device__ uint32_t at(int i, int e) const {
        return kVec ? 8 * (lane + (uint32_t)i * team) + (uint32_t)e : lane + (uint32_t)(8 * i + e) * team;
    }
    // The lane's values of a row as loaded: from the row's first values where
    // it has none of its own, so that no load waits behind a branch.
    template <class T>
    struct Raw {
        static constexpr int kParts = kVec ? 8 * I * (int)sizeof(T) / 16 : 8 * I;
        std::conditional_t<kVec, uint4, T> part[kParts];
    };
    template <class T>
    __device__ Raw<T> fetch(const T *p) const {
        Raw<T> raw;
        constexpr int kEach = Raw<T>::kParts / I;  // parts of 8 values
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if constexpr (kVec) {
                    const uint32_t c = at(i, 0) < d ? at(i, 0) : 0;
                    raw.part[kEach * i + k] = reinterpret_cast<const uint4 *>(p + c)[k];
                } else {
                    raw.part[kEach * i + k] = p[at(i, k) < d ? at(i, k) : 0];
                }
            }
        return raw;
    }
    template <class T, class F>
    __device__ void each(const Raw<T> &raw, F &&put) const {
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v;
                if constexpr (!kVec) {
                    if constexpr (sizeof(T) == 4)
                        v = raw.part[8 * i + e];
                    else
                        v = bf16(raw.part[8 * i + e]);
                } else {
                    constexpr int kPer = 16 / (int)sizeof(T);  // values of a part
                    const uint4 &q = raw.part[(8 * i + e) / kPer];
                    const int w = e % kPer * (int)sizeof(T) / 4;
                    const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
                    v = sizeof(T) == 4 ? __uint_as_float(u)
                        : e % 2        ? __uint_as_float(u & 0xFFFF0000u)
                                       : bf16(u & 0xFFFFu);
                }
                put(8 * i + e, at(i, e) < d ? v : 0.f);
            }
    }
    template <class T, class F>
    __device__ void load(const T *p, F &&put) const {
        each(fetch(p), put);
    }
    template <class F>
    __device__ void store(float *p, F &&get) const {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if constexpr (kVec) {
                if (at(i, 0) < d) {
                    *reinterpret_cast<float4 *>(p + at(i, 0)) =
                        make_float4(get(8 * i), get(8 * i + 1), get(8 * i + 2), get(8 * i + 3));
                    *reinterpret_cast<float4 *>(p + at(i, 0) + 4) =
                        make_float4(get(8 * i + 4), get(8 * i + 5), get(8 * i + 6), get(8 * i + 7));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at(i, e) < d) p[at(i, e)] = get(8 * i + e);
            }
        }
    }
    template <class F>
    __device__ void store(uint16_t *p, F &&get) const {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if constexpr (kVec) {
                if (at(i, 0) < d) {
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = to_bf16(get(8 * i + 2 * e)) | (to_bf16(get(8 * i + 2 * e + 1)) << 16);
                    *reinterpret_cast<uint4 *>(p + at(i, 0)) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at(i, e) < d) p[at(i, e)] = (uint16_t)to_bf16(get(8 * i + e));
            }
        }
    }
};

// Sum of N values over the team (16 lanes, a wave, or kTeam = 0: the
// workgroup, through LDS; every wave adds the waves' sums in the same order).
template <uint32_t kTeam, int N>
__device__ inline void team_sum(float (&v)[N], float (*lds)[kMaxTeamWaves]) {
    constexpr uint32_t kLanes = kTeam == 16 ? 16 : 64;
#pragma unroll
    for (uint32_t o = 1; o < kLanes; o *= 2)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], (int)o);
    if constexpr (kTeam == 0) {
        const uint32_t wave = threadIdx.x / 64, waves = blockDim.x / 64;
        __syncthreads();  // the last sums have been read
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) lds[k][wave] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.f;
            for (uint32_t w = 0; w < waves; ++w) v[k] += lds[k][w];
        }
    }
}

template <uint32_t kTeam, bool kVec, int I, class R>
__global__ __launch_bounds__(kTeam ? kTeamThreads : 1024) void afx_norm_kernel(const NormArgs p) {
    __shared__ float sums[1][kMaxTeamWaves];
    constexpr int N = 8 * I;
    const uint32_t team = kTeam ? kTeam : blockDim.x;
    const uint32_t teams = kTeam ? kTeamThreads / team : 1;
    const Lanes<kTeam, kVec, I> L{threadIdx.x % team, team, p.d};
    for (uint64_t row = (uint64_t)blockIdx.x * teams + threadIdx.x / team; row < p.m;
         row += (uint64_t)gridDim.x * teams) {
        float v[N];
        L.load(static_cast<const R *>(p.r) + row * p.r_stride, [&](int e, float x) { v[e] = x; });
        if (p.b) {
            float b[N];
            L.load(p.b + row * p.b_stride, [&](int e, float x) { b[e] = x; });
            if (p.w_post) {
                float s[1] = {0.f};
#pragma unroll
                for (int e = 0; e < N; ++e) s[0] = fmaf(b[e], b[e], s[0]);
                team_sum<kTeam>(s, sums);
                const float k = rsqrtf(s[0] * p.inv_d + p.eps);
                L.load(p.w_post, [&](int e, float x) { b[e] = b[e] * k * x; });
            }
            if (p.gate) L.load(p.gate + row * p.gate_stride, [&](int e, float x) { b[e] *= x; });
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = fmaf(p.scale, b[e], v[e]);
        }
        if (p.r_out) L.store(static_cast<R *>(p.r_out) + row * p.ro_stride, [&](int e) { return v[e]; });
        if (p.xn) {
            float s[1] = {0.f};
#pragma unroll
            for (int e = 0; e < N; ++e) s[0] = fmaf(v[e], v[e], s[0]);
            team_sum<kTeam>(s, sums);
            const float k = rsqrtf(s[0] * p.inv_d + p.eps);
            L.load(p.w_pre, [&](int e, float x) { v[e] = v[e] * k * x; });
            L.store(p.xn + row * p.xn_stride, [&](int e) { return v[e]; });
        }
    }
}

// Gradients. A workgroup goes through its rows with the sums over rows
// (dw_pre, dw_post, a shared gate's dgate) in registers and writes them once,
// for afx_norm_sum_kernel to add up in the order of the workgroups.
//
// For rows of up to 8192 values the next row is requested before this one is
// worked on (registers: 28, or 32 for single values), and the vectors w_post,
// w_pre and a shared gate are kept in LDS: read from memory in between, they
// would wait for that row, loads being counted in order. (4096 rows of 5120,
// FP32 stream: 109 us without, 126 with the request alone, 99 with both.)
template <uint32_t kTeam, bool kVec, int I, class R, uint32_t kThreads>
__global__ __launch_bounds__(kThreads) void afx_norm_grad_kernel(const NormArgs p) {
    __shared__ float sums[3][kMaxTeamWaves];
    constexpr int N = 8 * I;
    constexpr bool kAhead = I == 1;
    const uint32_t team = kTeam ? kTeam : blockDim.x;
    const uint32_t teams = kTeam ? kTeamThreads / team : 1;
    using Row = Lanes<kTeam, kVec, I>;
    const Row L{threadIdx.x % team, team, p.d};
    struct In {  // what a turn reads of its row
        typename Row::template Raw<R> r, dr_out;
        typename Row::template Raw<float> b;
        typename Row::template Raw<uint16_t> dxn;
    };
    auto fetch = [&](uint64_t row0) {
        const uint64_t row = row0 + threadIdx.x / team, rr = row < p.m ? row : 0;
        In in;
        in.r = L.fetch(static_cast<const R *>(p.r) + rr * p.r_stride);
        if (p.b) in.b = L.fetch(p.b + rr * p.b_stride);
        if (p.dr_out) in.dr_out = L.fetch(static_cast<const R *>(p.dr_out) + rr * p.dro_stride);
        if (p.dxn) in.dxn = L.fetch(p.dxn + rr * p.dxn_stride);
        return in;
    };
    const uint64_t step = (uint64_t)gridDim.x * teams;
    uint64_t row0 = (uint64_t)blockIdx.x * teams;
    In in, next;
    const uint16_t *w_pre = p.w_pre, *w_post = p.w_post, *gate = p.gate;
    if constexpr (kAhead) {
        __shared__ __attribute__((aligned(16))) uint16_t vectors[3][kTeam ? 8 * kTeam : 8 * kThreads];
        const uint16_t *from[3] = {p.w_pre, p.w_post, p.gate_stride ? nullptr : p.gate};
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (from[k])
                for (uint32_t c = threadIdx.x; c < p.d; c += blockDim.x) vectors[k][c] = from[k][c];
        if (row0 < p.m) next = fetch(row0);
        __syncthreads();
        w_pre = vectors[0];
        w_post = vectors[1];
        if (!p.gate_stride) gate = vectors[2];
    }
    float dw_pre[N] = {}, dw_post[N] = {}, dgate[N] = {};
    // every lane takes every turn: the sums below are over whole waves
    for (; row0 < p.m; row0 += step) {
        const uint64_t row = row0 + threadIdx.x / team;
        const bool ok = row < p.m;
        if constexpr (kAhead) {
            in = next;
            if (row0 + step < p.m) next = fetch(row0 + step);
        } else {
            in = fetch(row0);
        }
        float v[N], dr[N], b[N];
        float s[3] = {0.f, 0.f, 0.f};  // r'^2, dxn w_pre r', b^2
#pragma unroll
        for (int e = 0; e < N; ++e) dr[e] = b[e] = 0.f;
        L.each(in.r, [&](int e, float x) { v[e] = x; });
        if (p.b) L.each(in.b, [&](int e, float x) { b[e] = x; });
        if (p.dr_out) L.each(in.dr_out, [&](int e, float x) { dr[e] = x; });
        if (p.dxn) {
            float dn[N], dx[N];
            L.each(in.dxn, [&](int e, float x) { dx[e] = x; });
            L.load(w_pre, [&](int e, float x) { dn[e] = dx[e] * x; });
#pragma unroll
            for (int e = 0; e < N; ++e) {
                s[0] = fmaf(v[e], v[e], s[0]);
                s[1] = fmaf(dn[e], v[e], s[1]);
                s[2] = fmaf(b[e], b[e], s[2]);
            }
            team_sum<kTeam>(s, sums);
            const float k = rsqrtf(s[0] * p.inv_d + p.eps);
            const float c = s[1] * p.inv_d * k * k;  // mean(dn n') k'
#pragma unroll
            for (int e = 0; e < N; ++e) {
                dr[e] += k * (dn[e] - c * v[e]);
                if (ok) dw_pre[e] = fmaf(dx[e], v[e] * k, dw_pre[e]);
            }
        } else if (p.b && p.w_post) {
            float t[1] = {0.f};
#pragma unroll
            for (int e = 0; e < N; ++e) t[0] = fmaf(b[e], b[e], t[0]);
            team_sum<kTeam>(t, sums);
            s[2] = t[0];
        }
        if (ok && p.dr) L.store(static_cast<R *>(p.dr) + row * p.dr_stride, [&](int e) { return dr[e]; });
        if (!p.b) continue;
        // v: the gradient of bh from here on
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = dr[e] * p.scale;
        const float k = p.w_post ? rsqrtf(s[2] * p.inv_d + p.eps) : 1.f;
        if (p.gate) {
            float bh[N];
#pragma unroll
            for (int e = 0; e < N; ++e) bh[e] = b[e] * k;
            if (p.w_post) L.load(w_post, [&](int e, float x) { bh[e] *= x; });
            if (p.dgate_rows) {
                if (ok) L.store(p.dgate_rows + row * p.d, [&](int e) { return bh[e] * v[e]; });
            } else if (ok) {
#pragma unroll
                for (int e = 0; e < N; ++e) dgate[e] = fmaf(bh[e], v[e], dgate[e]);
            }
            L.load(gate + (ok ? row : 0) * p.gate_stride, [&](int e, float x) { v[e] *= x; });
        }
        if (p.w_post) {
            float t[1] = {0.f};
            if (ok) {
#pragma unroll
                for (int e = 0; e < N; ++e) dw_post[e] = fmaf(v[e], b[e] * k, dw_post[e]);
            }
            L.load(w_post, [&](int e, float x) { v[e] *= x; });
#pragma unroll
            for (int e = 0; e < N; ++e) t[0] = fmaf(v[e], b[e], t[0]);
            team_sum<kTeam>(t, sums);
            const float c = t[0] * p.inv_d * k * k;
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = k * (v[e] - c * b[e]);
        }
        if (ok && p.db) L.store(p.db + row * p.db_stride, [&](int e) { return v[e]; });
    }
    if (!p.part) return;
    float *out = p.part + (uint64_t)blockIdx.x * 3 * p.d;
    if constexpr (kTeam == 0) {
        L.store(out, [&](int e) { return dw_pre[e]; });
        L.store(out + p.d, [&](int e) { return dw_post[e]; });
        L.store(out + 2 * p.d, [&](int e) { return dgate[e]; });
    } else {
        // the workgroup's teams add up in LDS, in their order
        __shared__ float all[kTeamThreads / kTeam][8 * kTeam];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            __syncthreads();
            float *mine = all[threadIdx.x / kTeam];
#pragma unroll
            for (int e = 0; e < N; ++e) mine[L.at(0, e)] = q == 0 ? dw_pre[e] : q == 1 ? dw_post[e] : dgate[e];
            __syncthreads();
            for (uint32_t c = threadIdx.x; c < p.d; c += kTeamThreads) {
                float t = 0.f;
                for (uint32_t w = 0; w < kTeamThreads / kTeam; ++w) t += all[w][c];
                out[q * p.d + c] = t;
            }
        }
    }
}

// out[q] = sum over the workgroups' partial sums. 32 slices per column: slice y
// adds those of workgroups y, y + 32, .. in that order, and the slices are
// added in theirs.
constexpr uint32_t kSumSlices = 32, kSumCols = 32;
__global__ __launch_bounds__(kSumSlices *kSumCols) void afx_norm_sum_kernel(const float *part, uint32_t groups,
                                                                            uint32_t d, float *o0, float *o1,
                                                                            float *o2) {
    __shared__ float s[kSumSlices][kSumCols + 1];
    const uint32_t q = blockIdx.y, c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
    float *o = q == 0 ? o0 : q == 1 ? o1 : o2;
    if (!o) return;
    float t = 0.f;
    const float *in = part + (uint64_t)q * d + min(c, d - 1);
    constexpr uint32_t kAtOnce = 8;  // loads in flight; those past the last add 0
    for (uint32_t g = y; g < groups; g += kAtOnce * kSumSlices) {
        float v[kAtOnce];
#pragma unroll
        for (uint32_t k = 0; k < kAtOnce; ++k) v[k] = in[(uint64_t)min(g + k * kSumSlices, groups - 1) * 3 * d];
#pragma unroll
        for (uint32_t k = 0; k < kAtOnce; ++k) t += g + k * kSumSlices < groups ? v[k] : 0.f;
    }
    s[y][threadIdx.x % kSumCols] = t;
    __syncthreads();
    if (y == 0 && c < d) {
        for (uint32_t k = 1; k < kSumSlices; ++k) t += s[k][threadIdx.x];
        o[c] = t;
    }
}

// Threads that share a row, and workgroups of a launch.
struct NormShape {
    uint32_t team, threads, teams, iters;
};
NormShape norm_shape(uint64_t d) {
    if (d <= 128) return {16, kTeamThreads, kTeamThreads / 16, 1};
    if (d <= 512) return {64, kTeamThreads, kTeamThreads / 64, 1};
    const uint32_t iters = d <= 8192 ? 1 : d <= 16384 ? 2 : 4;
    const uint32_t threads = (uint32_t)((d + 8 * iters * 64 - 1) / (8 * iters * 64) * 64);
    return {0, threads, 1, iters};
}
uint32_t norm_blocks(const NormShape &s, uint32_t m, uint32_t most) {
    return (uint32_t)std::min<uint64_t>(((uint64_t)m + s.teams - 1) / s.teams, most);
}
constexpr uint32_t kForwardBlocks = 8192;
// Workgroups of the gradients' launch, each with its sums over its rows: one
// on a CU from 9 waves on, more where they are small (4096 rows of 1024, 2
// waves each: 37 us with 1024 workgroups, 44 with 512; of 500 values, 4 waves:
// 20 and 18).
uint32_t grad_blocks(const NormShape &s, uint32_t m) {
    return norm_blocks(s, m, s.threads > 512 ? 256 : s.threads > 128 ? 512 : 1024);
}

template <bool kGrad, uint32_t kTeam, bool kVec, int I, uint32_t kThreads>
const void *norm_kernel(bool fp32) {
    if constexpr (kGrad)
        return fp32 ? reinterpret_cast<const void *>(&afx_norm_grad_kernel<kTeam, kVec, I, float, kThreads>)
                    : reinterpret_cast<const void *>(&afx_norm_grad_kernel<kTeam, kVec, I, uint16_t, kThreads>);
    else
        return fp32 ? reinterpret_cast<const void *>(&afx_norm_kernel<kTeam, kVec, I, float>)
                    : reinterpret_cast<const void *>(&afx_norm_kernel<kTeam, kVec, I, uint16_t>);
}
template <bool kGrad, bool kVec>
const void *norm_kernel(const NormShape &s, bool fp32) {
    if (s.team == 16) return norm_kernel<kGrad, 16, kVec, 1, kTeamThreads>(fp32);
    if (s.team == 64) return norm_kernel<kGrad, 64, kVec, 1, kTeamThreads>(fp32);
    if (s.iters == 2) return norm_kernel<kGrad, 0, kVec, 2, 1024>(fp32);
    if (s.iters == 4) return norm_kernel<kGrad, 0, kVec, 4, 1024>(fp32);
    // (a workgroup of at most 12 waves has 168 registers a lane, one of 16 has 128)
    return s.threads <= 768 ? norm_kernel<kGrad, 0, kVec, 1, 768>(fp32) : norm_kernel<kGrad, 0, kVec, 1, 1024>(fp32);
}
template <bool kGrad>
int launch_norm(NormArgs &a, const NormShape &s, uint32_t blocks, bool vec, bool fp32, hipStream_t stream) {
    const void *fn = vec ? norm_kernel<kGrad, true>(s, fp32) : norm_kernel<kGrad, false>(s, fp32);
    void *args[] = {&a};
    return hipLaunchKernel(fn, dim3(blocks), dim3(s.threads), args, 0, stream) == hipSuccess ? AFX_OK : AFX_E_HIP;
}

// ---- argument checks ---------------------------------------------------------
struct Rows {  // one strided buffer of a call
    const void *p;
    uint64_t stride, elem;
    bool out;
};

int check_norm(const afx_block_norm *p) {
    if (!p || p->d == 0 || !(p->eps > 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->scale) ||
        p->r_type > AFX_TYPE_FP32)
        return AFX_E_INVALID_ARG;
    if (p->d > AFX_MAX_NORM_WIDTH) return AFX_E_UNSUPPORTED;
    if (p->gate && p->gate_stride && p->gate_stride < p->d) return AFX_E_INVALID_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(p->w_post) | reinterpret_cast<uintptr_t>(p->gate) |
                          reinterpret_cast<uintptr_t>(p->w_pre);
    return all & 1 ? AFX_E_MISALIGNED : AFX_OK;
}

constexpr uint64_t kMaxNormStride = 1ull << 28;  // (2^32 rows of them stay below 2^64 bytes)

RowSpan span(const Rows &r, uint32_t m, uint64_t d) {  // (stride 0: one row for all)
    return RowSpan{r.p, r.stride || m == 0 ? m : 1, d * r.elem, r.stride * r.elem};
}

// Strides, alignment, overlap (in_place: the pair of indices that may be one
// buffer), and whether every row can be accessed 8 values at a time.
int check_rows(const Rows *r, size_t n, uint32_t m, uint64_t d, size_t in0, size_t in1, bool *vec) {
    *vec = d % 8 == 0;
    for (size_t i = 0; i < n; ++i) {
        if (!r[i].p) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(r[i].p);
        if (r[i].stride && r[i].stride < d) return AFX_E_INVALID_ARG;
        if (r[i].stride >= kMaxNormStride) return AFX_E_UNSUPPORTED;
        if (at & (r[i].elem - 1)) return AFX_E_MISALIGNED;
        *vec &= r[i].stride % 8 == 0 && (at & 15) == 0;
    }
    for (size_t i = 0; i < n; ++i)
        for (size_t k = 0; k < n; ++k) {
            if (i == k || !r[i].out || !rows_overlap(span(r[i], m, d), span(r[k], m, d))) continue;
            const bool pair = (i == in0 && k == in1) || (i == in1 && k == in0);
            if (!pair || r[i].p != r[k].p || r[i].stride != r[k].stride) return AFX_E_INVALID_ARG;
        }
    return AFX_OK;
}

// Workgroups of the gradients' launch, and their partial sums.
uint64_t norm_space(const afx_block_norm *p, uint32_t m) {
    return (uint64_t)grad_blocks(norm_shape(p->d), m) * 3 * p->d * 4;
}

}  // namespace
}  // namespace afx

using namespace afx;

extern "C" {

int afx_block_norm_async(const afx_block_norm *p, uint32_t m, const float *b_dev, uint64_t b_stride, const void *r_dev,
                         uint64_t r_stride, void *r_out_dev, uint64_t r_out_stride, uint16_t *xn_dev,
                         uint64_t xn_stride, void *stream) {
    int rc = check_norm(p);
    if (rc != AFX_OK) return rc;
    if (!p->w_pre != !xn_dev || (b_dev && !r_out_dev) || (!r_out_dev && !xn_dev)) return AFX_E_INVALID_ARG;
    if (m == 0) return AFX_OK;
    if (!r_dev) return AFX_E_INVALID_ARG;
    if ((b_dev && b_stride < p->d) || r_stride < p->d || (r_out_dev && r_out_stride < p->d) ||
        (xn_dev && xn_stride < p->d))
        return AFX_E_INVALID_ARG;
    const uint64_t rb = p->r_type == AFX_TYPE_FP32 ? 4 : 2;
    const uint16_t *w_post = b_dev ? p->w_post : nullptr, *gate = b_dev ? p->gate : nullptr;
    const Rows rows[] = {{b_dev, b_stride, 4, false},   {r_dev, r_stride, rb, false},
                         {r_out_dev, r_out_stride, rb, true}, {xn_dev, xn_stride, 2, true},
                         {w_post, 0, 2, false},         {gate, p->gate_stride, 2, false},
                         {p->w_pre, 0, 2, false}};
    bool vec = false;
    rc = check_rows(rows, 7, m, p->d, 1, 2, &vec);
    if (rc != AFX_OK) return rc;
    NormArgs a{};
    a.b = b_dev;
    a.r = r_dev;
    a.r_out = r_out_dev;
    a.xn = xn_dev;
    a.w_post = w_post;
    a.gate = gate;
    a.w_pre = p->w_pre;
    a.b_stride = b_stride;
    a.r_stride = r_stride;
    a.ro_stride = r_out_stride;
    a.xn_stride = xn_stride;
    a.gate_stride = p->gate_stride;
    a.m = m;
    a.d = (uint32_t)p->d;
    a.eps = p->eps;
    a.scale = p->scale;
    a.inv_d = 1.f / (float)p->d;
    const NormShape s = norm_shape(p->d);
    return launch_norm<false>(a, s, norm_blocks(s, m, kForwardBlocks), vec, rb == 4, static_cast<hipStream_t>(stream));
}

int afx_block_norm_workspace(const afx_block_norm *p, uint32_t m, size_t *bytes) {
    const int rc = check_norm(p);
    if (rc != AFX_OK) return rc;
    if (!bytes) return AFX_E_INVALID_ARG;
    *bytes = norm_space(p, m);
    return AFX_OK;
}

int afx_block_norm_backward_async(const afx_block_norm *p, uint32_t m, const float *b_dev, uint64_t b_stride,
                                  const void *r_out_dev, uint64_t r_out_stride, const uint16_t *dxn_dev,
                                  uint64_t dxn_stride, const void *dr_out_dev, uint64_t dr_out_stride, void *dr_dev,
                                  uint64_t dr_stride, uint16_t *db_dev, uint64_t db_stride, float *dw_pre_dev,
                                  float *dw_post_dev, float *dgate_dev, void *ws_dev, size_t ws_bytes, void *stream) {
    int rc = check_norm(p);
    if (rc != AFX_OK) return rc;
    const bool per_row = p->gate && p->gate_stride;
    if ((!p->w_pre && (dxn_dev || dw_pre_dev)) || (!p->w_post && dw_post_dev) || (!p->gate && dgate_dev) ||
        (!dr_dev && !db_dev && !dw_pre_dev && !dw_post_dev && !dgate_dev))
        return AFX_E_INVALID_ARG;
    if (m && !b_dev && (db_dev || dw_post_dev || dgate_dev)) return AFX_E_INVALID_ARG;
    float *dgate_sum = per_row ? nullptr : dgate_dev;
    const bool sums = dw_pre_dev || dw_post_dev || dgate_sum;
    const uint64_t rb = p->r_type == AFX_TYPE_FP32 ? 4 : 2;
    const uint64_t need = sums ? norm_space(p, m) : 0;
    if (m) {
        if (!r_out_dev || (need && !ws_dev)) return AFX_E_INVALID_ARG;
        if ((b_dev && b_stride < p->d) || r_out_stride < p->d || (dxn_dev && dxn_stride < p->d) ||
            (dr_out_dev && dr_out_stride < p->d) || (dr_dev && dr_stride < p->d) || (db_dev && db_stride < p->d))
            return AFX_E_INVALID_ARG;
    }
    const uint16_t *w_post = b_dev ? p->w_post : nullptr, *gate = b_dev ? p->gate : nullptr;
    const Rows rows[] = {{b_dev, b_stride, 4, false},
                         {r_out_dev, r_out_stride, rb, false},
                         {dxn_dev, dxn_stride, 2, false},
                         {dr_out_dev, dr_out_stride, rb, false},
                         {dr_dev, dr_stride, rb, true},
                         {db_dev, db_stride, 2, true},
                         {w_post, 0, 2, false},
                         {gate, p->gate_stride, 2, false},
                         {dxn_dev ? p->w_pre : nullptr, 0, 2, false},
                         {per_row ? dgate_dev : nullptr, p->d, 4, true}};
    bool vec = false;
    rc = check_rows(rows, 10, m, p->d, 3, 4, &vec);
    if (rc != AFX_OK) return rc;
    // the sums over rows (one row each) and the workspace
    const Rows one[] = {{dw_pre_dev, p->d, 4, true},
                        {dw_post_dev, p->d, 4, true},
                        {dgate_sum, p->d, 4, true},
                        {need ? ws_dev : nullptr, 0, 1, true}};
    for (int i = 0; i < 4; ++i) {
        if (reinterpret_cast<uintptr_t>(one[i].p) & (i < 3 ? 3 : 15)) return AFX_E_MISALIGNED;
        const RowSpan mine{one[i].p, 1, i < 3 ? p->d * 4 : need, 0};
        for (const Rows &r : rows)
            if (rows_overlap(mine, span(r, m, p->d))) return AFX_E_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (rows_overlap(mine, RowSpan{one[k].p, 1, p->d * 4, 0})) return AFX_E_INVALID_ARG;
    }
    if (ws_bytes < need) return AFX_E_BUFFER_TOO_SMALL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    NormArgs a{};
    a.b = b_dev;
    a.r = r_out_dev;
    a.dxn = dxn_dev;
    a.dr_out = dr_out_dev;
    a.dr = dr_dev;
    a.db = db_dev;
    a.part = need ? static_cast<float *>(ws_dev) : nullptr;
    a.dgate_rows = per_row ? dgate_dev : nullptr;
    a.w_post = w_post;
    a.gate = gate;
    a.w_pre = p->w_pre;
    a.b_stride = b_stride;
    a.r_stride = r_out_stride;
    a.dxn_stride = dxn_stride;
    a.dro_stride = dr_out_stride;
    a.dr_stride = dr_stride;
    a.db_stride = db_stride;
    a.gate_stride = p->gate_stride;
    a.m = m;
    a.d = (uint32_t)p->d;
    a.eps = p->eps;
    a.scale = p->scale;
    a.inv_d = 1.f / (float)p->d;
    const NormShape shape = norm_shape(p->d);
    uint32_t blocks = grad_blocks(shape, m);
    if (m) {
        rc = launch_norm<true>(a, shape, blocks, vec, rb == 4, s);
        if (rc != AFX_OK) return rc;
    }
    if (!sums) return AFX_OK;
    uint32_t d = a.d;
    void *args[] = {&a.part, &blocks, &d, &dw_pre_dev, &dw_post_dev, &dgate_sum};
    return hipLaunchKernel(reinterpret_cast<const void *>(&afx_norm_sum_kernel),
                           dim3((d + kSumCols - 1) / kSumCols, 3), dim3(kSumSlices * kSumCols), args, 0,
                           s) == hipSuccess
               ? AFX_OK
               : AFX_E_HIP;
}

}  // extern "C"
