// afx_slab.h -- device pieces of the products that restore slabs of a coded
// matrix into LDS for the matrix cores (afx_gemm.hip, afx_gated_gemm.hip).
// Not installed.
#pragma once

#include <hip/hip_runtime.h>

#include "afx_device.h"

namespace afx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of x as the A operand (zeros for a token beyond m).
__device__ inline bf16x8 load_a(const uint16_t *p, bool ok) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) v = *reinterpret_cast<const uint4 *>(p);
    return __builtin_bit_cast(bf16x8, v);
}

// Stage four stream words (those at wa + i .. wa + i + 3) of a row segment,
// reversed: stream word wa + j goes to index kSegRev - j.
__device__ inline void put_seg4(uint32_t *seg, uint32_t i, uint4 v) {
    *reinterpret_cast<uint4 *>(seg + seg_put_index(i)) = make_uint4(v.w, v.z, v.y, v.x);
}

// Decode the 32 exponent codes of the lane's two groups, whose chains start
// at counters r1 and r2 of the row's staged segment (two interleaved
// buffered chains); ex1[j], ex2[j] receive the exponent bytes of elements
// 4j..4j+3. The starts come clamped (seg_chain_r0), so that 32 codes of <=
// 12 bits, and the chains' read-ahead, remain inside the slice even on a
// corrupt stream.
__device__ inline void decode_groups(const uint32_t *seg, uint32_t r1, uint32_t r2, const uint16_t *lut,
                                     uint32_t (&ex1)[8], uint32_t (&ex2)[8]) {
    BufChain A = buf_chain(seg, r1);
    BufChain B = buf_chain(seg, r2);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        uint32_t a01, b01, a23, b23;
        buf_chain_pairs(A, B, seg, lut, a01, b01);
        buf_chain_pairs(A, B, seg, lut, a23, b23);
        ex1[q] = join_halves(a01, a23);
        ex2[q] = join_halves(b01, b23);
    }
}

__device__ inline uint64_t quad_first(uint64_t v) {  // every lane gets lane 4 (l / 4)'s value
    const int lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)v, 0x00, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(v >> 32), 0x00, 0xF, 0xF, false);
    return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}

}  // namespace
}  // namespace afx
