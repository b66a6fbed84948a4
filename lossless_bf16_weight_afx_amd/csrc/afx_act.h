// afx_act.h -- the activations of the gated feed-forward block, in FP32.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/afx.h"

namespace afx {
namespace {

// act(g). SiLU: g / (1 + e^-g), whose limits for large |g| come out right
// without a case (e^-g overflows to infinity: g / inf = -0). GELU with tanh:
// 0.5 g (1 + tanh z) = g / (1 + e^-2z), z = sqrt(2/pi) (g + 0.044715 g^3),
// the same form as SiLU. GELU: 0.5 g (1 + erf(g / sqrt 2)).
constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;  // sqrt(2/pi)
__device__ inline float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }

template <uint32_t kAct>
__device__ inline float act(float g) {
    if constexpr (kAct == AFX_ACT_SILU) return g / (1.f + __expf(-g));
    if constexpr (kAct == AFX_ACT_GELU_TANH) return g / (1.f + __expf(-2.f * kGeluC * (g + kGeluA * g * g * g)));
    return 0.5f * g * erfcf(-0.7071067811865476f * g);  // 1 + erf(z) = erfc(-z), without its cancellation
}

// act(g) and act'(g). SiLU: s (1 + g (1 - s)); tanh form: with s =
// sigmoid(2z), s + g s (1 - s) 2 z'; GELU: cdf + g pdf. In the tanh form z'
// is taken at |g| <= 16, where 1 - s or s is 0 already (2z = 318): its square
// would overflow from |g| = 1.8e19 on, and infinity times 0 is NaN.
template <uint32_t kAct>
__device__ inline void act_grad(float g, float &a, float &da) {
    if constexpr (kAct == AFX_ACT_SILU) {
        const float s = sigmoid(g);
        a = act<kAct>(g);
        da = s * (1.f + g * (1.f - s));
    } else if constexpr (kAct == AFX_ACT_GELU_TANH) {
        const float s = sigmoid(2.f * kGeluC * (g + kGeluA * g * g * g));
        a = act<kAct>(g);
        const float t = fminf(fmaxf(g, -16.f), 16.f);
        da = s + t * s * (1.f - s) * (2.f * kGeluC) * (1.f + 3.f * kGeluA * t * t);
    } else {
        const float cdf = 0.5f * erfcf(-0.7071067811865476f * g);
        a = g * cdf;
        da = cdf + g * __expf(-0.5f * g * g) * 0.3989422804014327f;
    }
}

}  // namespace
}  // namespace afx
