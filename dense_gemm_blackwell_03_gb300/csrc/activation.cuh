// activation.cuh -- the gated layer's activations and their slopes, in fp32.
//
// silu(g) = g s(g) and gelu_tanh(g) = g (1 + tanh z) / 2 = g s(2 z) with the logistic
// function s(t) = 1 / (1 + exp(-t)) and z = sqrt(2 / pi) (g + 0.044715 g^3); gelu(g) = g Phi(g).
// The quotient is CUDA's fast one, good to 2 ulp, and so is exp, whose error grows with its argument:
// 2 + 1.2 |t| ulp, 2^-16 at the ends of its range -- results are rounded to 2^-9 or 2^-12 after them.
#pragma once

#include <cstdint>

#include "../../include/bwgemm.h"

namespace bwgemm {

// s(t), as exp(t) / (1 + exp(t)) for t < 0: nothing overflows, and what is below fp32's normal
// numbers (t < -87.3) is as coarse as they are; 0 from t = -104 on.
__device__ __forceinline__ float logistic(float t)
{
    const float e = __expf(-fabsf(t));
    return __fdividef(t < 0.f ? e : 1.f, 1.f + e);
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC3 = 0.044715f;

__device__ __forceinline__ float activate(float g, int activation)
{
    if (activation == BWGEMM_SILU)
        return g * logistic(g);
    if (activation == BWGEMM_GELU)
        return g * normcdff(g);
    return g * logistic(kGeluC * fmaf(kGeluC3 * g * g, g, g));
}

// The activation and its derivative.
__device__ __forceinline__ void activate_slope(float g, int activation, float& value, float& slope)
{
    if (activation == BWGEMM_GELU) {
        const float cdf = normcdff(g);
        value = g * cdf;
        slope = fmaf(g, 0.3989422804014327f * __expf(-0.5f * g * g), cdf);
        return;
    }
    // g s(t): slope s + g s (1 - s) t', with t' = 1 or the cubic's; 1 - s(t) = s(-t) without
    // cancellation
    float t = g, gdt = g;
    if (activation == BWGEMM_GELU_TANH) {
        // past 30 the slope is 0 or 1, and the cubic's is kept from infinity times zero
        const float c = g > 30.f ? 30.f : g < -30.f ? -30.f : g;
        t = kGeluC * fmaf(kGeluC3 * c * c, c, c);
        gdt = kGeluC * c * fmaf(3.f * kGeluC3 * c, c, 1.f);
    }
    const float s = logistic(t);
    value = g * s;
    slope = fmaf(gdt * s, logistic(-t), s);
}

}  // namespace bwgemm
