// The gate's activations and their derivatives, in float32.  The exponential and the reciprocal are the
// hardware's (2^x and 1 / x to about one unit in the last place; the exponent's product with log2 e adds
// |a| 2^-24): 2^-20 of the value at |a| = 16, where the results round to bfloat16 at 2^-8 or are
// given in float32.  gelu's distribution function is erfc(-a / sqrt 2) / 2, not (1 + erf) / 2, which cancels for
// negative gates (nothing left at -6): off by less than (a^2 + 20) 2^-23 of the value, of which (a^2 + 1) 1.5 2^-24 is the
// argument's rounding (999 slots of 37 leaves, 100 -> 2 x 385, on the GPU: 12.1 us, with erf 11.5).
// Rounding a itself to float32 moves silu by |a| 2^-24 and gelu by a^2 2^-24 of their values, so neither is off by
// much more than its argument.  A NaN stays NaN.
#pragma once
#include "ah_random.hpp"
#include "../../include/ah.h"

namespace ah {

__device__ __forceinline__ float logistic(float a) {  // 1 / (1 + e^-a); 0 where e^-a overflows
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * a));
}
__device__ __forceinline__ float normal_cdf(float a) { return 0.5f * erfcf(-0.70710678118654752f * a); }

__device__ __forceinline__ float activate(int act, float a) {
    if (act == AH_SILU) return a * logistic(a);
    if (act == AH_GELU) return a * normal_cdf(a);
    return a < 0.0f ? 0.0f : a;
}
__device__ __forceinline__ void activate_grad(int act, float a, float* f, float* df) {
    if (act == AH_SILU) {
        const float s = logistic(a);
        *f = a * s;
        *df = s + *f * (1.0f - s);
    } else if (act == AH_GELU) {
        const float c = normal_cdf(a);
        *f = a * c;
        *df = c + 0.39894228040143268f * a * __builtin_amdgcn_exp2f(-0.72134752044448170f * a * a);
    } else {
        *f = a < 0.0f ? 0.0f : a;
        *df = a > 0.0f ? 1.0f : a <= 0.0f ? 0.0f : a;
    }
}

}  // namespace ah
