// The per-token arithmetic of the gated linear recurrence, shared by its
// forward, decode and backward kernels so that they agree bit for bit.
#pragma once

#include "device_math.h"

namespace ssm {

// 1 - e^{2 la} for la <= 0, to about an ulp of itself: the recurrence weighs
// its input with the square root of this, and a slow channel's la is so small
// that 1 - a*a would keep few bits.  For 2 la > -1/2 the series of
// -expm1(2 la), whose first term left out is below 2^-26 of the sum; else
// 1 - a*a, where the subtraction costs at most two bits of a half.
__device__ __forceinline__ float one_minus_sq(float la, float a) {
    const float z = 2.0f * la;
    float s = fmaf(z, 1.0f / 40320.0f, 1.0f / 5040.0f);
    s = fmaf(z, s, 1.0f / 720.0f);
    s = fmaf(z, s, 1.0f / 120.0f);
    s = fmaf(z, s, 1.0f / 24.0f);
    s = fmaf(z, s, 1.0f / 6.0f);
    s = fmaf(z, s, 0.5f);
    s = fmaf(z, s, 1.0f);
    return z > -0.5f ? -z * s : fmaf(-a, a, 1.0f);
}

// e^-x, held below 2^126 so that 1 / (1 + e) and e / (1 + e) stay finite;
// sigma(x) = 1 / (1 + e^-x).
__device__ __forceinline__ float exp_neg(float x) {
    return fast_exp2(fminf(-x * kLog2e, 126.0f));
}
__device__ __forceinline__ float sigma_of(float e) { return fast_rcp(1.0f + e); }

// One token of one channel: the decay a and the weighted input b of
//   h <- a h + b,  a = exp(A r),  b = sqrt(1 - a^2) i x,
//   r = sigma(gate_a + bias_a),  i = sigma(gate_x + bias_x)
__device__ __forceinline__ void gated_token(float x, float ga, float gx, float A, float bias_a,
                                            float bias_x, float& a, float& b) {
    const float r = sigma_of(exp_neg(ga + bias_a));
    const float i = sigma_of(exp_neg(gx + bias_x));
    const float la = A * r;
    a = fast_exp2(la * kLog2e);
    b = __builtin_amdgcn_sqrtf(one_minus_sq(la, a)) * (i * x);
}

}  // namespace ssm
