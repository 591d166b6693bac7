// The per-token arithmetic of the gated linear recurrence, shared by its
// forward, decode and backward kernels.
#pragma once

#include "device_math.h"

namespace ssm {

// One channel's parameters, scaled for exp2: A log2 e, and the biases times
// -log2 e, so that e^-(gate + bias) and e^(A r) are one multiply(-add) and one
// v_exp_f32 each.
struct GatedChannel {
    float A2, ba, bx;
};
__device__ __forceinline__ GatedChannel gated_channel(float A, float bias_a, float bias_x) {
    return {A * kLog2e, bias_a * -kLog2e, bias_x * -kLog2e};
}

// e^-(gate + bias); sigma(x) = 1 / (1 + e^-x).  Beyond what fp32 holds e is
// inf and sigma zero.
__device__ __forceinline__ float exp_neg(float gate, float bias) {
    return fast_exp2(fmaf(gate, -kLog2e, bias));
}
// the same held below 2^126, for 1 - sigma = e sigma; the minimum that keeps a
// NaN (one instruction; fminf would shut the gate)
__device__ __forceinline__ float exp_neg_finite(float gate, float bias) {
    return fast_exp2(__builtin_elementwise_minimum(fmaf(gate, -kLog2e, bias), 126.0f));
}
__device__ __forceinline__ float sigma_of(float e) { return fast_rcp(1.0f + e); }

// 1 - a^2 for a = 2^y, y <= 0: the recurrence weighs its input with the square
// root of this, and a slow channel's y is so small that 1 - a*a would keep few
// bits.  With l = y ln 2,
//   1 - e^{2l} = -2 e^l sinh(l) = -2 l a (1 + l^2/6 + l^4/120 + l^6/5040 + ...):
// for l > -1/2 the first term left out is below 2^-26 of the sum, and nothing
// cancels.  Below, 1 - a*a is above 0.63.
__device__ __forceinline__ float one_minus_sq(float y, float a) {
    constexpr float k0 = -2.0f * kLn2, k1 = k0 * kLn2 * kLn2 / 6.0f;
    constexpr float k2 = k1 * kLn2 * kLn2 / 20.0f, k3 = k2 * kLn2 * kLn2 / 42.0f;
    const float t = y * y;
    float s = fmaf(t, k3, k2);
    s = fmaf(t, s, k1);
    s = fmaf(t, s, k0);
    return y > -0.72f ? y * a * s : fmaf(-a, a, 1.0f);
}

// One token of one channel: the decay a and the weighted input b of
//   h <- a h + b,  a = exp(A r),  b = sqrt(1 - a^2) i x,
//   r = sigma(gate_a + bias_a),  i = sigma(gate_x + bias_x)
__device__ __forceinline__ void gated_token(float x, float ga, float gx, const GatedChannel& p,
                                            float& a, float& b) {
    const float y = p.A2 * sigma_of(exp_neg(ga, p.ba));
    a = fast_exp2(y);
    b = __builtin_amdgcn_sqrtf(one_minus_sq(y, a)) * (sigma_of(exp_neg(gx, p.bx)) * x);
}

}  // namespace ssm
