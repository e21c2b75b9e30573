// gate.cuh -- silu(gate) * up and its gradient, in fp32 for every finite gate.
//
// With h = exp(-|gate| / 2) and q = h^2 the logistic function is 1 / (1 + q), for a negative
// gate q / (1 + q), so that nothing leaves fp32 (exp(-gate) itself is past it below -88.7, and
// its reciprocal below -87.3).  Of h the approximate exp2 takes 2^-22 and the rounded argument
// |gate| 2^-24, of the result the reciprocal 2^-23: below 2^-15 in all for |gate| <= 120, past
// which the result leaves bf16's range, and 2^-18 for |gate| <= 16; its rounding is 2^-9.
#pragma once

#include "common.cuh"

namespace moe {

struct Logistic {
    float by, inv, q;        // h for a negative gate and 1 for another, 1 / (1 + q), q
};

__device__ __forceinline__ Logistic logistic(float gate)
{
    constexpr float kHalfLog2E = 0.72134752044448f;
    float h, inv;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(-kHalfLog2E * fabsf(gate)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(h, h, 1.f)));
    return {gate < 0.f ? h : 1.f, inv, h * h};
}

// silu(gate) * up.
__device__ __forceinline__ float gated_output(float gate, float up)
{
    const Logistic l = logistic(gate);
    return (gate * l.by) * l.inv * (l.by * up);
}

// Gradient of it in gate and in up, for the gradient d of the output: d up s (1 + gate (1 - s))
// and d gate s, where s = by^2 inv and 1 - s = inv (negative gate) or q inv.
__device__ __forceinline__ void gated_gradient(float gate, float up, float d, float &d_gate, float &d_up)
{
    const Logistic l = logistic(gate);
    const float rest = gate < 0.f ? gate * l.inv : gate * l.q * l.inv;
    d_gate = (d * l.by) * (l.by * up) * (l.inv * (1.f + rest));
    d_up = (gate * l.by) * l.inv * (l.by * d);
}

}  // namespace moe
