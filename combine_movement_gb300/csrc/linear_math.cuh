// linear_math.cuh -- the activations of the dense products and their
// derivatives, in fp32, shared by the products' epilogue and the gradient.
//
// silu(v) = v s(v), s(v) = 1 / (1 + e^-v), with approximate exponential and
// reciprocal, as the experts' gate: off by (8 + 2 |v|) 2^-23 of its value. Both
// s(v) and s(-v) come from e^-|v|, which does not overflow, over a divisor in
// [1, 2]. gelu(v) = v P(v), P the normal distribution's cumulative function: with
// a = |v| / sqrt 2, P(-|v|) = e^(-a^2) g(a) / 2 where g(a) = e^(a^2) erfc(a) is
// smooth, a polynomial of degree 9 in u = 1 / (1 + 0.3 a) (fitted here for a in [0, 9.6],
// where P passes fp32's smallest: off by 1.6e-8 of itself), so that the tail keeps
// its relative precision: (16 + v^2) 2^-23, of which v^2 is the exponent's rounding.
#pragma once

#include <cuda_runtime.h>

#include "../../include/ep.h"

namespace ep {

__device__ __forceinline__ float approx_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

struct Sigmoid {
    float of;     // s(v)
    float minus;  // s(-v) = 1 - s(v)
};
__device__ __forceinline__ Sigmoid sigmoids(float v) {
    const float t = __expf(-fabsf(v)), r = approx_reciprocal(1.0f + t);
    return v < 0.0f ? Sigmoid{t * r, r} : Sigmoid{r, t * r};
}
__device__ __forceinline__ float silu(float v) {
    const float t = __expf(-fabsf(v));
    return (v < 0.0f ? v * t : v) * approx_reciprocal(1.0f + t);
}
__device__ __forceinline__ float silu_slope(float v) {
    const Sigmoid s = sigmoids(v);
    return fmaf(v * s.of, s.minus, s.of);
}
__device__ __forceinline__ float approx_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
struct Normal {
    float cdf;       // P(v)
    float exponent;  // e^(-v^2 / 2)
};
__device__ __forceinline__ Normal normal(float v) {
    const float u = approx_reciprocal(fmaf(0.3f * 0.70710678118654752f, fabsf(v), 1.0f));
    float g = -0.12543776631355286f;
    g = fmaf(g, u, 0.46274301409721375f);
    g = fmaf(g, u, -0.4568597674369812f);
    g = fmaf(g, u, 0.4710356593132019f);
    g = fmaf(g, u, -0.028110980987548828f);
    g = fmaf(g, u, 0.1774287223815918f);
    g = fmaf(g, u, 0.16204634308815002f);
    g = fmaf(g, u, 0.1675841361284256f);
    g = fmaf(g, u, 0.16959325969219208f);
    g = fmaf(g, u, -2.2634743800153956e-05f);
    const float e = approx_exp2(v * v * -0.72134752044448170f);
    const float t = 0.5f * g * e;
    return {v < 0.0f ? t : 1.0f - t, e};
}

// The activations of one value (swiglu has two).
__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case EP_ACT_GELU: return v * normal(v).cdf;
        case EP_ACT_SILU: return silu(v);
        default: return v;
    }
}
__device__ __forceinline__ float activate_slope(float v, int act) {
    switch (act) {
        case EP_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
        case EP_ACT_GELU: {
            const Normal p = normal(v);
            return fmaf(v * 0.39894228040143268f, p.exponent, p.cdf);
        }
        case EP_ACT_SILU: return silu_slope(v);
        default: return 1.0f;
    }
}

}  // namespace ep
