// linear_math.cuh -- the activations of the dense products and their
// derivatives, in fp32, shared by the products' epilogue and the gradient.
//
// silu(v) = v s(v), s(v) = 1 / (1 + e^-v), with approximate exponential and
// reciprocal, as the experts' gate: off by (8 + 2 |v|) 2^-23 of its value. Both
// s(v) and s(-v) come from e^-|v|, which does not overflow, over a divisor in
// [1, 2]. gelu(v) = v P(v), P the normal distribution's cumulative function,
// as erfc(-v / sqrt 2) / 2: the tail keeps its relative precision.
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
__device__ __forceinline__ float normal_cdf(float v) {
    return 0.5f * erfcf(v * -0.70710678118654752f);
}

// The activations of one value (swiglu has two).
__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case EP_ACT_GELU: return v * normal_cdf(v);
        case EP_ACT_SILU: return silu(v);
        default: return v;
    }
}
__device__ __forceinline__ float activate_slope(float v, int act) {
    switch (act) {
        case EP_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
        case EP_ACT_GELU:
            // (at infinity the density is 0: no 0 * inf)
            return normal_cdf(v) + v * (0.39894228040143268f * expf(-0.5f * fminf(v * v, 256.0f)));
        case EP_ACT_SILU: return silu_slope(v);
        default: return 1.0f;
    }
}

}  // namespace ep
