// linear_out.cuh -- the end of a dense product: from the sums of a few
// neighbouring values of a row to what is stored of them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "combine_math.cuh"
#include "kernels.cuh"
#include "linear_math.cuh"

namespace ep {

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// N (4 or 1) neighbouring values of a row.
template <int N>
struct Values {
    float v[N];
};
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]));
    else
        *p = __bfloat16_as_ushort(__float2bfloat16_rn(r.v[0]));
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    else
        *p = r.v[0];
}

// What is added to N values of out, as it lies in memory until it is added.
template <int N>
struct Residual {
    uint32_t bits[N];
};
template <int N>
__device__ __forceinline__ Residual<N> load_residual(const LinearArgs& a, int64_t at) {
    Residual<N> r = {};
    if constexpr (N == 4) {
        if (a.out_f32) {
            const uint4 f = *reinterpret_cast<const uint4*>(static_cast<const float*>(a.residual) + at);
            r.bits[0] = f.x, r.bits[1] = f.y, r.bits[2] = f.z, r.bits[3] = f.w;
        } else {
            const uint2 f = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.residual) + at);
            r.bits[0] = f.x, r.bits[1] = f.y;
        }
    } else {
        if (a.out_f32)
            r.bits[0] = static_cast<const uint32_t*>(a.residual)[at];
        else
            r.bits[0] = static_cast<uint32_t>(static_cast<const uint16_t*>(a.residual)[at]) << 16;
    }
    return r;
}
template <int N>
__device__ __forceinline__ Values<N> residual_values(const LinearArgs& a, const Residual<N>& r) {
    if constexpr (N == 4) {
        if (!a.out_f32)
            return {{bf16_low(r.bits[0]), bf16_high(r.bits[0]), bf16_low(r.bits[1]), bf16_high(r.bits[1])}};
        return {{__uint_as_float(r.bits[0]), __uint_as_float(r.bits[1]), __uint_as_float(r.bits[2]),
                 __uint_as_float(r.bits[3])}};
    } else {
        return {{__uint_as_float(r.bits[0])}};
    }
}

// What is added to N columns from `col` on of b's sums.
template <int N>
__device__ __forceinline__ Values<N> load_bias(const LinearArgs& a, int64_t col) {
    Values<N> r = {};
    if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = __ldg(a.bias + col + i);
    }
    return r;
}

// The end of N values of out's row `row` from column `col` on: sums with their
// bias in `v` (gated: the up half's in `up`), `residual` what is added.
template <int N, bool kGated>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t row, int64_t col, Values<N> v,
                                       const Values<N>& up, const Residual<N>& residual) {
    if (a.z != nullptr) {
        uint16_t* z = a.z + row * (kGated ? 2 * a.n : a.n) + col;
        store_bf16<N>(z, v);
        if (kGated) store_bf16<N>(z + a.n, up);
    }
    const Values<N> res = residual_values<N>(a, residual);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v.v[i] = kGated ? silu(v.v[i]) * up.v[i] : activate(v.v[i], a.act);
        v.v[i] += res.v[i];
    }
    const int64_t at = row * a.n + col;
    if (a.out_f32)
        store_f32<N>(static_cast<float*>(a.out) + at, v);
    else
        store_bf16<N>(static_cast<uint16_t*>(a.out) + at, v);
}
template <int N>
__device__ __forceinline__ Values<N> sum(const Values<N>& x, const Values<N>& y) {
    Values<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = x.v[i] + y.v[i];
    return r;
}

}  // namespace ep
