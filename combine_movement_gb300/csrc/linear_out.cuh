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

template <int N>
__device__ __forceinline__ Values<N> sum(const Values<N>& x, const Values<N>& y) {
    Values<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = x.v[i] + y.v[i];
    return r;
}

// The activation of `v` (gated: with `up`), for the whole array at once, so that
// what it is is asked once.
template <int kCount, int N, bool kGated>
__device__ __forceinline__ void activate_all(Values<N> (&v)[kCount], const Values<N> (&up)[kCount],
                                             int act) {
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kCount; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) v[i].v[j] = f(v[i].v[j], up[i].v[j]);
    };
    if (kGated)
        each([](float g, float u) { return silu(g) * u; });
    else if (act == EP_ACT_RELU)
        each([](float z, float) { return activate(z, EP_ACT_RELU); });
    else if (act == EP_ACT_GELU)
        each([](float z, float) { return activate(z, EP_ACT_GELU); });
    else if (act == EP_ACT_SILU)
        each([](float z, float) { return activate(z, EP_ACT_SILU); });
}

// The end of kCount times N values of out, `apart` rows apart from row `row` on,
// of which `rows` (as many as are there) are stored: sums with their bias in `v`
// (gated: the up half's in `up`), `residual` what is added.
template <int kCount, int N, bool kGated>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t row, int64_t col, int apart,
                                       int rows, Values<N> (&v)[kCount], const Values<N> (&up)[kCount],
                                       const Residual<N> (&residual)[kCount]) {
    if (a.z != nullptr) {
        const int64_t pitch = kGated ? 2 * a.n : a.n;
        uint16_t* z = a.z + row * pitch + col;
#pragma unroll
        for (int i = 0; i < kCount; ++i, z += apart * pitch) {
            if (i >= rows) continue;
            store_bf16<N>(z, v[i]);
            if (kGated) store_bf16<N>(z + a.n, up[i]);
        }
    }
    activate_all<kCount, N, kGated>(v, up, a.act);
    if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = sum<N>(v[i], residual_values<N>(a, residual[i]));
    }
    const int64_t at = row * a.n + col, step = apart * a.n;
    if (a.out_f32) {
        float* p = static_cast<float*>(a.out) + at;
#pragma unroll
        for (int i = 0; i < kCount; ++i, p += step)
            if (i < rows) store_f32<N>(p, v[i]);
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
        for (int i = 0; i < kCount; ++i, p += step)
            if (i < rows) store_bf16<N>(p, v[i]);
    }
}

}  // namespace ep
