// linear_out.cuh -- the end of a dense product: from the sums of neighbouring values
// of a row to what is stored of them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "combine_math.cuh"
#include "kernels.cuh"
#include "linear_math.cuh"

namespace ep {

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// N (4, 2 or 1) neighbouring values of a row whose length N divides: in memory they
// are aligned as one.
template <int N>
struct Values {
    float v[N];
};
template <int N>
__device__ __forceinline__ Values<N> operator+(const Values<N>& x, const Values<N>& y) {
    Values<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = x.v[i] + y.v[i];
    return r;
}

template <int N>
__device__ __forceinline__ Values<N> load_bias(const float* bias, int64_t col) {
    Values<N> r = {};
    if (bias != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = __ldg(bias + col + i);
    }
    return r;
}

// What is added to N values, as it lies in memory until it is added.
template <int N>
struct Residual {
    uint32_t bits[N];
};
template <int N>
__device__ __forceinline__ Residual<N> load_residual(const LinearArgs& a, int64_t at) {
    Residual<N> r = {};
    if (a.out_f32) {
        const uint32_t* p = static_cast<const uint32_t*>(a.residual) + at;
        if constexpr (N == 4) {
            const uint4 f = *reinterpret_cast<const uint4*>(p);
            r.bits[0] = f.x, r.bits[1] = f.y, r.bits[2] = f.z, r.bits[3] = f.w;
        } else if constexpr (N == 2) {
            const uint2 f = *reinterpret_cast<const uint2*>(p);
            r.bits[0] = f.x, r.bits[1] = f.y;
        } else {
            r.bits[0] = *p;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.residual) + at;
        if constexpr (N == 4) {
            const uint2 f = *reinterpret_cast<const uint2*>(p);
            r.bits[0] = f.x, r.bits[1] = f.y;
        } else if constexpr (N == 2) {
            r.bits[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            r.bits[0] = *p;
        }
    }
    return r;
}
template <int N>
__device__ __forceinline__ Values<N> residual_values(const LinearArgs& a, const Residual<N>& r) {
    Values<N> v;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v.v[i] = a.out_f32 ? __uint_as_float(r.bits[i])
                           : (i % 2 == 0 ? bf16_low(r.bits[i / 2]) : bf16_high(r.bits[i / 2]));
    return v;
}

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]));
    else if constexpr (N == 2)
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(r.v[0], r.v[1]);
    else
        *p = __bfloat16_as_ushort(__float2bfloat16_rn(r.v[0]));
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    else if constexpr (N == 2)
        *reinterpret_cast<float2*>(p) = make_float2(r.v[0], r.v[1]);
    else
        *p = r.v[0];
}

// act(v), gated silu(v) * up, of all at once, so that what it is is asked once.
template <int N, bool kGated, int kCount>
__device__ __forceinline__ void activate(const LinearArgs& a, Values<N> (&v)[kCount],
                                         const Values<N> (&up)[kCount]) {
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kCount; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) v[j].v[i] = f(v[j].v[i], up[j].v[i]);
    };
    if (kGated)
        each([](float g, float u) { return silu(g) * u; });
    else if (a.act == EP_ACT_RELU)
        each([](float z, float) { return activate(z, EP_ACT_RELU); });
    else if (a.act == EP_ACT_GELU)
        each([](float z, float) { return activate(z, EP_ACT_GELU); });
    else if (a.act == EP_ACT_SILU)
        each([](float z, float) { return activate(z, EP_ACT_SILU); });
}

// The end of kCount times N values of out: those of the rows row, row + apart and so on,
// of which `rows` are there, from column `col` on. `v` the sums with their bias (gated:
// the up half's in `up`), `residual` what is added.
template <int N, bool kGated, int kCount>
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
    activate<N, kGated>(a, v, up);
    if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) v[i] = v[i] + residual_values<N>(a, residual[i]);
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

// f with the number of values that rows of length n hold aligned, as a type's `value`.
template <typename F>
__device__ __forceinline__ void by_width(int64_t n, F f) {
    if (n % 4 == 0)
        f(std::integral_constant<int, 4>());
    else if (n % 2 == 0)
        f(std::integral_constant<int, 2>());
    else
        f(std::integral_constant<int, 1>());
}

}  // namespace ep
