// linear_out.cuh -- the end of a dense product: from the sums of four neighbouring
// values of a row to what is stored of them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "combine_math.cuh"
#include "kernels.cuh"
#include "linear_math.cuh"

namespace ep {

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Four neighbouring values of a row. In memory `left` of them (at most four) are
// there; rows of a multiple of four values hold them all, 16-byte (in bf16 8-byte)
// aligned (`vec`).
struct Four {
    float v[4];
};
__device__ __forceinline__ Four operator+(const Four& x, const Four& y) {
    return {{x.v[0] + y.v[0], x.v[1] + y.v[1], x.v[2] + y.v[2], x.v[3] + y.v[3]}};
}
__device__ __forceinline__ Four four(float4 f) { return {{f.x, f.y, f.z, f.w}}; }

__device__ __forceinline__ Four load_bias(const float* bias, int64_t col, int64_t left) {
    Four r = {};
    if (bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) r.v[i] = __ldg(bias + col + i);
    }
    return r;
}

// What is added to four values, as it lies in memory until it is added.
struct Residual {
    uint32_t bits[4];
};
__device__ __forceinline__ Residual load_residual(const LinearArgs& a, int64_t at, int64_t left,
                                                  bool vec) {
    Residual r = {};
    if (a.out_f32) {
        const uint32_t* p = static_cast<const uint32_t*>(a.residual) + at;
        if (vec) {
            const uint4 f = *reinterpret_cast<const uint4*>(p);
            r.bits[0] = f.x, r.bits[1] = f.y, r.bits[2] = f.z, r.bits[3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) r.bits[i] = p[i];
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.residual) + at;
        if (vec) {
            const uint2 f = *reinterpret_cast<const uint2*>(p);
            r.bits[0] = f.x, r.bits[1] = f.y;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) r.bits[i] = p[i];
        }
    }
    return r;
}
__device__ __forceinline__ Four residual_values(const LinearArgs& a, const Residual& r, bool vec) {
    const uint32_t* b = r.bits;
    if (a.out_f32)
        return {{__uint_as_float(b[0]), __uint_as_float(b[1]), __uint_as_float(b[2]), __uint_as_float(b[3])}};
    if (vec) return {{bf16_low(b[0]), bf16_high(b[0]), bf16_low(b[1]), bf16_high(b[1])}};
    return {{bf16_low(b[0]), bf16_low(b[1]), bf16_low(b[2]), bf16_low(b[3])}};
}

__device__ __forceinline__ void store_bf16(uint16_t* p, const Four& r, int64_t left, bool vec) {
    const uint32_t lo = pack_bf16x2(r.v[0], r.v[1]), hi = pack_bf16x2(r.v[2], r.v[3]);
    if (vec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
        return;
    }
    if (0 < left) p[0] = static_cast<uint16_t>(lo);
    if (1 < left) p[1] = static_cast<uint16_t>(lo >> 16);
    if (2 < left) p[2] = static_cast<uint16_t>(hi);
    if (3 < left) p[3] = static_cast<uint16_t>(hi >> 16);
}
__device__ __forceinline__ void store_out(const LinearArgs& a, int64_t at, const Four& r, int64_t left,
                                          bool vec) {
    if (!a.out_f32) {
        store_bf16(static_cast<uint16_t*>(a.out) + at, r, left, vec);
        return;
    }
    float* p = static_cast<float*>(a.out) + at;
    if (vec) {
        *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = r.v[i];
}

// act(v), gated silu(v) * up, of all at once, so that what it is is asked once.
template <bool kGated, int kCount>
__device__ __forceinline__ void activate(const LinearArgs& a, Four (&v)[kCount],
                                         const Four (&up)[kCount]) {
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kCount; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j].v[i] = f(v[j].v[i], up[j].v[i]);
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

// z, where it is kept: row `row`'s values from column `col` on, sums with their
// bias in `v` (gated: the up half's in `up`).
template <bool kGated>
__device__ __forceinline__ void keep_z(const LinearArgs& a, int64_t row, int64_t col, const Four& v,
                                       const Four& up, int64_t left, bool vec) {
    if (a.z == nullptr) return;
    uint16_t* z = a.z + row * (kGated ? 2 * a.n : a.n) + col;
    store_bf16(z, v, left, vec);
    if (kGated) store_bf16(z + a.n, up, left, vec);
}

// All of it, for sums without their bias.
template <bool kGated>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t row, int64_t col, const Four& sums,
                                       const Four& up_sums, const Residual& residual, int64_t left,
                                       bool vec) {
    Four v[1] = {sums + load_bias(a.bias, col, left)}, up[1] = {up_sums};
    if (kGated) up[0] = up[0] + load_bias(a.bias, a.n + col, left);
    keep_z<kGated>(a, row, col, v[0], up[0], left, vec);
    activate<kGated>(a, v, up);
    if (a.residual != nullptr) v[0] = v[0] + residual_values(a, residual, vec);
    store_out(a, row * a.n + col, v[0], left, vec);
}

}  // namespace ep
