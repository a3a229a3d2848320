// fp8_math.cuh -- the block quantiser's arithmetic, shared by the dispatch
// that quantises rows and the expert product that quantises its activation,
// so both round alike.
//
// A block of up to 128 values v: m = max(max|v|, 1e-30), scale = m / 448,
// q = e4m3_rne(v * (448 / m)), each step one correctly rounded fp32 operation.
// 448 is e4m3's largest value, so q uses the whole range; the floor keeps
// 448 / m finite, and a block of zeros gets zeros. The maximum is taken over
// the values' bit patterns, where infinities and NaN are the largest: a
// block that holds one gets a scale that is not finite, so that it shows
// (values times scale are then not finite either).
#pragma once

#include <cstdint>

namespace ep {

constexpr int kFp8Block = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;

// Bits of |v|: ordered like |v|, NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct BlockScale {
    float scale;    // what q is multiplied with to get the value back
    float inverse;  // what the value is multiplied with before rounding
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
    const uint32_t floor_bits = __float_as_uint(kAmaxFloor);
    const float m = __uint_as_float(amax_bits > floor_bits ? amax_bits : floor_bits);
    return {__fdiv_rn(m, kE4m3Max), __fdiv_rn(kE4m3Max, m)};
}

// Four fp32 values -> four e4m3 (round to nearest even), v0 in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float v0, float v1, float v2, float v3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v1), "f"(v0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v3), "f"(v2));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace ep
