// route.cu -- the router: each token's experts and their weights from its
// logits, and the gradient of those weights.
//
// For a token with logits l[e] and, where given, a bias b[e] (for the choice
// alone, to keep the experts' load even):
//
//   s_e = 1 / (1 + e^-l_e)   or   e^(l_e - m) / sum_j e^(l_j - m),  m = max l
//   c_e = l_e without a bias (scores ascend with logits), else s_e + b_e
//   groups: of E / G consecutive experts each, worth its largest c or the sum of
//           its two largest (of scores, where there is no bias); the best
//           topk_groups stay
//   the K largest c of what stays, equal ones by the lower index; weights
//   w_k = scale * s_k, or scale * s_k / sum of the chosen s
//
// An expert whose logit or bias is -inf is out; entries that no expert is left
// for are -1 with weight 0. NaN counts as larger than any number, so that it
// shows.
//
// Which of two experts is larger is decided as in 64 bits, so that a choice has one
// right answer: c is computed in 32 with a bound on its error, and where the bound
// leaves an order open it is settled with the values as they are, then in 64 bits,
// among the experts concerned (a few tokens of a thousand get as far).
//
// Mapping: a warp to a token; lane i holds the V = ceil(E / 32) experts (rounded up
// to a power of two) from i * V on, as integers of their values' order, and sorts
// its own. A round of the choice is one warp-wide integer maximum of the lanes'
// first ones and one ballot, and ties fall to the lower index by themselves.
//
// Bound by instructions, half of them on the integer pipe, which takes two a cycle:
// 16384 tokens, 256 experts, bias, 8 groups, top-8 take 20-27 us (950 instructions a
// token; without groups 19, without a bias 15; the bytes would be 2.7). One token: 3.2 us,
// the chain of its rounds. Measured on the way: arguments passed by address to a function
// that is not inlined make a copy of them in local memory, unless they are constant
// (__grid_constant__); groups' worths from integers with lost bits alone sent a token of
// a thousand into 64 bits, 14 us until the last was done; a persistent grid with the next
// token on its way was 20 % slower (registers); 2, 4 and 8 warps to a CTA are alike. The
// gradient of 16383 tokens, 128 experts, dense: 8.0-8.8 us (440 instructions a token).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace ep {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr float kInf = __builtin_huge_valf();
constexpr int kWarps = 4;

// Integers ordered like the values: 0 for "out" (no value has it), NaN the
// largest, both zeros alike.
__device__ __forceinline__ uint32_t key_of(float v) {
    // -0 + 0 = +0, and a sum's NaN is 0x7FFFFFFF
    const int32_t b = __float_as_int(__fadd_rn(v, 0.0f));
    return static_cast<uint32_t>(b ^ (b >> 31 | static_cast<int32_t>(0x80000000u)));
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (v != v) return ~0ull;
    const long long b = __double_as_longlong(v + 0.0);
    return b < 0 ? ~static_cast<unsigned long long>(b)
                 : static_cast<unsigned long long>(b) | 0x8000000000000000ull;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ double value_of(unsigned long long key) {
    const unsigned long long b = (key >> 63) ? key & 0x7FFFFFFFFFFFFFFFull : ~key;
    return __longlong_as_double(static_cast<long long>(b));
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
    if (a.bf16_logits) {
        const uint16_t v = __ldg(static_cast<const uint16_t*>(a.logits) + at);
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
    return __ldg(static_cast<const float*>(a.logits) + at);
}

// V values from lane * V on of a row that starts at `at`; what lies past its E
// values is `past`. kFull: there is none, and the rows are 16-byte aligned.
template <int V, bool kFull>
__device__ __forceinline__ void load_part(const void* p, bool bf16, int64_t at, int E, float past,
                                          float (&v)[V]) {
    const int e0 = (threadIdx.x & 31) * V;
    if constexpr (kFull && V >= 2) {
        constexpr int kAtOnce = V < 8 ? V : 8;  // 16 bytes of bf16
#pragma unroll
        for (int i = 0; i < V; i += kAtOnce) {
            uint32_t w[kAtOnce];
            if (bf16) {
                const uint16_t* q = static_cast<const uint16_t*>(p) + at + e0 + i;
                if constexpr (kAtOnce == 8) {
                    const uint4 f = __ldg(reinterpret_cast<const uint4*>(q));
                    w[0] = f.x, w[1] = f.y, w[2] = f.z, w[3] = f.w;
                } else if constexpr (kAtOnce == 4) {
                    const uint2 f = __ldg(reinterpret_cast<const uint2*>(q));
                    w[0] = f.x, w[1] = f.y;
                } else {
                    w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    v[i + j] = __uint_as_float(j % 2 == 0 ? w[j / 2] << 16 : w[j / 2] & 0xFFFF0000u);
            } else {
                const float* q = static_cast<const float*>(p) + at + e0 + i;
                if constexpr (kAtOnce == 2) {
                    const float2 f = __ldg(reinterpret_cast<const float2*>(q));
                    v[i] = f.x, v[i + 1] = f.y;
                } else {
#pragma unroll
                    for (int j = 0; j < kAtOnce; j += 4) {
                        const float4 f = __ldg(reinterpret_cast<const float4*>(q + j));
                        v[i + j] = f.x, v[i + j + 1] = f.y, v[i + j + 2] = f.z, v[i + j + 3] = f.w;
                    }
                }
            }
        }
    } else {
        // all loads, then what is made of them: a branch or a shift between them would
        // wait for each (the last expert again in the place of those past it)
        uint32_t w[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t e = at + min(e0 + j, E - 1);
            w[j] = bf16 ? __ldg(static_cast<const uint16_t*>(p) + e)
                        : __ldg(static_cast<const uint32_t*>(p) + e);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = e0 + j >= E ? past : __uint_as_float(bf16 ? w[j] << 16 : w[j]);
    }
}

template <int V, bool kFull>
__device__ __forceinline__ void store_part(void* p, bool bf16, int64_t at, int E, const float (&v)[V]) {
    const int e0 = (threadIdx.x & 31) * V;
    if constexpr (kFull && V >= 4) {
        if (bf16) {
            uint16_t* q = static_cast<uint16_t*>(p) + at + e0;
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<uint2*>(q + i) =
                    make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
        } else {
            float* q = static_cast<float*>(p) + at + e0;
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4*>(q + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (e0 + j >= E) continue;
            if (bf16)
                static_cast<__nv_bfloat16*>(p)[at + e0 + j] = __float2bfloat16_rn(v[j]);
            else
                static_cast<float*>(p)[at + e0 + j] = v[j];
        }
    }
}

// The largest number of the warp; -inf of none (NaN alone).
__device__ __forceinline__ float warp_max(float v) {
    return value_of(__reduce_max_sync(kFullMask, v == v ? key_of(v) : key_of(-kInf)));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(kFullMask, v, d);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ float approx_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float approx_exp(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.44269504088896341f));
    return r;
}
// e^(l - m), l <= m. The difference's rounding, half a unit of 2^-24 of up to 128, would be
// up to 32 units of 2^-23 of the result: what l and m have lost in it is put back.
__device__ __forceinline__ float exp_difference(float l, float m) {
    const float d = l - m, l_in = d + m, m_in = l_in - d;
    const float e = expf(d), lost = (l - l_in) - (m - m_in);
    return e > 0.0f ? fmaf(e, lost, e) : e;  // (of infinities nothing is put back)
}
// The weights' divisions are rounded ones: of their K values they cost 1 % of the call. The
// gradient's score, a factor of a few roundings already, takes the approximate one (rounded
// it would cost 3-6 %).
__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }
__device__ __forceinline__ float approx_sigmoid(float l) { return approx_reciprocal(1.0f + expf(-l)); }

// The groups to keep, as a bit mask, from each lane's group (`key` of its worth,
// 0 where it has no expert left).
template <typename Key>
__device__ __forceinline__ uint32_t best_groups(Key key, const RouteArgs& a) {
    const int lane = threadIdx.x & 31;
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.groups; ++g) {
        const Key o = __shfl_sync(kFullMask, key, g);
        rank += g < lane ? (o >= key ? 1 : 0) : (o > key ? 1 : 0);
    }
    return __ballot_sync(kFullMask, lane < a.groups && rank < a.topk_groups && key != 0);
}

// c in 64 bits: of every expert into the warp's `keys` [E] (0: out). Not inlined:
// a few tokens of ten thousand come here.
struct Exact {
    double m, z;
};
__device__ __noinline__ Exact exact_softmax(const RouteArgs& a, int64_t row) {
    const int lane = threadIdx.x & 31;
    float top = -kInf;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, load_logit(a, row + e));
    const double m = warp_max(top);
    double z = 0.0;
    for (int e = lane; e < a.E; e += 32) {
        const double l = load_logit(a, row + e);
        z += l == -kInf ? 0.0 : exp(l - m);
    }
    return {m, warp_sum(z)};
}
__device__ __noinline__ double exact_score(const RouteArgs& a, const Exact& x, float l) {
    const double ld = l;
    return a.softmax ? exp(ld - x.m) / x.z : 1.0 / (1.0 + exp(-ld));
}
__device__ __noinline__ void exact_keys(const RouteArgs& a, int64_t row, unsigned long long* keys) {
    const int lane = threadIdx.x & 31;
    const bool scores = a.bias != nullptr || (a.groups > 1 && a.group_top2);
    Exact x{};
    if (a.softmax && scores) x = exact_softmax(a, row);
    for (int e = lane; e < a.E; e += 32) {
        const float l = load_logit(a, row + e);
        const float b = a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
        double c = l;
        if (scores) c = exact_score(a, x, l) + b;
        keys[e] = l == -kInf || b == -kInf ? 0ull : key_of(c);
    }
    __syncwarp();
}

// The groups that stay, by values in 64 bits; leaves exact_keys.
__device__ __noinline__ uint32_t exact_groups(const RouteArgs& a, int64_t row, unsigned long long* keys) {
    const int lane = threadIdx.x & 31, size = a.group_size;
    exact_keys(a, row, keys);
    unsigned long long worth = 0;
    if (lane < a.groups) {
        unsigned long long first = 0, second = 0;
        for (int i = 0; i < size; ++i) {
            const unsigned long long k = keys[lane * size + i];
            if (k > first) {
                second = first;
                first = k;
            } else if (k > second) {
                second = k;
            }
        }
        worth = first;
        if (a.group_top2 && second != 0) worth = key_of(value_of(first) + value_of(second));
    }
    return best_groups(worth, a);
}

// The choice in 64 bits by the whole warp. Returns the entry of each lane k < K,
// or -1.
__device__ __noinline__ int exact_choice(const RouteArgs& a, int64_t row, unsigned long long* keys) {
    const int lane = threadIdx.x & 31, E = a.E;
    if (a.groups > 1) {
        const int size = E / a.groups;
        const uint32_t kept = exact_groups(a, row, keys);
        for (int e = lane; e < E; e += 32)
            if (!((kept >> (e / size)) & 1)) keys[e] = 0;
        // without a bias experts go by their logits, not by what scores are left
        // of them
        if (a.bias == nullptr)
            for (int e = lane; e < E; e += 32)
                if (keys[e] != 0) keys[e] = key_of(static_cast<double>(load_logit(a, row + e)));
        __syncwarp();
    } else {
        exact_keys(a, row, keys);
    }
    int mine = -1;
    for (int k = 0; k < a.K; ++k) {
        unsigned long long best = 0;
        int at = 0;
        for (int e = lane; e < E; e += 32)
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
        const unsigned long long top = warp_max(best);
        if (top == 0) break;
        const int e = __reduce_min_sync(kFullMask, best == top ? at : 0x7FFFFFFF);
        if (lane == k) mine = e;
        if ((e & 31) == lane) keys[e] = 0;
        __syncwarp();
    }
    return mine;
}

// The order of the warp's candidates (lane i's `e`, -1: none) in 64 bits, among
// which the chosen ones are: returns lane k's.
__device__ __noinline__ int exact_order(const RouteArgs& a, int64_t row, int e) {
    const int lane = threadIdx.x & 31;
    const float l = e >= 0 ? load_logit(a, row + e) : 0.0f;
    unsigned long long key = 0;
    if (a.bias != nullptr) {
        Exact x{};
        if (a.softmax) x = exact_softmax(a, row);
        const double c = exact_score(a, x, l) + (e >= 0 ? __ldg(a.bias + e) : 0.0f);
        if (e >= 0) key = key_of(c);
    } else if (e >= 0) {
        key = key_of(static_cast<double>(l));
    }
    int rank = 0;
    for (int i = 0; i < 32; ++i) {
        const unsigned long long o = __shfl_sync(kFullMask, key, i);
        const int oe = __shfl_sync(kFullMask, e, i);
        rank += (o > key || (o == key && oe < e && oe >= 0)) ? 1 : 0;
    }
    int mine = -1;
    for (int i = 0; i < 32; ++i) {
        const int oe = __shfl_sync(kFullMask, e, i), to = __shfl_sync(kFullMask, rank, i);
        if (oe >= 0 && to == lane) mine = oe;
    }
    return lane < a.K ? mine : -1;
}

// Descending, by odd-even merging.
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[V]) {
#pragma unroll
    for (int p = 1; p < V; p <<= 1)
#pragma unroll
        for (int k = p; k > 0; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = v[i + j], y = v[i + j + k];
                        v[i + j] = max(x, y);
                        v[i + j + k] = min(x, y);
                    }
}

// Scores as the choice first takes them, with approximate functions, and a bound
// on their error. With t = e^-l off by (2^-22 + |l| 2^-23) of itself, sigmoid
// is off by s (1 - s) of that, s (1 - s) |l| < 0.23, and by the reciprocal's
// 2^-23: less than 2^-21. A softmax score, r = 1 / sum: its own exponential by
// 2^-22 + |l - m| 2^-23 of itself, at most 5 2^-24 of the largest score r; the sum
// by its V + 5 additions, 2^-22, and the exponents' part, at most ln E + 1 < 10 times
// 2^-23 of itself; the product and the reciprocal by 2 2^-23.
struct Scores {
    bool softmax;
    float m, r;
    float bound;
    __device__ __forceinline__ float of(float l) const {
        return softmax ? approx_exp(l - m) * r : approx_reciprocal(1.0f + approx_exp(-l));
    }
};

// The groups that stay, where what the choice's integers have lost leaves it open: by
// scores as they are in 32 bits, and where that leaves it open too in 64. The groups'
// experts are those of neighbouring lanes, else 64 bits decide at once.
template <int V, bool kFull>
__device__ __noinline__ uint32_t settle_groups(const RouteArgs& a, int64_t row, const Scores& score,
                                               unsigned long long* keys) {
    if (!kFull || a.group_lanes == 0) return exact_groups(a, row, keys);
    const int lane = threadIdx.x & 31;
    const bool scores = a.bias != nullptr || a.group_top2;
    float l[V], b[V] = {};
    load_part<V, kFull>(a.logits, a.bf16_logits, row, a.E, -kInf, l);
    if (a.bias != nullptr) load_part<V, kFull>(a.bias, false, 0, a.E, -kInf, b);
    // the two largest of a group, over its lanes, to the lane of its number
    auto join = [&](auto& first, auto& second) {
        for (int d = 1; d < a.group_lanes; d <<= 1) {
            const auto f = __shfl_xor_sync(kFullMask, first, d), s = __shfl_xor_sync(kFullMask, second, d);
            second = max(min(first, f), max(second, s));
            first = max(first, f);
        }
        first = __shfl_sync(kFullMask, first, lane * a.group_lanes);
        second = __shfl_sync(kFullMask, second, lane * a.group_lanes);
    };
    if (scores) {
        uint32_t first = 0, second = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool out = l[j] == -kInf || b[j] == -kInf;
            const uint32_t k = out ? 0u : key_of(score.of(l[j]) + b[j]);
            second = max(second, min(first, k));
            first = max(first, k);
        }
        join(first, second);
        float value = value_of(first), error = score.bound + fabsf(value) * 0x1p-23f;
        uint32_t worth = lane < a.groups ? first : 0;
        if (a.group_top2 && second != 0) {
            const float v2 = value_of(second);
            error += score.bound + fabsf(v2) * 0x1p-23f;
            value += v2;
            error += fabsf(value) * 0x1p-23f;
            if (worth != 0) worth = key_of(value);
        }
        const uint32_t kept = best_groups(worth, a);
        const bool stays = (kept >> lane) & 1;
        const uint32_t low =
            __reduce_min_sync(kFullMask, worth != 0 && stays ? key_of(value - error) : 0xFFFFFFFFu);
        const uint32_t high =
            __reduce_max_sync(kFullMask, worth != 0 && !stays ? key_of(value + error) : 0u);
        // (a sum past fp32's range, infinite here, has another value in 64 bits)
        if (high < low && low < key_of(kInf)) return kept;
    }
    Exact x{};
    if (a.softmax && scores) x = exact_softmax(a, row);
    unsigned long long first = 0, second = 0;
#pragma unroll 1
    for (int j = 0; j < V; ++j) {
        const int e = lane * V + j;
        const float le = load_logit(a, row + e), be = a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
        double c = le;
        if (scores) c = exact_score(a, x, le) + be;
        const unsigned long long k = le == -kInf || be == -kInf ? 0ull : key_of(c);
        second = max(second, min(first, k));
        first = max(first, k);
    }
    join(first, second);
    unsigned long long worth = lane < a.groups ? first : 0;
    if (a.group_top2 && worth != 0 && second != 0) worth = key_of(value_of(first) + value_of(second));
    return best_groups(worth, a);
}

// Integers of out experts: at most that of -inf, whatever their last bits.
constexpr uint32_t kOutKey = 0x007FFFFFu;

// kFull: E = 32 V in 16-byte aligned rows.
template <int V, bool kFull>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 7 : 2) route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ unsigned long long smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long* const keys64 = smem + static_cast<int64_t>(warp) * a.E;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.E;
    const bool scores = a.bias != nullptr || (a.groups > 1 && a.group_top2);
    const bool by_logit = a.bias == nullptr;  // what the experts go by, if not the groups
    float l[V], b[V];
    load_part<V, kFull>(a.logits, a.bf16_logits, row, a.E, -kInf, l);
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = 0.0f;
    if (a.bias != nullptr) load_part<V, kFull>(a.bias, false, 0, a.E, -kInf, b);
    constexpr uint32_t kLast = V - 1;
    static_assert((V & (V - 1)) == 0, "a power of two");
    constexpr bool kSort = V <= 16;
    // An integer without its last bits, which say which of the lane's experts it is (the
    // lower the index, the larger). What is lost with them shows where the chosen
    // ones' values are compared.
    auto pack = [&](float c, int j) { return (key_of(c) & ~kLast) | (kLast - j); };

    float m = 0.0f, z = 1.0f;
    if (a.softmax && (scores || !a.renormalize)) {
        float top = -kInf;
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, l[j]);
        m = warp_max(top);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += l[j] == -kInf ? 0.0f : expf(l[j] - m);
        z = warp_sum(sum);
    }
    Scores score{a.softmax, m, approx_reciprocal(z), 0x1p-21f};
    if (a.softmax) score.bound = score.r * static_cast<float>(V + 40) * 0x1p-24f;
    uint32_t key[V];
    if (scores) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = pack(l[j] == -kInf || b[j] == -kInf ? -kInf : score.of(l[j]) + b[j], j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = pack(l[j], j);
    }
    if constexpr (kSort) sort_descending<V>(key);
    if (a.groups > 1) {
        uint32_t first = 0, second = 0;
        const int lanes = kFull && kSort ? a.group_lanes : 0;
        const int size = a.group_size;
        if (lanes > 0) {  // a group's experts are those of `lanes` neighbouring lanes
            first = key[0];
            second = V > 1 ? key[V > 1 ? 1 : 0] : 0;
            for (int d = 1; d < lanes; d <<= 1) {
                const uint32_t f = __shfl_xor_sync(kFullMask, first, d);
                const uint32_t s = __shfl_xor_sync(kFullMask, second, d);
                second = max(min(first, f), max(second, s));
                first = max(first, f);
            }
            // to the lane of the group's number
            first = __shfl_sync(kFullMask, first, lane * lanes);
            second = __shfl_sync(kFullMask, second, lane * lanes);
        } else {
            uint32_t* keys = reinterpret_cast<uint32_t*>(keys64);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = lane * V + static_cast<int>(kLast - (key[j] & kLast));
                if (e < a.E) keys[e] = key[j];
            }
            __syncwarp();
            if (lane < a.groups)
                for (int e = lane * size; e < (lane + 1) * size; ++e) {
                    const uint32_t k = keys[e];
                    second = max(second, min(first, k));
                    first = max(first, k);
                }
            __syncwarp();
        }
        first &= ~kLast;
        second &= ~kLast;
        uint32_t worth = lane < a.groups && first > kOutKey ? first : 0;
        if (a.group_top2 && worth != 0 && second > kOutKey)
            worth = key_of(value_of(first) + value_of(second));
        uint32_t kept = best_groups(worth, a);
        // Are the worst that stays and the best that does not clearly apart? Each is
        // off by two scores' errors, three roundings and twice the lost bits, up to
        // V units of 2^-23 of what was added, of which no part is larger than 1 + the
        // sum's magnitude (by logits: the lost bits alone).
        const bool stays = (kept >> lane) & 1;
        const uint32_t low = __reduce_min_sync(kFullMask, worth != 0 && stays ? worth : 0xFFFFFFFFu);
        const uint32_t high = __reduce_max_sync(kFullMask, stays ? 0u : worth);
        if (high != 0) {
            bool clear = low > (0xFF800000u | kLast) && high < (0xFF800000u | kLast);  // NaN first
            if (!scores) {
                clear |= low > high;
            } else {
                const float v1 = value_of(low), v2 = value_of(high);
                float parts = fabsf(v1) + fabsf(v2);
                if (a.group_top2) parts += 2.0f * warp_max(fabsf(value_of(first)) < kInf ? fabsf(value_of(first)) : 0.0f);
                clear |= v1 - v2 > 4.0f * score.bound + parts * (static_cast<float>(2 * V + 4) * 0x1p-23f);
            }
            if (!clear) kept = settle_groups<V, kFull>(a, row, score, keys64);
        }
        if (scores && by_logit) {  // from here on by logits
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = pack(l[j], j);
            if constexpr (kSort) sort_descending<V>(key);
        }
        if (lanes > 0) {  // (a lane whose largest is out takes no part)
            key[0] = (kept >> (lane >> a.log_group_lanes)) & 1 ? key[0] : 0;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = lane * V + static_cast<int>(kLast - (key[j] & kLast));
                // (e / size: a float's error is far below half of 1 / size)
                const int g = static_cast<int>((static_cast<float>(e) + 0.5f) * a.group_part);
                if (e >= a.E || !((kept >> g) & 1)) key[j] = key[j] & kLast;
            }
            if constexpr (kSort) sort_descending<V>(key);
        }
    }
    // A round: the largest that is left becomes lane k's (and the last one's).
    // (its index: the lane it was found in, and the last bits)
    int mine_owner = -1, last_owner = -1;
    uint32_t mine_head = 0, last_head = 0;
    auto take = [&](int k) {
        uint32_t head = key[0];
        if constexpr (!kSort) {
#pragma unroll
            for (int j = 1; j < V; ++j) head = max(head, key[j]);
        }
        const uint32_t most = __reduce_max_sync(kFullMask, head & ~kLast);
        if (most <= kOutKey) return false;
        const int owner = __ffs(__ballot_sync(kFullMask, (head & ~kLast) == most)) - 1;
        last_owner = owner;
        last_head = __shfl_sync(kFullMask, head, owner);
        const bool won = lane == owner, here = lane == k;
        mine_owner = here ? last_owner : mine_owner;
        mine_head = here ? last_head : mine_head;
        if constexpr (kSort) {
#pragma unroll
            for (int j = 0; j + 1 < V; ++j) key[j] = won ? key[j + 1] : key[j];
            key[V - 1] = won ? 0u : key[V - 1];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = won && key[j] == head ? 0u : key[j];
        }
        return true;
    };
    // Whether one is larger than the next by more than both may be off: their own
    // error, c's rounding and the lost bits, up to V units of 2^-23 of the value. (By
    // logits only the lost bits matter. NaN goes before all.)
    auto clear = [&](uint32_t k1, uint32_t k2) {
        k1 &= ~kLast;
        k2 &= ~kLast;
        if (by_logit) return k1 > k2;
        const float c1 = value_of(k1), c2 = value_of(k2);
        const float off =
            2.0f * score.bound + (fabsf(c1) + fabsf(c2)) * (static_cast<float>(V + 1) * 0x1p-23f);
        return c1 - c2 > off || (k1 > 0xFF800000u && k2 <= 0xFF800000u);
    };
    int n = 0;  // K, and the one that the last of them has to be larger than
    while (n <= a.K && take(n)) ++n;
    auto index = [&](int owner, uint32_t head) {
        return owner < 0 ? -1 : owner * V + static_cast<int>(kLast - (head & kLast));
    };
    int mine = index(mine_owner, mine_head);
    {
        uint32_t next_head = __shfl_down_sync(kFullMask, mine_head, 1);
        if (lane == 31) next_head = last_head;  // (K = 32)
        bool doubt = lane < min(n - 1, a.K) && !clear(mine_head, next_head);
        const uint32_t first_doubts = __ballot_sync(kFullMask, doubt);
        if (first_doubts != 0) {
            // with the lost bits back, and equal ones by their index
            auto settled = [&](int e1, float l1, int e2, float l2) {
                if (by_logit) {
                    const uint32_t k1 = key_of(l1), k2 = key_of(l2);
                    return k1 > k2 || (k1 == k2 && e1 < e2);
                }
                const float b1 = __ldg(a.bias + e1), b2 = __ldg(a.bias + e2);
                const float c1 = score.of(l1) + b1, c2 = score.of(l2) + b2;
                const float off = 2.0f * score.bound + (fabsf(c1) + fabsf(c2)) * 0x1p-22f;
                return (l1 == l2 && b1 == b2 && e1 < e2) || c1 - c2 > off ||
                       (c1 != c1 && (c2 == c2 || e1 < e2));
            };
            int next = __shfl_down_sync(kFullMask, mine, 1);
            if (lane == 31) next = index(last_owner, last_head);
            if (doubt)
                doubt = !settled(mine, load_logit(a, row + mine), next, load_logit(a, row + next));
            // Is the last of the K also larger than what was not taken, of which the lost
            // bits may hide a larger one?
            bool beaten = false;
            if ((first_doubts >> (a.K - 1)) & 1) {
                const int in = __shfl_sync(kFullMask, mine, a.K - 1);
                const uint32_t in_head = __shfl_sync(kFullMask, mine_head, a.K - 1);
                const float in_l = load_logit(a, row + in);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // (of sorted ones none follows one that is out)
                    if (((kSort ? key[0] : key[j]) & ~kLast) <= kOutKey) continue;
                    if ((key[j] & ~kLast) <= kOutKey || clear(in_head, key[j])) continue;
                    const int e = index(lane, key[j]);
                    beaten |= !settled(in, in_l, e, load_logit(a, row + e));
                }
            }
            if (__any_sync(kFullMask, doubt || beaten)) {
                // the candidates for the K places, down to a clear step (with an order in
                // doubt the last of the K need not be the least of them)
                int count = a.K;
                bool found = true;
                if ((first_doubts >> (a.K - 1)) & 1) {
                    found = false;
                    for (count = n; !found && count < 32;) {
                        const uint32_t before = last_head;
                        if (!take(count) || clear(before, last_head))
                            found = true;
                        else
                            ++count;
                    }
                    mine = index(mine_owner, mine_head);
                }
                mine = found ? exact_order(a, row, lane < count ? mine : -1)
                             : exact_choice(a, row, keys64);
            }
        }
    }
    if (lane >= a.K) mine = -1;
    const float lk = mine >= 0 ? load_logit(a, row + mine) : -kInf;

    // weights: lane k's
    float w = 0.0f;
    if (a.renormalize) {
        if (!a.softmax && __any_sync(kFullMask, lk >= 0.0f)) {
            w = mine >= 0 ? sigmoid(lk) : 0.0f;
        } else if (const float high = warp_max(lk); a.softmax) {
            w = mine >= 0 ? exp_difference(lk, high) : 0.0f;
        } else {
            // by e^high, so that scores below fp32's range keep their ratios
            w = mine >= 0 ? __fdiv_rn(exp_difference(lk, high) * (1.0f + expf(high)), 1.0f + expf(lk))
                          : 0.0f;
        }
        const float sum = warp_sum(w);
        w = mine >= 0 ? __fdiv_rn(w, sum) : 0.0f;
    } else if (mine >= 0) {
        w = a.softmax ? __fdiv_rn(exp_difference(lk, m), z) : sigmoid(lk);
    }
    if (lane < a.K) {
        a.topk_idx[t * a.K + lane] = mine;
        a.topk_w[t * a.K + lane] = w * a.scale;
    }
}

// The gradient. With g_k the gradient of w_k times scale, over the chosen
// entries (p_k: the renormalised weights, before scale):
//   softmax               d_e = s_e (sum over k with idx_k = e of g_k - sum_j g_j s_j)
//   softmax, renormalised d_k = p_k (g_k - sum_j g_j p_j)
//   sigmoid               d_k = g_k s_k (1 - s_k)
//   sigmoid, renormalised d_k = p_k (1 - s_k) (g_k - sum_j g_j p_j)
// and zero where nothing is said. A warp to a token: lane k an entry, then the row,
// of which a lane holds V neighbouring experts as in the choice (V = 0: in shared
// memory, for more than 8). An expert that a token has twice gets the sum of
// both, in their order.
template <int V, bool kFull>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ unsigned long long smem[];
    constexpr bool kHeld = V > 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* const d_row = reinterpret_cast<float*>(smem) + static_cast<int64_t>(warp) * a.E;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.E;
    const bool dense = a.softmax && !a.renormalize;

    int64_t idx = lane < a.K ? __ldg(a.topk_idx + t * a.K + lane) : -1;
    const float dw = lane < a.K ? __ldg(a.d_topk_w + t * a.K + lane) : 0.0f;
    float l[kHeld ? V : 1];
    if constexpr (kHeld) {
        if (dense) load_part<V, kFull>(a.logits, a.bf16_logits, row, a.E, -kInf, l);
    }
    if (idx < -1 || idx >= a.E) {
        set_status(a.status, EP_ERR_BAD_EXPERT);
        idx = -1;
    }
    const int mine = static_cast<int>(idx);
    const float lk = mine >= 0 ? load_logit(a, row + mine) : -kInf;
    const float g = dw * a.scale;
    const bool live = lk != -kInf;  // (an expert taken out has score 0)
    float m = 0.0f, z = 1.0f;
    if (dense) {
        float top = -kInf, sum = 0.0f;
        if constexpr (kHeld) {
#pragma unroll
            for (int j = 0; j < V; ++j) top = fmaxf(top, l[j]);
            m = warp_max(top);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                l[j] = l[j] == -kInf ? 0.0f : expf(l[j] - m);
                sum += l[j];
            }
        } else {
            for (int e = lane; e < a.E; e += 32) top = fmaxf(top, load_logit(a, row + e));
            m = warp_max(top);
            for (int e = lane; e < a.E; e += 32) {
                const float v = load_logit(a, row + e);
                sum += v == -kInf ? 0.0f : expf(v - m);
            }
        }
        z = warp_sum(sum);
    }
    float d = 0.0f, dot = 0.0f;
    if (a.renormalize) {
        const float high = warp_max(lk);
        float p = 0.0f;
        if (live) {
            if (a.softmax)
                p = exp_difference(lk, high);
            else if (high >= 0.0f)
                p = approx_sigmoid(lk);
            else
                p = __fdiv_rn(exp_difference(lk, high) * (1.0f + expf(high)), 1.0f + expf(lk));
        }
        const float sum = warp_sum(p);
        p = live ? __fdiv_rn(p, sum) : 0.0f;
        dot = warp_sum(live ? g * p : 0.0f);
        d = live ? p * (g - dot) : 0.0f;
        if (live && !a.softmax) d *= approx_sigmoid(-lk);
    } else if (a.softmax) {
        dot = warp_sum(live ? g * __fdiv_rn(exp_difference(lk, m), z) : 0.0f);
        d = live ? g : 0.0f;
    } else if (live) {
        d = g * approx_sigmoid(lk) * approx_sigmoid(-lk);
    }
    if constexpr (kHeld) {
        float out[V] = {};
        const int e0 = lane * V;
        for (int k = 0; k < a.K; ++k) {
            const int e = __shfl_sync(kFullMask, mine, k) - e0;
            const float dk = __shfl_sync(kFullMask, d, k);
#pragma unroll
            for (int j = 0; j < V; ++j)
                out[j] += e == j ? dk : 0.0f;
        }
        if (dense) {
            const float r = __fdiv_rn(1.0f, z);
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = l[j] == 0.0f ? 0.0f : l[j] * r * (out[j] - dot);
        }
        store_part<V, kFull>(a.d_logits, a.bf16_logits, row, a.E, out);
    } else {
        for (int e = lane; e < a.E; e += 32) d_row[e] = 0.0f;
        float sum = 0.0f;
        bool first = mine >= 0;
        for (int k = 0; k < a.K; ++k) {
            const int e = __shfl_sync(kFullMask, mine, k);
            const float dk = __shfl_sync(kFullMask, d, k);
            if (mine >= 0 && e == mine) {
                sum += dk;
                if (k < lane) first = false;
            }
        }
        __syncwarp();
        if (first) d_row[mine] = sum;
        __syncwarp();
        for (int e = lane; e < a.E; e += 32) {
            float v = d_row[e];
            if (dense) {
                const float le = load_logit(a, row + e);
                v = le == -kInf ? 0.0f : __fdiv_rn(expf(le - m), z) * (v - dot);
            }
            if (a.bf16_logits)
                static_cast<__nv_bfloat16*>(a.d_logits)[row + e] = __float2bfloat16_rn(v);
            else
                static_cast<float*>(a.d_logits)[row + e] = v;
        }
    }
}

// kernel(a) with a token to a warp.
cudaError_t launch_tokens(void (*kern)(RouteArgs), const RouteArgs& a, size_t smem,
                          cudaStream_t stream) {
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(kern, static_cast<int>((a.T + kWarps - 1) / kWarps), kWarps * 32, smem,
                            stream, a);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int V>
cudaError_t launch_route_v(RouteArgs a, size_t smem, cudaStream_t stream) {
    if (a.E != 32 * V || !aligned16(a.logits) || !aligned16(a.bias))
        return launch_tokens(route_kernel<V, false>, a, smem, stream);
    const int lanes = 32 / a.groups;
    if (a.groups > 1 && lanes * a.groups == 32 && (lanes & (lanes - 1)) == 0) {
        a.group_lanes = lanes;
        while ((1 << a.log_group_lanes) < lanes) ++a.log_group_lanes;
    }
    return launch_tokens(route_kernel<V, true>, a, smem, stream);
}

template <int V>
cudaError_t launch_route_grad_v(const RouteArgs& a, cudaStream_t stream) {
    if (a.E != 32 * V || !aligned16(a.logits) || !aligned16(a.d_logits))
        return launch_tokens(route_grad_kernel<V, false>, a, 0, stream);
    return launch_tokens(route_grad_kernel<V, true>, a, 0, stream);
}

}  // namespace

cudaError_t launch_route(RouteArgs a, cudaStream_t stream) {
    a.group_size = a.E / a.groups;
    a.group_part = 1.0f / static_cast<float>(a.group_size);
    const size_t smem = sizeof(unsigned long long) * kWarps * static_cast<size_t>(a.E);
    const int v = (a.E + 31) / 32;
    if (v <= 1) return launch_route_v<1>(a, smem, stream);
    if (v <= 2) return launch_route_v<2>(a, smem, stream);
    if (v <= 4) return launch_route_v<4>(a, smem, stream);
    if (v <= 8) return launch_route_v<8>(a, smem, stream);
    if (v <= 16) return launch_route_v<16>(a, smem, stream);
    if (v <= 32) return launch_route_v<32>(a, smem, stream);
    return launch_route_v<128>(a, smem, stream);
}

cudaError_t launch_route_grad(const RouteArgs& a, cudaStream_t stream) {
    const int v = (a.E + 31) / 32;
    if (v <= 1) return launch_route_grad_v<1>(a, stream);
    if (v <= 2) return launch_route_grad_v<2>(a, stream);
    if (v <= 4) return launch_route_grad_v<4>(a, stream);
    if (v <= 8) return launch_route_grad_v<8>(a, stream);
    return launch_tokens(route_grad_kernel<0, false>, a,
                         sizeof(float) * kWarps * static_cast<size_t>(a.E), stream);
}

}  // namespace ep
