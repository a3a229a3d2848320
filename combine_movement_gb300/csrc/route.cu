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
// right answer: c is computed in 32 with a bound on its error, and a token
// whose order the bound leaves open (a few of ten thousand) goes through the
// choice again in 64 bits (route_exact).
//
// Mapping: a warp to a token; lane i holds the V = ceil(E / 32) experts from
// i * V on, as fp32 values and as integers of the same order, so that the K
// rounds of the choice are one warp-wide integer maximum and one ballot each and
// ties fall to the lower index by themselves.
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
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 + 0 = +0)
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    if (v != v) return ~0ull;
    const long long b = __double_as_longlong(v + 0.0);
    return b < 0 ? ~static_cast<unsigned long long>(b)
                 : static_cast<unsigned long long>(b) | 0x8000000000000000ull;
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

__device__ __forceinline__ float warp_max(float v) {  // NaN only of NaN alone
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, d));
    return v;
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

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.0f, 1.0f + expf(-l)); }

// The groups to keep, as a bit mask, from each lane's group (`key` of its worth,
// 0 where it has no expert left).
template <typename Key>
__device__ __forceinline__ uint32_t best_groups(Key key, const RouteArgs& a) {
    const int lane = threadIdx.x & 31;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const Key o = __shfl_sync(kFullMask, key, g);
        rank += (o > key || (o == key && g < lane)) ? 1 : 0;
    }
    return __ballot_sync(kFullMask, lane < a.groups && rank < a.topk_groups && key != 0);
}

// The choice in 64 bits, by the whole warp; `keys` is the warp's [E]. Returns
// the entry of each lane k < K, or -1.
__device__ __noinline__ int route_exact(const RouteArgs& a, int64_t t, unsigned long long* keys) {
    const int lane = threadIdx.x & 31, E = a.E;
    const int64_t row = t * E;
    double m = 0.0, z = 1.0;
    if (a.softmax) {
        float top = -kInf;
        for (int e = lane; e < E; e += 32) top = fmaxf(top, load_logit(a, row + e));
        m = warp_max(top);
        z = 0.0;
        for (int e = lane; e < E; e += 32) {
            const double l = load_logit(a, row + e);
            z += l == -kInf ? 0.0 : exp(l - m);
        }
        z = warp_sum(z);
    }
    for (int e = lane; e < E; e += 32) {
        const float l = load_logit(a, row + e);
        const float b = a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
        const double ld = l;
        const double s = a.softmax ? exp(ld - m) / z : 1.0 / (1.0 + exp(-ld));
        keys[e] = l == -kInf || b == -kInf ? 0ull : key_of(s + b);
    }
    __syncwarp();
    if (a.groups > 1) {
        const int size = E / a.groups;
        unsigned long long worth = 0;
        if (lane < a.groups) {
            unsigned long long first = 0, second = 0;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const unsigned long long k = keys[e];
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
        const uint32_t kept = best_groups(worth, a);
        for (int e = lane; e < E; e += 32)
            if (!((kept >> (e / size)) & 1)) keys[e] = 0;
        // without a bias experts go by their logits, not by what scores are left
        // of them
        if (a.bias == nullptr)
            for (int e = lane; e < E; e += 32)
                if (keys[e] != 0) keys[e] = key_of(static_cast<double>(load_logit(a, row + e)));
        __syncwarp();
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

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
    extern __shared__ unsigned long long smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long* const keys64 = smem + static_cast<int64_t>(warp) * a.E;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.E;
    const int e0 = lane * V;

    float l[V];
    float top = -kInf;
    bool odd = false;  // whether the choice has to be made again in 64 bits
#pragma unroll
    for (int j = 0; j < V; ++j) {
        l[j] = e0 + j < a.E ? load_logit(a, row + e0 + j) : -kInf;
        top = fmaxf(top, l[j]);
    }
    const bool scores = a.bias != nullptr || (a.groups > 1 && a.group_top2);
    float m = 0.0f, z = 1.0f;
    if (a.softmax) {
        m = warp_max(top);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) sum += l[j] == -kInf ? 0.0f : expf(l[j] - m);
        z = warp_sum(sum);
    }
    uint32_t key[V];
    float c[V];
    // bound on a score's error: sigmoid's exponential, sum and division are off by
    // less than 4 units of 2^-23 together; a softmax score besides by the sum's
    // V + 5 additions and by l - m's rounding, |l - m| 2^-24 times the score,
    // at most 0.37 2^-24 of the largest
    const float bound =
        a.softmax ? __fdiv_rn(static_cast<float>(V + 20), z) * 0x1p-23f : 0x1p-20f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float b = 0.0f;
        if (a.bias != nullptr && e0 + j < a.E) b = __ldg(a.bias + e0 + j);
        c[j] = l[j];
        if (scores) {
            const float s = a.softmax ? __fdiv_rn(expf(l[j] - m), z) : sigmoid(l[j]);
            c[j] = s + b;
        }
        const bool out = l[j] == -kInf || b == -kInf;
        key[j] = out ? 0u : key_of(c[j]);
        odd |= scores && !out && c[j] != c[j];
    }
    const int size = a.E / a.groups;
    if (a.groups > 1) {
        // each lane's group from shared memory
        uint32_t* keys = reinterpret_cast<uint32_t*>(keys64);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j < a.E) keys[e0 + j] = key[j];
        __syncwarp();
        uint32_t worth = 0;
        float value = 0.0f, error = 0.0f;
        if (lane < a.groups) {
            uint32_t first = 0, second = 0;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const uint32_t k = keys[e];
                second = max(second, min(first, k));
                first = max(first, k);
            }
            auto of = [](uint32_t k) {
                return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
            };
            worth = first;
            if (first != 0) {
                value = of(first);
                error = bound + fabsf(value) * 0x1p-23f;
                if (a.group_top2 && second != 0) {
                    error += bound + fabsf(of(second)) * 0x1p-23f;
                    value += of(second);
                    error += fabsf(value) * 0x1p-23f;
                    worth = key_of(value);
                }
            }
        }
        const uint32_t kept = best_groups(worth, a);
        if (scores) {
            const bool has = lane < a.groups && worth != 0, mine = (kept >> lane) & 1;
            const float low = -warp_max(has && mine ? error - value : -kInf);
            const float high = warp_max(has && !mine ? value + error : -kInf);
            odd |= high > -kInf && !(low > high);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e0 + j >= a.E || !((kept >> ((e0 + j) / size)) & 1)) key[j] = 0;
        if (scores && a.bias == nullptr) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] != 0) key[j] = key_of(l[j]);
        }
        __syncwarp();
    }
    // K rounds, and one more where the next value decides whether the last of
    // them is settled
    const bool check = a.bias != nullptr;
    int mine = -1;
    float c_before = 0.0f, l_before = 0.0f, b_before = 0.0f;
    for (int k = 0; k < a.K + (check ? 1 : 0); ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) best = max(best, key[j]);
        const uint32_t most = __reduce_max_sync(kFullMask, best);
        if (most == 0) break;
        const int owner = __ffs(__ballot_sync(kFullMask, best == most)) - 1;
        int at = 0;
        float lv = 0.0f, cv = 0.0f;
        if (lane == owner) {
#pragma unroll
            for (int j = V - 1; j >= 0; --j)
                if (key[j] == most) {
                    at = j;
                    lv = l[j];
                    cv = c[j];
                }
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == at) key[j] = 0;
        }
        const int e = __shfl_sync(kFullMask, e0 + at, owner);
        if (k < a.K && lane == k) mine = e;
        if (check) {
            lv = __shfl_sync(kFullMask, lv, owner);
            cv = __shfl_sync(kFullMask, cv, owner);
            const float b = __ldg(a.bias + e);
            if (k > 0 && !(lv == l_before && b == b_before))
                odd |= !(c_before - cv > 2.0f * bound + (fabsf(c_before) + fabsf(cv)) * 0x1p-22f);
            c_before = cv;
            l_before = lv;
            b_before = b;
        }
    }
    if (__any_sync(kFullMask, odd)) mine = route_exact(a, t, keys64);

    // weights: lane k's
    const float lk = mine >= 0 ? load_logit(a, row + mine) : -kInf;
    float w = 0.0f;
    if (a.renormalize) {
        const float high = warp_max(lk);
        if (a.softmax) {
            w = mine >= 0 ? expf(lk - high) : 0.0f;
        } else if (high >= 0.0f) {
            w = mine >= 0 ? sigmoid(lk) : 0.0f;
        } else {
            // by e^high, so that scores below fp32's range keep their ratios
            w = mine >= 0 ? __fdiv_rn(expf(lk - high) * (1.0f + expf(high)), 1.0f + expf(lk)) : 0.0f;
        }
        const float sum = warp_sum(w);
        w = mine >= 0 ? __fdiv_rn(w, sum) : 0.0f;
    } else if (mine >= 0) {
        w = a.softmax ? __fdiv_rn(expf(lk - m), z) : sigmoid(lk);
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
// and zero where nothing is said. A warp to a token: lane k an entry, then the row
// through shared memory. An expert that a token has twice gets the sum of both, in
// their order.
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const RouteArgs a) {
    extern __shared__ unsigned long long smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* const d_row = reinterpret_cast<float*>(smem) + static_cast<int64_t>(warp) * a.E;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    const int64_t row = t * a.E;

    int64_t idx = lane < a.K ? __ldg(a.topk_idx + t * a.K + lane) : -1;
    if (idx < -1 || idx >= a.E) {
        set_status(a.status, EP_ERR_BAD_EXPERT);
        idx = -1;
    }
    const bool on = idx >= 0;
    const float lk = on ? load_logit(a, row + idx) : -kInf;
    const float g = on ? __ldg(a.d_topk_w + t * a.K + lane) * a.scale : 0.0f;
    const bool dense = a.softmax && !a.renormalize;
    float m = 0.0f, z = 1.0f;
    if (dense) {
        float top = -kInf;
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, load_logit(a, row + e));
        m = warp_max(top);
        float sum = 0.0f;
        for (int e = lane; e < a.E; e += 32) {
            const float l = load_logit(a, row + e);
            sum += l == -kInf ? 0.0f : expf(l - m);
        }
        z = warp_sum(sum);
    }
    const bool live = on && lk != -kInf;  // (an expert taken out has score 0)
    float d = 0.0f, dot = 0.0f;
    if (a.renormalize) {
        const float high = warp_max(lk);
        float p = 0.0f;
        if (live) {
            if (a.softmax)
                p = expf(lk - high);
            else if (high >= 0.0f)
                p = sigmoid(lk);
            else
                p = __fdiv_rn(expf(lk - high) * (1.0f + expf(high)), 1.0f + expf(lk));
        }
        const float sum = warp_sum(p);
        p = live ? __fdiv_rn(p, sum) : 0.0f;
        dot = warp_sum(live ? g * p : 0.0f);
        d = live ? p * (g - dot) : 0.0f;
        if (live && !a.softmax) d *= sigmoid(-lk);
    } else if (a.softmax) {
        dot = warp_sum(live ? g * __fdiv_rn(expf(lk - m), z) : 0.0f);
        d = live ? g : 0.0f;
    } else if (live) {
        d = g * sigmoid(lk) * sigmoid(-lk);
    }
    for (int e = lane; e < a.E; e += 32) d_row[e] = 0.0f;
    float sum = 0.0f;
    bool first = on;
    for (int k = 0; k < a.K; ++k) {
        const int e = __shfl_sync(kFullMask, static_cast<int>(idx), k);
        const float dk = __shfl_sync(kFullMask, d, k);
        if (on && e == static_cast<int>(idx)) {
            sum += dk;
            if (k < lane) first = false;
        }
    }
    __syncwarp();
    if (first) d_row[idx] = sum;
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) {
        float v = d_row[e];
        if (dense) {
            const float l = load_logit(a, row + e);
            v = l == -kInf ? 0.0f : __fdiv_rn(expf(l - m), z) * (v - dot);
        }
        if (a.bf16_logits)
            static_cast<__nv_bfloat16*>(a.d_logits)[row + e] = __float2bfloat16_rn(v);
        else
            static_cast<float*>(a.d_logits)[row + e] = v;
    }
}

template <int V>
cudaError_t launch_route_v(const RouteArgs& a, size_t smem, cudaStream_t stream) {
    auto kern = route_kernel<V>;
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(kern, static_cast<int>((a.T + kWarps - 1) / kWarps), kWarps * 32, smem,
                            stream, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
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
    const size_t smem = sizeof(float) * kWarps * static_cast<size_t>(a.E);
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(
            route_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_dependent(route_grad_kernel, static_cast<int>((a.T + kWarps - 1) / kWarps),
                            kWarps * 32, smem, stream, a);
}

}  // namespace ep
