// linear_grad.cu -- what comes before the dense products' gradients: from the
// gradient dy of y = act(z) + residual,
//
//   dz[m, n]  = bf16_rne( dy[m, n] * act'(z[m, n]) )
//   d_bias[n] = sum over m of dz[m, n] before its rounding     (fp32)
//
// (gated, z = [g, u]: dz = [dy u silu'(g), dy silu(g)]). The products that
// follow take bf16 operands, so dz is rounded to it, as z was when it was kept; the
// sums are not.
//
// Mapping: a CTA to a strip of 64 columns (32 where they are odd in number;
// a quarter of those where few columns are summed) and every c-th group of rows, a thread to a few columns of a row; a strip's
// rows go to the c CTAs of a cluster. A thread adds its rows, the CTA its threads,
// the cluster its CTAs, each in a fixed order, so that equal calls give equal
// bits. All of a thread's loads go out before anything is made of them: a shift or a
// branch between two waits for the first (4096 x 1075: 44 us, so 14).
//
// Bound by memory, or for sums and odd rows by what is in flight: 4096 x 2048 gated 16.2
// us (5.2 TB/s), 16384 x 2048 54.5 (6.2); with d_bias, for which a strip has eight
// CTAs, 19.2 and for 16384 x 7168, silu, 146 (4.8).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "kernels.cuh"
#include "linear_math.cuh"
#include "product.cuh"

namespace ep {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

// W values of a row as they lie in memory.
template <int W>
struct Raw {
    uint32_t bits[W];
};
template <int W>
__device__ __forceinline__ Raw<W> load_row(const void* p, bool f32, int64_t at) {
    Raw<W> r;
    if (f32) {
        const uint32_t* q = static_cast<const uint32_t*>(p) + at;
        if constexpr (W == 1) {
            r.bits[0] = __ldg(q);
        } else if constexpr (W == 2) {
            const uint2 f = __ldg(reinterpret_cast<const uint2*>(q));
            r.bits[0] = f.x, r.bits[1] = f.y;
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 f = __ldg(reinterpret_cast<const uint4*>(q + i));
                r.bits[i] = f.x, r.bits[i + 1] = f.y, r.bits[i + 2] = f.z, r.bits[i + 3] = f.w;
            }
        }
        return r;
    }
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if constexpr (W == 1) {
        r.bits[0] = __ldg(q);  // (shifted where it is used: here it would wait for the load)
    } else if constexpr (W == 2) {
        r.bits[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
    } else if constexpr (W == 4) {
        const uint2 f = __ldg(reinterpret_cast<const uint2*>(q));
        r.bits[0] = f.x, r.bits[1] = f.y;
    } else {
        const uint4 f = __ldg(reinterpret_cast<const uint4*>(q));
        r.bits[0] = f.x, r.bits[1] = f.y, r.bits[2] = f.z, r.bits[3] = f.w;
    }
    return r;
}
// Value i of them.
template <int W>
__device__ __forceinline__ float value(const Raw<W>& r, bool f32, int i) {
    if (f32) return __uint_as_float(r.bits[i]);
    if (W == 1) return __uint_as_float(r.bits[0] << 16);
    return __uint_as_float(i % 2 == 0 ? r.bits[i / 2] << 16 : r.bits[i / 2] & 0xFFFF0000u);
}
template <int W>
__device__ __forceinline__ void store_row(uint16_t* q, const float (&v)[W]) {
    if constexpr (W == 1) {
        *q = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else if constexpr (W == 2) {
        *reinterpret_cast<uint32_t*>(q) = pack_bf16x2(v[0], v[1]);
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
        st_v4(q, round8(v));
    }
}

// W columns to a thread, kLanes threads to a row's part.
// kSums: d_bias is asked for.
template <int W, int kLanes, bool kGated, bool kF32, bool kSums>
__global__ void __launch_bounds__(kThreads, kSums ? 2 : 3) act_grad_kernel(const ActGradArgs a) {
    constexpr int kHalves = kGated ? 2 : 1, kRows = kThreads / kLanes, kCols = W * kLanes;
    constexpr int kAtOnce = W == 8 ? (kGated || kF32 ? 2 : 4) : W == 4 ? 4 : W == 2 ? 8 : 16;  // rows whose loads are in flight
    __shared__ float part[kThreads / 32][kHalves][kCols];
    __shared__ float total[kHalves][kCols];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cl = threadIdx.x % kLanes, rl = threadIdx.x / kLanes;
    const int64_t col = static_cast<int64_t>(blockIdx.y) * kCols + cl * W;
    const bool in = col < a.n;  // (W divides n)
    float sum[kHalves][W] = {};
    const int64_t wide = kHalves * a.n;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows + rl; r0 < a.m && in;
         r0 += kAtOnce * step) {
        Raw<W> dy[kAtOnce], z[kAtOnce], zu[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t r = min(r0 + j * step, a.m - 1);  // (rows past the last: it again)
            dy[j] = load_row<W>(a.dy, kF32, r * a.n + col);
            if (a.act != EP_ACT_NONE) z[j] = load_row<W>(a.z, false, r * wide + col);
            if (kGated) zu[j] = load_row<W>(a.z, false, r * wide + a.n + col);
        }
        // (what the activation is, is asked once for all of them)
        auto each = [&](auto slope) {
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int64_t r = r0 + j * step;
                if (r >= a.m) continue;
                float g[W], u[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float d = value<W>(dy[j], kF32, i), v = value<W>(z[j], false, i);
                    if (kGated) {
                        u[i] = d * silu(v);
                        g[i] = d * value<W>(zu[j], false, i) * silu_slope(v);
                        if (kSums) sum[kHalves - 1][i] += u[i];
                    } else {
                        g[i] = slope(d, v);
                    }
                    if (kSums) sum[0][i] += g[i];
                }
                if (a.dz != nullptr) {
                    store_row<W>(a.dz + r * a.pitch + col, g);
                    if (kGated) store_row<W>(a.dz + r * a.pitch + a.n + col, u);
                }
            }
        };
        if (kGated || a.act == EP_ACT_NONE)
            each([](float d, float) { return d; });
        else if (a.act == EP_ACT_RELU)
            each([](float d, float v) { return d * activate_slope(v, EP_ACT_RELU); });
        else if (a.act == EP_ACT_GELU)
            each([](float d, float v) { return d * activate_slope(v, EP_ACT_GELU); });
        else
            each([](float d, float v) { return d * activate_slope(v, EP_ACT_SILU); });
    }
    if constexpr (kSums) {
        // over the warp's rows, then the CTA's warps, then the cluster's CTAs
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int i = 0; i < W; ++i) {
#pragma unroll
                for (int d = kLanes; d < 32; d <<= 1)
                    sum[h][i] += __shfl_xor_sync(kFullMask, sum[h][i], d);
                if (lane < kLanes) part[warp][h][cl * W + i] = sum[h][i];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < kHalves * kCols; i += kThreads) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) s += part[w][i / kCols][i % kCols];
            total[i / kCols][i % kCols] = s;
        }
        cluster_arrive();
        cluster_wait();
        if (cluster_rank() == 0) {
            for (int i = threadIdx.x; i < kHalves * kCols; i += kThreads) {
                const int64_t c = static_cast<int64_t>(blockIdx.y) * kCols + i % kCols;
                if (c >= a.n) continue;
                float s = 0.0f;
                for (uint32_t p = 0; p < gridDim.x; ++p)
                    s += load_cluster_f32(cluster_map(smem_u32(&total[i / kCols][i % kCols]), p));
                a.d_bias[i / kCols * a.n + c] = s;
            }
        }
        cluster_arrive();
        cluster_wait();  // no CTA reads this one's sums any more
    }
}

template <int W, int kLanes, bool kGated, bool kF32>
cudaError_t launch(const ActGradArgs& a, int num_sms, bool partition, cudaStream_t stream) {
    constexpr int kRows = kThreads / kLanes, kCols = W * kLanes;
    const int64_t strips = (a.n + kCols - 1) / kCols;
    const int64_t groups = a.m > 0 ? (a.m + kRows - 1) / kRows : 1;
    // with sums the grid's rows of CTAs are a cluster, of one where a partition's SMs
    // may not hold more; else as many as there is work for
    int64_t parts = 8 * num_sms / strips + 1;
    if (a.d_bias != nullptr) {
        int64_t c = partition ? 1 : kMaxCluster;
        while (c > 1 && c > groups) c /= 2;
        parts = c;
    } else if (parts > groups) {
        parts = groups;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(parts), static_cast<unsigned>(strips));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = launch_overlap_allowed(stream) ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.d_bias != nullptr ? static_cast<unsigned>(parts) : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (a.d_bias == nullptr)
        return cudaLaunchKernelEx(&cfg, act_grad_kernel<W, kLanes, kGated, kF32, false>, a);
    return cudaLaunchKernelEx(&cfg, act_grad_kernel<W, kLanes, kGated, kF32, true>, a);
}

// Strips of a quarter of the columns where the clusters of whole ones leave SMs
// idle.
template <int W, int kLanes, bool kGated, bool kF32>
cudaError_t launch_lanes(const ActGradArgs& a, int num_sms, bool partition, cudaStream_t stream) {
    const int64_t strips = (a.n + W * kLanes - 1) / (W * kLanes);
    if (a.d_bias != nullptr && strips * (partition ? 1 : kMaxCluster) < num_sms)
        return launch<W, kLanes / 4, kGated, kF32>(a, num_sms, partition, stream);
    return launch<W, kLanes, kGated, kF32>(a, num_sms, partition, stream);
}

template <bool kGated, bool kF32>
cudaError_t launch_width(const ActGradArgs& a, int num_sms, bool partition, cudaStream_t stream) {
    if (a.n % 8 == 0) return launch_lanes<8, 8, kGated, kF32>(a, num_sms, partition, stream);
    if (a.n % 4 == 0) return launch_lanes<4, 16, kGated, kF32>(a, num_sms, partition, stream);
    if (a.n % 2 == 0) return launch_lanes<2, 32, kGated, kF32>(a, num_sms, partition, stream);
    return launch_lanes<1, 32, kGated, kF32>(a, num_sms, partition, stream);
}

}  // namespace

cudaError_t launch_act_grad(const ActGradArgs& a, int num_sms, bool partition, cudaStream_t stream) {
    if (a.act == EP_ACT_SWIGLU)
        return a.dy_f32 ? launch_width<true, true>(a, num_sms, partition, stream)
                        : launch_width<true, false>(a, num_sms, partition, stream);
    return a.dy_f32 ? launch_width<false, true>(a, num_sms, partition, stream)
                    : launch_width<false, false>(a, num_sms, partition, stream);
}

}  // namespace ep
