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
// Mapping: a CTA to a strip of 64 columns (32 where rows do not start on 8 bytes)
// and every c-th group of rows, a thread to a few columns of a row; a strip's
// rows go to the c CTAs of a cluster. A thread adds its rows, the CTA its threads,
// the cluster its CTAs, each in a fixed order, so that equal calls give equal
// bits.
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

template <int W>
__device__ __forceinline__ void load_row(const void* p, bool f32, int64_t at, float (&v)[W]) {
    if (f32) {
        const float* q = static_cast<const float*>(p) + at;
        if constexpr (W == 1) {
            v[0] = __ldg(q);
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(q + i));
                v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
            }
        }
        return;
    }
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if constexpr (W == 1) {
        v[0] = __uint_as_float(static_cast<uint32_t>(__ldg(q)) << 16);
    } else if constexpr (W == 4) {
        const uint2 f = __ldg(reinterpret_cast<const uint2*>(q));
        const uint32_t w[2] = {f.x, f.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const uint4 f = __ldg(reinterpret_cast<const uint4*>(q));
        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
template <int W>
__device__ __forceinline__ void store_row(uint16_t* q, const float (&v)[W]) {
    if constexpr (W == 1) {
        *q = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
        st_v4(q, round8(v));
    }
}

// W columns to a thread, kLanes threads to a row's part.
template <int W, int kLanes, bool kGated>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const ActGradArgs a) {
    constexpr int kHalves = kGated ? 2 : 1, kRows = kThreads / kLanes, kCols = W * kLanes;
    constexpr int kAtOnce = W == 8 ? 2 : 4;  // rows whose loads are in flight
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
        float dy[kAtOnce][W], g[kAtOnce][W], u[kAtOnce][W];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t r = r0 + j * step;
            if (r >= a.m) break;
            load_row<W>(a.dy, a.dy_f32, r * a.n + col, dy[j]);
            if (a.act != EP_ACT_NONE) load_row<W>(a.z, false, r * wide + col, g[j]);
            if (kGated) load_row<W>(a.z, false, r * wide + a.n + col, u[j]);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t r = r0 + j * step;
            if (r >= a.m) break;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (kGated) {
                    const float du = dy[j][i] * silu(g[j][i]);
                    g[j][i] = dy[j][i] * u[j][i] * silu_slope(g[j][i]);
                    u[j][i] = du;
                    sum[kHalves - 1][i] += du;
                } else {
                    g[j][i] = a.act == EP_ACT_NONE ? dy[j][i] : dy[j][i] * activate_slope(g[j][i], a.act);
                }
                sum[0][i] += g[j][i];
            }
            if (a.dz != nullptr) {
                store_row<W>(a.dz + r * a.pitch + col, g[j]);
                if (kGated) store_row<W>(a.dz + r * a.pitch + a.n + col, u[j]);
            }
        }
    }
    if (a.d_bias == nullptr) return;
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

template <int W, int kLanes, bool kGated>
cudaError_t launch(const ActGradArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int kRows = kThreads / kLanes, kCols = W * kLanes;
    const int64_t strips = (a.n + kCols - 1) / kCols;
    const int64_t groups = a.m > 0 ? (a.m + kRows - 1) / kRows : 1;
    // with sums the grid's rows of CTAs are a cluster; else as many as there is
    // work for
    int64_t parts = 8 * num_sms / strips + 1;
    if (a.d_bias != nullptr) {
        int64_t c = kMaxCluster;
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
    return cudaLaunchKernelEx(&cfg, act_grad_kernel<W, kLanes, kGated>, a);
}

template <bool kGated>
cudaError_t launch_width(const ActGradArgs& a, int num_sms, cudaStream_t stream) {
    if (a.n % 8 == 0) return launch<8, 8, kGated>(a, num_sms, stream);
    if (a.n % 4 == 0) return launch<4, 16, kGated>(a, num_sms, stream);
    return launch<1, 32, kGated>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_act_grad(const ActGradArgs& a, int num_sms, cudaStream_t stream) {
    return a.act == EP_ACT_SWIGLU ? launch_width<true>(a, num_sms, stream)
                                  : launch_width<false>(a, num_sms, stream);
}

}  // namespace ep
