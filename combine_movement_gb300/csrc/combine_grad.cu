// combine_grad.cu -- the gradient of combine. With y[t] = sum over k of
// w[t,k] * e[slot[t,k]] and the gradient dy of y:
//
//   d_e[slot[t,k], :] = bf16_rne( w[t,k] * dy[t, :] )
//   d_w[t,k]          = sum over h of dy[t,h] * e[slot[t,k], h]     (fp32)
//
// (a masked entry has d_w = 0). No two entries share a receive row, so nothing
// is accumulated across warps and the result does not depend on their order.
//
// Mapping: one (t, k) entry to a group of warps (one, or for few entries up
// to eight, which split the row and add their parts of d_w in a fixed order).
// A lane reads 16 bytes of dy and of the expert row, writes 16 bytes of d_e
// and keeps eight fp32 partial sums. Entries of one token go to neighbouring
// warps of a CTA, so that dy comes from L1 for all but the first of them. On
// the whole GPU an entry goes to a group of a small CTA, and the SMs that
// finish first take the next CTAs; on a smaller SM budget (one CTA per SM of
// it) the entries go round the groups of the budget.
//
// Bound by memory: T = 4096, H = 7168, top-8 reads 470 MB of expert rows, writes as
// many and reads 59 MB of dy in 151.4 us, 6.6 TB/s, 0.97 of a plain copy's
// rate (with one CTA per SM 163 us; two entries to a warp 156 us). T = 128,
// H = 1024, top-2: about the launch, 6.5 us.
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace ep {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kSmallThreads = 256;
constexpr int64_t kMaxGrid = 0x7FFFFFFF;
constexpr int kUnroll = 4;            // 16-byte loads of each row in flight per lane
constexpr int kWarpCols = 32 * 8;

// kSplit warps to an entry.
template <int kSplit>
__global__ void __launch_bounds__(kThreads, 1) combine_grad_kernel(const CombineGradArgs a) {
    __shared__ float parts[2][kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kGroups = (blockDim.x >> 5) / kSplit;
    const int group = warp / kSplit, member = warp % kSplit;
    const int64_t entries = a.T * a.K;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kGroups;
    int round = 0;
    for (int64_t e0 = first; e0 < entries; e0 += stride, round ^= 1) {
        const int64_t e = e0 + group;
        const bool valid = e < entries;
        float sum = 0.0f;
        int32_t slot = valid ? __ldg(a.slot + e) : -1;
        if (slot >= a.num_recv) {
            set_status(a.status, EP_ERR_BAD_SLOT);
            slot = -1;
        }
        if (slot >= 0) {
            const float w = __ldg(a.topk_w + e);
            const int64_t t = e / a.K;
            const uint16_t* dy = a.dy + t * a.H;
            const uint16_t* row = a.expert_out + static_cast<int64_t>(slot) * a.H;
            uint16_t* out = a.d_expert_out + static_cast<int64_t>(slot) * a.H;
            float acc[8] = {};
            for (int64_t c0 = member * kWarpCols + lane * 8; c0 < a.H;
                 c0 += kUnroll * kSplit * kWarpCols) {
                uint4 g[kUnroll], v[kUnroll];
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    const int64_t c = c0 + j * kSplit * kWarpCols;
                    if (c < a.H) {
                        v[j] = a.d_topk_w != nullptr ? ld_nc_v4(row + c) : make_uint4(0, 0, 0, 0);
                        g[j] = __ldg(reinterpret_cast<const uint4*>(dy + c));
                    }
                }
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    const int64_t c = c0 + j * kSplit * kWarpCols;
                    if (c >= a.H) continue;
                    const uint32_t gw[4] = {g[j].x, g[j].y, g[j].z, g[j].w};
                    const uint32_t vw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                    float d[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float g0 = __uint_as_float(gw[i] << 16);
                        const float g1 = __uint_as_float(gw[i] & 0xFFFF0000u);
                        acc[2 * i] = fmaf(g0, __uint_as_float(vw[i] << 16), acc[2 * i]);
                        acc[2 * i + 1] =
                            fmaf(g1, __uint_as_float(vw[i] & 0xFFFF0000u), acc[2 * i + 1]);
                        d[2 * i] = w * g0;
                        d[2 * i + 1] = w * g1;
                    }
                    if (a.d_expert_out != nullptr) st_v4(out + c, round8(d));
                }
            }
            sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
        if (kSplit > 1) {
            // the other buffer is read until the next round's barrier
            if (lane == 0) parts[round][warp] = sum;
            __syncthreads();
            if (member == 0) {
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kSplit; ++i) sum += parts[round][warp + i];
            }
        }
        if (valid && member == 0 && lane == 0 && a.d_topk_w != nullptr) a.d_topk_w[e] = sum;
    }
}

template <int kSplit>
cudaError_t launch_split(const CombineGradArgs& a, int num_sms, cudaStream_t stream) {
    auto kern = combine_grad_kernel<kSplit>;
    if (a.whole_gpu) {  // an entry to a group of warps
        constexpr int64_t kPer = kSmallThreads / 32 / kSplit;
        if (a.T * a.K <= kMaxGrid * kPer)
            return launch_dependent(kern, static_cast<int>((a.T * a.K + kPer - 1) / kPer),
                                    kSmallThreads, 0, stream, a);
    }
    constexpr int kGroups = kWarps / kSplit;
    const int64_t ctas = (a.T * a.K + kGroups - 1) / kGroups;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kExclusiveSmem));
    if (err != cudaSuccess) return err;
    return launch_dependent(kern, static_cast<int>(ctas < num_sms ? ctas : num_sms), kThreads,
                            kExclusiveSmem, stream, a);
}

}  // namespace

cudaError_t launch_combine_grad(const CombineGradArgs& a, int num_sms, int budget,
                                cudaStream_t stream) {
    // as many warps to an entry as leave every warp an entry's part, and every
    // warp of it a full round of loads. (By the budget, not by a partition's
    // SMs: the split sets the order of d_w's sum, which the stream must not.
    // In a partition of 24 SMs that takes 13.8 us instead of 14.3 for 200 entries
    // of H = 16384, 16.2 instead of 14.6 for 1000 of 4096, 18.7 instead of 15.3 for
    // 2400 of 2048.)
    const int64_t warps = static_cast<int64_t>(budget) * kWarps, entries = a.T * a.K;
    const int64_t rounds = (a.H + kUnroll * kWarpCols - 1) / (kUnroll * kWarpCols);
    if (entries * 8 <= warps && rounds >= 8) return launch_split<8>(a, num_sms, stream);
    if (entries * 4 <= warps && rounds >= 4) return launch_split<4>(a, num_sms, stream);
    if (entries * 2 <= warps && rounds >= 2) return launch_split<2>(a, num_sms, stream);
    return launch_split<1>(a, num_sms, stream);
}

}  // namespace ep
