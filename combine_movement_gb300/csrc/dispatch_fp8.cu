// dispatch_fp8.cu -- dispatch that quantises on the way: every token row goes
// to the receive rows of its K experts as e4m3 with one fp32 scale for each
// block of 128 values (fp8_math.cuh), half the bytes of a bf16 dispatch.
//
// A row is read and quantised once and written K times. A unit is 512 or 1024
// columns of one token: a lane takes 16 columns (two 16-byte loads), eight
// lanes a block, whose maximum goes round by three shuffles; each lane then
// stores its 16 bytes to each of the K receive rows, 512 contiguous bytes a
// warp.
//
// On the whole GPU a unit goes to a warp of a small CTA, and the SMs that
// finish first take the next CTAs; on a smaller SM budget (one CTA per SM of
// it) the units are split evenly over the warps of the budget.
//
// Bound by the writes: T = 4096, H = 7168, top-8 moves 301 MB (a fifth of it reads) in
// 46.6 us, 6.5 TB/s, 0.95 of a plain copy's rate; with one CTA per SM it took
// 54 us (some SMs write a quarter slower than others), with two or four units
// to a warp 50 and 53 us. T = 128: about the launch, 6 us.
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "fp8_math.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "work_split.cuh"

namespace ep {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kThreads = 1024;
constexpr int kSmallThreads = 256;
constexpr int kLaneCols = 16;
constexpr int kWarpCols = 32 * kLaneCols;
constexpr int64_t kMaxGrid = 0x7FFFFFFF;
constexpr int kBlockLanes = kFp8Block / kLaneCols;

// The two bf16 values of a word, widened exactly.
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// kParts: 512-column parts of a unit.
template <int kParts>
__global__ void __launch_bounds__(kThreads, 1) dispatch_fp8_kernel(const DispatchFp8Args a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kUnitCols = kParts * kWarpCols;
    const int64_t n_units = (a.H + kUnitCols - 1) / kUnitCols;  // of a row
    const int64_t units = a.T * n_units;
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
    const int64_t nw = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const int64_t u0 = split_begin(units, gw, nw), u1 = split_begin(units, gw + 1, nw);
    int64_t t = div_floor(u0, n_units);
    int64_t part = u0 - t * n_units;
    int64_t tok = -1;
    int32_t slot = -1;  // lane k's
    for (int64_t u = u0; u < u1; ++u) {
        uint4 v[kParts][2];
        bool in[kParts];
        const int64_t col0 = part * kUnitCols + lane * kLaneCols;
        const uint16_t* src = a.x + t * a.H + col0;
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            in[j] = col0 + j * kWarpCols < a.H;  // H is a multiple of 16
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[j][i] = in[j] ? ld_nc_v4(src + j * kWarpCols + i * 8) : make_uint4(0, 0, 0, 0);
        }
        if (t != tok) {
            tok = t;
            slot = lane < a.K ? __ldg(a.slot + t * a.K + lane) : -1;
            if (slot >= a.num_recv) {
                set_status(a.status, EP_ERR_BAD_SLOT);
                slot = -1;
            }
        }
        if (part == 0 && slot >= 0) {
            if (a.recv_w != nullptr) a.recv_w[slot] = __ldg(a.topk_w + t * a.K + lane);
            if (a.recv_src != nullptr) a.recv_src[slot] = static_cast<int32_t>(t * a.K + lane);
        }
        uint4 q[kParts];
        float scale[kParts];
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            const uint32_t w[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w,
                                   v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, max(abs_bits(lo(w[i])), abs_bits(hi(w[i]))));
#pragma unroll
            for (int d = 1; d < kBlockLanes; d <<= 1) top = max(top, __shfl_xor_sync(kFullMask, top, d));
            const BlockScale bs = block_scale(top);
            scale[j] = bs.scale;
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = pack_e4m3x4(lo(w[2 * i]) * bs.inverse, hi(w[2 * i]) * bs.inverse,
                                   lo(w[2 * i + 1]) * bs.inverse, hi(w[2 * i + 1]) * bs.inverse);
            q[j] = make_uint4(p[0], p[1], p[2], p[3]);
        }
        for (int k = 0; k < a.K; ++k) {
            const int64_t row = __shfl_sync(kFullMask, slot, k);
            if (row < 0) continue;
#pragma unroll
            for (int j = 0; j < kParts; ++j) {
                if (!in[j]) continue;
                const int64_t col = col0 + j * kWarpCols;
                st_v4(a.recv_q + row * a.H + col, q[j]);
                if (lane % kBlockLanes == 0)
                    a.recv_scale[row * a.blocks + col / kFp8Block] = scale[j];
            }
        }
        if (++part == n_units) {
            part = 0;
            ++t;
        }
    }
}

template <int kParts>
cudaError_t launch_parts(const DispatchFp8Args& a, int num_sms, cudaStream_t stream) {
    const int64_t units = a.T * ((a.H + kParts * kWarpCols - 1) / (kParts * kWarpCols));
    auto kern = dispatch_fp8_kernel<kParts>;
    if (a.whole_gpu) {  // a unit to a warp
        constexpr int64_t kPer = kSmallThreads / 32;
        if (units <= kMaxGrid * kPer)
            return launch_dependent(kern, static_cast<int>((units + kPer - 1) / kPer), kSmallThreads,
                                    0, stream, a);
    }
    const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kExclusiveSmem));
    if (err != cudaSuccess) return err;
    return launch_dependent(kern, static_cast<int>(ctas < num_sms ? ctas : num_sms), kThreads,
                            kExclusiveSmem, stream, a);
}

}  // namespace

cudaError_t launch_dispatch_fp8(const DispatchFp8Args& a, int num_sms, cudaStream_t stream) {
    // wide units (more loads in flight) where every warp still gets two of them
    const int64_t wide = a.T * ((a.H + 2 * kWarpCols - 1) / (2 * kWarpCols));
    if (wide >= 2ll * num_sms * (kThreads / 32)) return launch_parts<2>(a, num_sms, stream);
    return launch_parts<1>(a, num_sms, stream);
}

}  // namespace ep
