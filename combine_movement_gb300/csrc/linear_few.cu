// linear_few.cu -- the dense products (linear.cu) for a token or a few: no tile to
// fill, the time is that of reading the weights once.
//
// Mapping: eight weight rows (gated: four of each half) to a CTA, whose threads
// go along k, or for short rows to each of its warps; a thread reads 16 bytes of
// each weight row and of each of x's rows at a time and keeps their products' sums
// in fp32. Sums are joined over the lanes, then over the warps in order.
//
// Bound by memory once it runs: one row of 7168 x 2 x 2048, gated, 10.5 us (58.7 MB, 5.6
// TB/s), of which 2 are the start and the first loads' latency; all 512 CTAs are
// resident at once (with more registers to a thread, 456, it took 15.3).
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "linear_out.cuh"
#include "ptx.cuh"

namespace ep {
namespace {

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWeightRows = 8;

// Sums of N values over the warp's lanes: lane l is left with that of value
// index(l) = l's highest bits.
template <int N, int kStep>
__device__ __forceinline__ float sum_lanes(const float (&v)[N], int lane) {
    if constexpr (N == 1) {
        float s = v[0];
#pragma unroll
        for (int d = kStep; d > 0; d >>= 1) s += __shfl_xor_sync(kFullMask, s, d);
        return s;
    } else {
        const bool high = (lane & kStep) != 0;
        float half[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = high ? v[i + N / 2] : v[i], give = high ? v[i] : v[i + N / 2];
            half[i] = keep + __shfl_xor_sync(kFullMask, give, kStep);
        }
        return sum_lanes<N / 2, kStep / 2>(half, lane);
    }
}

// kRows of x; kLong: a CTA's warps share its weight rows.
template <int kRows, bool kGated, bool kLong>
__global__ void __launch_bounds__(kThreads, kRows == 1 ? 4 : kRows == 2 ? 3 : 2)
    few_kernel(const LinearArgs a) {
    constexpr int kSums = kRows * kWeightRows, kLanesEach = 32 / kSums;
    constexpr int kCols = kGated ? kWeightRows / 2 : kWeightRows;
    __shared__ float part[kWarps][kSums];  // [weight row][row of x]
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t group = kLong ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t col0 = group * kCols;
    // (rows past the last are computed along with it)
    const uint16_t* w[kWeightRows];
#pragma unroll
    for (int i = 0; i < kWeightRows; ++i) {
        const int64_t c = min(col0 + i % kCols, a.n - 1);
        w[i] = a.b + (c + (i >= kCols ? a.n : 0)) * a.b_pitch;
    }
    const uint16_t* x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) x[i] = a.a + min(static_cast<int64_t>(i), a.m - 1) * a.a_pitch;
    float acc[kSums] = {};
    constexpr int kStep = kLong ? kThreads * 8 : 32 * 8;
#pragma unroll 1
    for (int64_t k = (kLong ? threadIdx.x : lane) * 8; k < a.k; k += kStep) {
        uint4 wv[kWeightRows];
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i) wv[i] = ld_nc_v4(w[i] + k);
        float xf[kRows][8];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(x[i] + k));
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[i][2 * j] = bf16_low(q[j]), xf[i][2 * j + 1] = bf16_high(q[j]);
        }
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i) {
            const uint32_t q[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float& s = acc[i * kRows + r];
                    s = fmaf(bf16_low(q[j]), xf[r][2 * j], s);
                    s = fmaf(bf16_high(q[j]), xf[r][2 * j + 1], s);
                }
        }
    }
    const float mine = sum_lanes<kSums, 16>(acc, lane);
    if (lane % kLanesEach == 0) part[warp][lane / kLanesEach] = mine;
    if (kLong)
        __syncthreads();
    else
        __syncwarp();
    const int i = kLong ? threadIdx.x : lane;
    if (i >= kCols * kRows) return;
    const int c = i % kCols, r = i / kCols;
    const int64_t col = col0 + c;
    if (r >= a.m || col >= a.n) return;
    Values<1> v[1] = {}, up[1] = {};
    Residual<1> res[1] = {};
    if (a.residual != nullptr) res[0] = load_residual<1>(a, r * a.n + col);
    if (kLong) {
#pragma unroll
        for (int p = 0; p < kWarps; ++p) {
            v[0].v[0] += part[p][c * kRows + r];
            if (kGated) up[0].v[0] += part[p][(c + kCols) * kRows + r];
        }
    } else {
        v[0].v[0] = part[warp][c * kRows + r];
        if (kGated) up[0].v[0] = part[warp][(c + kCols) * kRows + r];
    }
    v[0] = v[0] + load_bias<1>(a.bias, col);
    if (kGated) up[0] = up[0] + load_bias<1>(a.bias, a.n + col);
    finish<1, kGated>(a, r, col, 0, 1, v, up, res);
}

template <int kRows, bool kGated>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
    constexpr int kCols = kGated ? kWeightRows / 2 : kWeightRows;
    const int64_t groups = (a.n + kCols - 1) / kCols;
    if (a.k >= 1024)
        return launch_dependent(few_kernel<kRows, kGated, true>, static_cast<int>(groups), kThreads, 0,
                                stream, a);
    return launch_dependent(few_kernel<kRows, kGated, false>,
                            static_cast<int>((groups + kWarps - 1) / kWarps), kThreads, 0, stream, a);
}

template <bool kGated>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t stream) {
    if (a.m == 1) return launch<1, kGated>(a, stream);
    if (a.m == 2) return launch<2, kGated>(a, stream);
    return launch<4, kGated>(a, stream);
}

}  // namespace

// One row always; two where the weights are at most 32 MB, up to four where they are at most
// 16: the more rows the fewer loads its registers leave in flight (7168 x 2048: 2 rows 7.6 us
// here, 8.8 in tiles, 4 rows 9.7 and 8.9; gated 2 x 2048 x 2048: 2 rows 5.8 and 7.0, 4 rows 6.7
// and 7.0; of 58.7 MB, gated, 1 row 10.5 and 13.3, 2 rows 15.4 and 13.3; 4 x 1000 x 1000
// 4.3 and 4.4).
bool linear_few_takes(const LinearArgs& a) {
    if (a.a_by_k || a.b_by_k || a.m > 4) return false;
    const int64_t rows = a.act == EP_ACT_SWIGLU ? 2 * a.n : a.n;
    return a.m == 1 || rows * a.k <= (int64_t{a.m == 2 ? 16 : 8} << 20);
}

cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t stream) {
    return a.act == EP_ACT_SWIGLU ? launch_rows<true>(a, stream) : launch_rows<false>(a, stream);
}

}  // namespace ep
