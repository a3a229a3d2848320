// clear_rows.cu -- zeros in the rows of a receive buffer that no (token, k)
// entry maps to (masked entries leave them), so that they can take part in
// what is computed from the whole buffer: the experts' weight gradients, where
// a zero gradient meets whatever the row holds.
//
// Which rows those are only the slots say. Row r belongs to CTA r mod G (G a
// power of two); a CTA reads all slots, marks its own used rows in a bit map in
// shared memory and then clears the others, a row to a warp. So nothing is
// kept between launches and no workspace is needed, at the cost of reading the
// slots G times, from L2.
//
// Bound by that reading where few rows are cleared: T = 4096, top-8, H = 7168
// takes 7.5-8 us with no entry masked, 14-15 with a tenth, 43-46 with half (235
// MB, 5.3 TB/s); clearing the whole buffer instead took 116 us. T = 128: 2.7 us.
// Many short rows: 131072 x 8 of H = 512 183-260 us (the whole buffer 264).
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "routing.cuh"

namespace ep {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kLoads = 8;  // slots of a thread in flight
constexpr int64_t kMapBits = static_cast<int64_t>(kExclusiveSmem) * 8;  // rows of a CTA at a time

__global__ void __launch_bounds__(kThreads, 1) clear_rows_kernel(const ClearRowsArgs a) {
    extern __shared__ uint32_t used[];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t cta = static_cast<int32_t>(blockIdx.x), mask = (1 << a.log_ctas) - 1;
    // this CTA's rows: cta + i * G, i < own
    const int64_t own = (a.num_recv - cta + mask) >> a.log_ctas;
    for (int64_t i0 = 0; i0 < own; i0 += kMapBits) {
        const int count = static_cast<int>(min(own - i0, kMapBits));
        for (int i = threadIdx.x; i < (count + 31) / 32; i += kThreads) used[i] = 0;
        __syncthreads();
        for (int64_t e0 = threadIdx.x; e0 < a.entries; e0 += kLoads * kThreads) {
            int32_t s[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int64_t e = e0 + j * kThreads;
                s[j] = e < a.entries ? __ldg(a.slot + e) : -1;
            }
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                if (s[j] >= a.num_recv) set_status(a.status, EP_ERR_BAD_SLOT);
                // (a slot past the rows has an i of at least count)
                const int64_t i = (s[j] >> a.log_ctas) - i0;
                if (s[j] >= 0 && (s[j] & mask) == cta && i >= 0 && i < count)
                    atomicOr(used + (i >> 5), 1u << (i & 31));
            }
        }
        __syncthreads();
        for (int i = warp; i < count; i += kWarps) {
            if ((used[i >> 5] >> (i & 31)) & 1u) continue;
            uint16_t* row = a.rows + (((i0 + i) << a.log_ctas) + cta) * a.H;
            for (int64_t c = lane * 8; c < a.H; c += 32 * 8) st_v4(row + c, make_uint4(0, 0, 0, 0));
        }
        __syncthreads();  // the map is read until here
    }
}

}  // namespace

cudaError_t launch_clear_rows(ClearRowsArgs a, int num_sms, cudaStream_t stream) {
    // as many CTAs as leave every warp a row, at most one to an SM
    a.log_ctas = 0;
    while ((2 << a.log_ctas) <= num_sms && (static_cast<int64_t>(kWarps) << a.log_ctas) < a.num_recv)
        ++a.log_ctas;
    const cudaError_t err = cudaFuncSetAttribute(
        clear_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kExclusiveSmem));
    if (err != cudaSuccess) return err;
    return launch_dependent(clear_rows_kernel, 1 << a.log_ctas, kThreads, kExclusiveSmem, stream, a);
}

}  // namespace ep
