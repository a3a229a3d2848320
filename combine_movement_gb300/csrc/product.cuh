// product.cuh -- what the kernels that feed the tensor cores share: shared-memory
// and cluster accesses, waits that give up, rings, and the tensor maps' encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/ep.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace ep {

__device__ __forceinline__ uint32_t load_shared(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float load_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 load_shared_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void store_shared(uint32_t addr, uint32_t v) {
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void store_shared_v4(uint32_t addr, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ float4 load_shared_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 load_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float load_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Cluster barrier, reached by a warp's lanes in their roles' branches. Every
// thread passes it twice, whatever its CTA found to do: the hardware's barrier
// has no limit of its own, the waits before it have.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Wait of a whole warp on a barrier; false, in every lane, once a lane gave up
// after kWaitLimitNs or another warp did (the word at `abort`). The timer is
// slow to read, so the first tries go without. kCluster: arrivals come from other
// CTAs too.
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort,
                                          int32_t* status) {
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xFFFFFFFFu, try_wait<kCluster>(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (__all_sync(0xFFFFFFFFu, try_wait<kCluster>(bar, parity))) return true;
        const bool late = global_timer_ns() - t0 > kWaitLimitNs;
        if (late) {
            store_shared(abort, 1);
            set_status(status, EP_ERR_TIMEOUT);
        }
        if (__any_sync(0xFFFFFFFFu, late || load_shared(abort) != 0)) return false;
    }
}
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort,
                                          int32_t* status) {
    if (__all_sync(0xFFFFFFFFu, try_wait<kCluster>(bar, parity))) return true;
    return wait_slow<kCluster>(bar, parity, abort, status);
}

// Position in a ring of N: index, and the parity of its current round.
template <int N>
struct Ring {
    uint32_t i = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            round ^= 1u;
        }
    }
};

// ---- tensor maps ------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's, looked up once (a failure is not kept).
inline EncodeFn encode_fn() {
    static std::atomic<EncodeFn> known{nullptr};
    EncodeFn fn = known.load(std::memory_order_acquire);
    if (fn != nullptr) return fn;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    fn = reinterpret_cast<EncodeFn>(p);
    known.store(fn, std::memory_order_release);
    return fn;
}

// A map of a matrix of rows of `width` values, `stride` bytes from one to the next, in boxes of
// box_rows x box_width; what lies out of range reads 0 and is not written.
inline bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t rows,
                      int64_t width, int64_t stride, int box_rows, int box_width,
                      CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_width), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    auto encode = [&] {
        return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // The driver wants a current context, and a thread that has made no call of the runtime
    // yet has none: it gets its device's.
    int device = 0;
    return cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess && encode();
}

}  // namespace ep
