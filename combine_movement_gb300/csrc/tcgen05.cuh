// tcgen05.cuh -- inline-PTX primitives of the fifth-generation tensor cores
// on sm_103a (tensor memory, tcgen05.mma on e4m3 and bf16 operands, 2-D tensor copies),
// next to the bulk-copy primitives of ptx.cuh. Written from the public PTX
// ISA.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "ptx.cuh"

namespace ep {

// ---- tensor memory ----------------------------------------------------------
// Allocation and release are warp-collective; the same warp does both.

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

// Order tcgen05 operations against other threads' through the barriers
// between them.
__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 lanes x 16 columns of fp32 from tensor memory: register i of a lane is
// column i of its row. A warp reads only the 32 rows of its quarter (warp
// index mod 4).
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// Wait for this warp's tensor-memory loads; `v`, a load's registers, pass
// through so that nothing reads them before.
__device__ __forceinline__ void tmem_load_wait16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                   "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                   "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// The same way back, and the wait for it.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---- matrix product ------------------------------------------------------------

// Shared-memory operand descriptor of a K-major tile whose rows are 128 bytes
// (128 e4m3 values), as a tensor copy with 128-byte swizzle leaves it: groups
// of 8 rows, 1024 bytes apart; the tile starts on a 1024-byte boundary. A
// step of 32 bytes along K adds 32 to the address.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem_addr) {
    constexpr uint64_t kLeading = uint64_t{1} << 16;        // unused with a swizzle
    constexpr uint64_t kStride = uint64_t{1024 >> 4} << 32; // between groups of 8 rows
    constexpr uint64_t kVersion = uint64_t{1} << 46;
    constexpr uint64_t kSwizzle128 = uint64_t{2} << 61;
    return kLeading | kStride | kVersion | kSwizzle128 | ((smem_addr & 0x3FFFFu) >> 4);
}

// The same of a tile whose rows run along M (or N): groups of 64 bf16 values
// along it, each 64 rows of 128 bytes along K, 8192 bytes apart; groups of 8
// rows 1024 bytes apart. A step of 16 values along K adds 2048 to the address.
__device__ __forceinline__ uint64_t operand_desc_by_k(uint32_t smem_addr) {
    constexpr uint64_t kLeading = uint64_t{8192 >> 4} << 16;
    constexpr uint64_t kStride = uint64_t{1024 >> 4} << 32;
    constexpr uint64_t kVersion = uint64_t{1} << 46;
    constexpr uint64_t kSwizzle128 = uint64_t{2} << 61;
    return kLeading | kStride | kVersion | kSwizzle128 | ((smem_addr & 0x3FFFFu) >> 4);
}

// Instruction descriptor: fp32 accumulators, both operands e4m3 and K-major.
constexpr uint32_t mma_desc_e4m3(uint32_t m, uint32_t n) {
    return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D[tmem] = A B^T (+ D where `accumulate`), 32 values along K; one thread.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t desc,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// Instruction descriptor: fp32 accumulators, both operands bf16, each K-major or
// (by_k) with its rows along M or N.
constexpr uint32_t mma_desc_bf16(uint32_t m, uint32_t n, bool a_by_k, bool b_by_k) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_by_k ? 1u << 15 : 0u) | (b_by_k ? 1u << 16 : 0u) |
           ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D[tmem] = A B^T (+ D where `accumulate`), 16 values along K; one thread.
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t desc,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// Arrive on `bar` when every tcgen05.mma this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// ---- pairs of CTAs ----------------------------------------------------------------
// The two CTAs of a cluster work on one tile of twice the rows: each holds its
// rows of A, half of B's and its rows' sums; rank 0 issues the products. Tensor
// memory is allocated and released by a warp of each.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t desc,
                                              bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// Arrive on `bar` of both CTAs.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ---- registers ------------------------------------------------------------------
// By all warps of a warpgroup; the kernel's warpgroups together stay within
// the registers it was launched with.
template <int N>
__device__ __forceinline__ void set_max_registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- tensor copies --------------------------------------------------------------

__device__ __forceinline__ void prefetch_tensor_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Box of `map` at (x, y) -> shared memory, completing its bytes on `bar`. x
// times the element size is a multiple of 16; out-of-range elements read 0.
__device__ __forceinline__ void tensor_load_2d(uint32_t dst_smem, const CUtensorMap* map, int32_t x,
                                               int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst_smem),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared memory -> box of `map` at (x, y), both 0 or more, tracked by this thread's
// bulk async-group; what lies out of range is not written.
__device__ __forceinline__ void tensor_store_2d(const CUtensorMap* map, int32_t x, int32_t y,
                                                uint32_t src_smem) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(src_smem)
        : "memory");
}

// The same into this CTA's shared memory, completing on `bar`, a shared::cluster
// address in either CTA of the pair.
__device__ __forceinline__ void tensor_load_2d_pair(uint32_t dst_smem, const CUtensorMap* map,
                                                    int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst_smem),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// ---- small asynchronous copies ------------------------------------------------------
// Four bytes global -> shared by this lane; copy_async_arrive makes one
// (already counted) arrival on `bar` when this lane's copies so far are done.
__device__ __forceinline__ void copy_async4(uint32_t dst_smem, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// An arrival as one predicated instruction, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool arrive) {
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "setp.ne.u32 P, %1, 0;\n\t"
        "@P mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(arrive))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// On a barrier of either CTA of a cluster (a shared::cluster address).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace ep
