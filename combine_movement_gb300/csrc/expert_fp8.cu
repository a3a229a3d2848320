// expert_fp8.cu -- the experts' products on received rows, in e4m3 with one
// fp32 scale for each block of 128 (rows: 1 x 128, weights: 128 x 128):
//
//   y[r, n] = sum_b a_scale[r, b] * w_scale[e, n / 128, b]
//                   * sum_{k in block b} a[r, k] * w[e, n, k]
//
// for the rows r of expert e (offsets[e] <= r < offsets[e + 1]); either y in
// bf16, or, for a first product whose columns are a gate half and an up half,
// h = silu(y[r, i]) * y[r, I + i] quantised in blocks of 128 columns again.
//
// Mapping: a persistent grid, one CTA per SM. A tile is 128 rows of one expert
// times two blocks of 128 weight rows (neighbours; for the gated form block j
// of the gate half and block j of the up half, so that the tile holds a whole
// quantisation block of h). Per 128 values along K one of four stages of
// shared memory takes the operands (tensor copies, 128-byte swizzle), and four
// tcgen05.mma of 128 x 256 x 32 leave the block's plain sums in one of two
// places in tensor memory. The scales differ between rows and between blocks
// along K, so they cannot ride in the tensor core's sum: four warpgroups read
// the sums back and add them, scaled, into fp32 registers (a thread holds 32
// columns of both weight blocks of one row), while the tensor cores work on
// the next block. One warp issues the tensor copies, one the products, one the
// scales' copies (four bytes each, asynchronous, up to sixteen blocks ahead).
//
// What bounds it: few rows to an expert, the weights' bytes (256 experts x
// 7168 x 2048 for 1024 rows: 520-537 us, 7 TB/s; one row each for eight experts
// of 4096 x 7168: 41-43 us, 5.6 TB/s). Many rows, the adding: a block's products
// take the tensor cores 512 cycles, a block's adding about 800, mostly
// latencies (a barrier that is ready takes 70-150 cycles to ask, a load from
// tensor memory 50-70) with 384 of them in the fma pipe (131072 rows x 7168 x
// 4096 on 128 experts: 3.0-3.1 ms, 2.5 PFLOP/s; run for seconds, the board's
// power limit brings it to 3.5 ms). Measured on the way:
//  - eight adding warps with 64 columns of each block: 18 % slower;
//  - a branch around the adding for rows a tile lacks: 25 % slower at 128 rows
//    an expert;
//  - a product of 128 x 128 for each half of the columns, which two warpgroups
//    add: 1.5-3 % slower (the products then read their rows twice, all of
//    shared memory's bandwidth);
//  - pairs of CTAs on tiles of 256 rows (cta_group::2: two thirds of the bytes
//    from L2): 4-5 % faster at 1000 rows an expert, 18-33 % slower at 128 and
//    fewer.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "fp8_math.cuh"
#include "kernels.cuh"
#include "per_device.cuh"
#include "routing.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTileRows = 128;
constexpr int kTileK = 128;                    // bytes and values of one stage row
constexpr int kTileCols = 2 * kFp8Block;       // weight rows of a tile
constexpr uint32_t kStageA = kTileRows * kTileK;
constexpr uint32_t kStageB = kFp8Block * kTileK;  // one of the tile's two weight blocks
constexpr uint32_t kStageBytes = kStageA + 2 * kStageB;
constexpr int kStages = 4;
constexpr int kSlots = 2;                      // of a block's sums in tensor memory
constexpr int kAccWarps = 16;
constexpr int kAccGroups = kAccWarps / 4;      // warpgroups
constexpr int kAccCols = kFp8Block / kAccGroups;  // of each weight block, in one thread
constexpr int kProductWarp = kAccWarps, kCopyWarp = kAccWarps + 1, kScaleWarp = kAccWarps + 2;
constexpr int kThreads = (kAccWarps + 4) * 32;  // the last warp idles
// Registers per thread: the launch's 96 (640 threads) move from the last
// warpgroup to the four that hold the sums: 512 x 104 + 128 x 64 = 640 x 96.
constexpr int kAccRegs = 104, kOtherRegs = 64, kLaunchRegs = 96;
static_assert(kAccWarps * 32 * kAccRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
              "register split");
constexpr uint32_t kTmemCols = kSlots * kTileCols;
constexpr int kRowBoxes = 4;                   // row boxes of 16, 32, 64, 128

// Scales: of the CTA's 128 rows and of the two weight blocks, for kScaleGroup
// blocks along K at a time (a tile's last group may have fewer), in a ring of
// their own between the scale warp and the adding warps.
constexpr int kScaleGroup = 4;
constexpr int kScaleGroups = 4;
// With a tile's first group goes what the adding warps need to know of the
// tile when they write it. The scale warp is at most kScaleGroups groups, and
// so tiles, ahead of the last adding warp.
constexpr int kTileNotes = 2 * kScaleGroups;
struct TileNote {
    int row0, rows, col_tile;
};

// A tile shared by a cluster: its fp32 sums, [row][column], in the stages' place;
// a row's pitch keeps both ways through them free of bank conflicts.
constexpr uint32_t kSharedPitch = kTileCols * 4 + 16;
static_assert(kTileRows * kSharedPitch <= kStages * kStageBytes, "shared sums");
constexpr int kMaxSplit = 8;

struct Maps {
    CUtensorMap rows[kRowBoxes];
    CUtensorMap weights;
};

struct Control {
    uint64_t full[kStages];       // the copies have landed
    uint64_t done[kStages];       // the stage's product is done: stage free, sums there
    uint64_t scales[kScaleGroups];       // a group has landed: the scale warp's lanes, and its note
    uint64_t scales_read[kScaleGroups];  // and has been read: the adding warps
    alignas(16) uint64_t sums_read[kSlots];
    uint64_t joined;       // accumulating warps, once per tile
    uint64_t drained;      // after an abort: products still in flight
    uint32_t tmem;
    int32_t abort;
    TileNote notes[kTileNotes];
    uint32_t amax[2][kAccGroups][kTileRows];
    float row_scale[kScaleGroups][kScaleGroup][kTileRows];
    alignas(8) float weight_scale[kScaleGroups][kScaleGroup][2];
};

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
// slow to read, so the first tries go without.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort,
                                          int32_t* status) {
    for (int i = 0; i < 256; ++i)
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        const bool late = global_timer_ns() - t0 > kWaitLimitNs;
        if (late) {
            store_shared(abort, 1);
            set_status(status, EP_ERR_TIMEOUT);
        }
        if (__any_sync(0xFFFFFFFFu, late || load_shared(abort) != 0)) return false;
    }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort,
                                          int32_t* status) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    return wait_slow(bar, parity, abort, status);
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

// One tile: up to 128 rows of an expert times two blocks of its weight rows.
struct Tile {
    int expert;
    int col_tile;
    int row0;   // first row
    int rows;   // 1 .. 128
};

__device__ __forceinline__ uint32_t row_tiles_of(int rows) {
    return (static_cast<uint32_t>(rows) + kTileRows - 1) / kTileRows;
}

// The tiles of expert e are cum[e] .. cum[e + 1], row tiles innermost: tiles
// that read the same weights run at the same time.
__device__ __forceinline__ Tile find_tile(int t, const int32_t* cum, const ExpertArgs& a) {
    int lo = 0, hi = a.E;  // cum[lo] <= t < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int begin = __ldg(a.offsets + lo), end = __ldg(a.offsets + lo + 1);
    const uint32_t local = t - cum[lo], row_tiles = row_tiles_of(end - begin);
    Tile tile;
    tile.expert = lo;
    tile.col_tile = static_cast<int>(local / row_tiles);
    const int rt = static_cast<int>(local - tile.col_tile * row_tiles);
    tile.row0 = begin + rt * kTileRows;
    tile.rows = min(kTileRows, end - tile.row0);
    return tile;
}

// Rows of expert e, or 0 where the offsets are not a valid split of the
// num_recv rows (reported as EP_ERR_BAD_SLOT).
__device__ __forceinline__ int expert_rows(int e, const ExpertArgs& a) {
    const int begin = __ldg(a.offsets + e), end = __ldg(a.offsets + e + 1);
    if (begin < 0 || end < begin || end > a.num_recv) {
        set_status(a.status, EP_ERR_BAD_SLOT);
        return 0;
    }
    return end - begin;
}

// acc[i0 ..] += s * v for 16 columns, two to an instruction, each rounded as by
// fmaf. (A pair takes three cycles of the fma pipe, two single fmas two; but it
// takes one issue slot instead of two, and the four warps of a scheduler come
// to more issue slots than the block's products leave them: 5 % faster.)
__device__ __forceinline__ void add_scaled(float (&acc)[kAccCols], int i0, const uint32_t (&v)[16],
                                           float s) {
    uint64_t s2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        uint64_t d, sum;
        asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(v[i]), "r"(v[i + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(sum) : "f"(acc[i0 + i]), "f"(acc[i0 + i + 1]));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(d), "l"(s2));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i0 + i]), "=f"(acc[i0 + i + 1]) : "l"(sum));
    }
}

// 1 / v for v in [1, 2], within one unit.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// p[i] of lane j <-> p[j] of lane i, i and j within each four lanes; `j` is
// lane mod 4.
__device__ __forceinline__ void transpose4(uint4 (&p)[4], int j) {
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        // exchange the halves that differ in bit d of both i and j
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            uint4& low = p[i];
            uint4& high = p[i + d];
            const bool up = (j & d) != 0;
            uint4 give = up ? low : high;
            give.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, d);
            give.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, d);
            give.z = __shfl_xor_sync(0xFFFFFFFFu, give.z, d);
            give.w = __shfl_xor_sync(0xFFFFFFFFu, give.w, d);
            if (up)
                low = give;
            else
                high = give;
        }
    }
}

// The kParts CTAs' sums of the rows r = rank mod kParts, joined into this
// CTA's; always eight 16-byte loads of a thread in flight.
template <int kParts>
__device__ __forceinline__ void sum_parts(uint32_t sums, int rows, int rank) {
    constexpr int kPieces = kTileCols / 4, kAtOnce = 8 / kParts, kStep = kAccWarps * 32;
    const int pieces = (rows + kParts - 1 - rank) / kParts * kPieces;  // (0 of 0 rows)
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < pieces; i0 += kAtOnce * kStep) {
        uint32_t addr[kAtOnce];
        float4 v[kAtOnce][kParts];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = i0 + j * kStep;
            addr[j] = sums + (i / kPieces * kParts + rank) * kSharedPitch + i % kPieces * 16;
            if (i >= pieces) continue;
#pragma unroll
            for (int p = 0; p < kParts; ++p) v[j][p] = load_cluster_v4(cluster_map(addr[j], p));
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (i0 + j * kStep >= pieces) continue;
            float4 sum = v[j][0];
#pragma unroll
            for (int p = 1; p < kParts; ++p) {
                sum.x += v[j][p].x;
                sum.y += v[j][p].y;
                sum.z += v[j][p].z;
                sum.w += v[j][p].w;
            }
            store_shared_v4(addr[j], sum);  // (only this CTA reads these rows of its own)
        }
    }
}

// The sums of a tile that the cluster's CTAs took parts of K of: each CTA
// lays its own out in shared memory, and CTA p joins those of the rows
// r = p mod split, in the order of the parts, so that a row's result does not
// depend on its place. `row` is the thread's, `at` where its columns start in
// a row; `rows` 0 after a wait that gave up.
__device__ __forceinline__ void join_parts(float (&acc)[2][kAccCols], uint32_t sums, int rows, int row,
                                           uint32_t at, int rank, int split) {
    const uint32_t own = sums + row * kSharedPitch + at;
    if (row < rows) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < kAccCols; i += 4)
                store_shared_v4(own + b * kFp8Block * 4 + i * 4,
                                make_float4(acc[b][i], acc[b][i + 1], acc[b][i + 2], acc[b][i + 3]));
    }
    cluster_arrive();
    cluster_wait();
    if (split == 2)
        sum_parts<2>(sums, rows, rank);
    else if (split == 4)
        sum_parts<4>(sums, rows, rank);
    else
        sum_parts<8>(sums, rows, rank);
    cluster_arrive();  // the other CTAs' sums have been read; waited for at the end
    asm volatile("bar.sync 1, %0;" ::"n"(kAccWarps * 32) : "memory");
    // (other rows' threads read something that is not stored)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < kAccCols; i += 4) {
            const float4 v = load_shared_v4(own + b * kFp8Block * 4 + i * 4);
            acc[b][i] = v.x;
            acc[b][i + 1] = v.y;
            acc[b][i + 2] = v.z;
            acc[b][i + 3] = v.w;
        }
}

// A CTA's first tile and the step to its next; a cluster has one tile, t0. The
// grid's registers are read where they are used: the adding warps have none to
// keep them in (kept, they cost the large products 1 % cool, 4 % at the power
// limit).
template <bool kSplit>
__device__ __forceinline__ int first_tile(int t0) {
    return kSplit ? t0 : static_cast<int>(blockIdx.x);
}
template <bool kSplit>
__device__ __forceinline__ int tile_step(int tiles) {
    return kSplit ? tiles : static_cast<int>(gridDim.x);
}

// kSplit: a tile's blocks along K go to the CTAs of a cluster, a tile to a
// cluster; else a CTA takes whole tiles, one after the other.
template <bool kGateUp, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const ExpertArgs a, const __grid_constant__ Maps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;
    // stages on a 1024-byte boundary (the swizzle's period), then cum[E + 1]
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int32_t* cum = reinterpret_cast<int32_t*>(smem_raw + (base - smem_u32(smem_raw)) +
                                              kStages * kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(ctl.full), done = smem_u32(ctl.done);
    const uint32_t sums_read = smem_u32(ctl.sums_read);
    const uint32_t scales = smem_u32(ctl.scales), scales_read = smem_u32(ctl.scales_read);
    const uint32_t joined = smem_u32(&ctl.joined);
    const uint32_t abort = smem_u32(&ctl.abort);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < kScaleGroups; ++i) {
            mbar_init(scales + 8 * i, 32 + 1);
            mbar_init(scales_read + 8 * i, kAccWarps);
        }
        for (int i = 0; i < kSlots; ++i) mbar_init(sums_read + 8 * i, kAccWarps);
        mbar_init(joined, kAccWarps);
        mbar_init(smem_u32(&ctl.drained), 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == kProductWarp) tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
    if (warp == kCopyWarp && lane == 0) {
        for (int i = 0; i < a.row_boxes; ++i) prefetch_tensor_map(&maps.rows[i]);
        prefetch_tensor_map(&maps.weights);
    }
    griddep_wait();
    griddep_launch_dependents();

    // cum[e] = tiles of the experts before e. (The host lets kMaxTiles through
    // at most for offsets that ascend; others may claim rows twice and come to
    // more, which is refused here.)
    {
        const int per = (a.E + kThreads - 1) / kThreads;
        const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
        int64_t mine = 0, total = 0;
        for (int e = e0; e < e1; ++e)
            mine += static_cast<int64_t>(row_tiles_of(expert_rows(e, a))) * a.col_tiles;
        int64_t run = block_exclusive_scan(mine, &total);
        for (int e = e0; e < e1; ++e) {
            cum[e] = static_cast<int32_t>(min(run, static_cast<int64_t>(kMaxTiles)));
            run += static_cast<int64_t>(row_tiles_of(expert_rows(e, a))) * a.col_tiles;
        }
        if (threadIdx.x == 0) {
            cum[a.E] = total <= kMaxTiles ? static_cast<int32_t>(total) : 0;
            if (total > kMaxTiles) set_status(a.status, EP_ERR_BAD_SLOT);
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = ctl.tmem;
    const int tiles = cum[a.E];
    const int kb_count = a.k_blocks;
    const int split = kSplit ? a.split : 1;
    const int part = kSplit ? static_cast<int>(cluster_rank()) : 0;
    const int t0 = kSplit ? static_cast<int>(blockIdx.x) / split : 0;
    // this CTA's blocks along K
    const int kb_first = kSplit ? static_cast<int>(static_cast<int64_t>(kb_count) * part / split) : 0;
    const int kb_end =
        kSplit ? static_cast<int>(static_cast<int64_t>(kb_count) * (part + 1) / split) : kb_count;
    uint32_t fills = 0;  // stages filled so far (the copying warp's)

    if (warp >= kAccWarps) {
        set_max_registers_down<kOtherRegs>();
        if (warp == kCopyWarp) {
            // ---- copies: one lane fills the stages in order ----
            // Of a tile with few rows only those are copied, and the stage's others
            // cleared once: products of whatever the last tile left there cost
            // power, and with it clock rate. Four bits a stage: the row box that
            // may hold something.
            // (At first, boxes that no tile fills are left as they are.)
            uint32_t row_fill = 0x11111111u * static_cast<uint32_t>(a.row_boxes - 1);
            static_assert(kStages <= 8, "four bits a stage");
            Ring<kStages> st;
            bool ok = true;
            for (int t = first_tile<kSplit>(t0); ok && t < tiles; t += tile_step<kSplit>(tiles)) {
                const Tile tile = find_tile(t, cum, a);
                const int box = tile.rows > 64 ? 3 : tile.rows > 32 ? 2 : tile.rows > 16 ? 1 : 0;
                const int w0 = tile.expert * a.n + tile.col_tile * (kGateUp ? kFp8Block : kTileCols);
                const int w1 = w0 + (kGateUp ? a.n / 2 : kFp8Block);
                for (int kb = kb_first; kb < kb_end; ++kb, st.next(), ++fills) {
                    ok = warp_wait(done + 8 * st.i, st.round ^ 1u, abort, a.status);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t dst = base + st.i * kStageBytes, bar = full + 8 * st.i;
                        const int x = kb * kTileK;
                        const int filled = max(box, static_cast<int>(row_fill >> (4 * st.i)) & 15);
                        mbar_arrive_expect_tx(bar, (16u << filled) * kTileK + 2 * kStageB);
                        tensor_load_2d(dst, &maps.rows[box], x, tile.row0, bar);
                        for (int i = box; i < filled; ++i)  // (rows past the last read as zeros)
                            tensor_load_2d(dst + (16u << i) * kTileK, &maps.rows[i], 0,
                                           static_cast<int>(a.num_recv), bar);
                        tensor_load_2d(dst + kStageA, &maps.weights, x, w0, bar);
                        tensor_load_2d(dst + kStageA + kStageB, &maps.weights, x, w1, bar);
                    }
                    __syncwarp();
                    row_fill = (row_fill & ~(15u << (4 * st.i))) | (static_cast<uint32_t>(box) << (4 * st.i));
                }
            }
        } else if (warp == kProductWarp) {
            // ---- products: one lane ----
            constexpr uint32_t kDesc = mma_desc_e4m3(kTileRows, kTileCols);
            const uint64_t desc0 = operand_desc(base);
            Ring<kStages> st;
            Ring<kSlots> slot;
            bool ok = true;
            for (int t = first_tile<kSplit>(t0); ok && t < tiles; t += tile_step<kSplit>(tiles)) {
                for (int kb = kb_first; kb < kb_end; ++kb, st.next(), slot.next()) {
                    ok = warp_wait(full + 8 * st.i, st.round, abort, a.status) &&
                         warp_wait(sums_read + 8 * slot.i, slot.round ^ 1u, abort, a.status);
                    if (!ok) break;
                    tcgen05_fence_after();
                    if (elect_one()) {
                        const uint64_t da = desc0 + st.i * (kStageBytes >> 4);
                        const uint64_t db = da + (kStageA >> 4);
#pragma unroll
                        for (int k = 0; k < kTileK / 32; ++k)
                            mma_e4m3(tmem + slot.i * kTileCols, da + 2 * k, db + 2 * k, kDesc, k > 0);
                        mma_commit(done + 8 * st.i);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == kScaleWarp) {
            // ---- scales: small copies, ahead of the sums by the stages' depth ----
            const int n_blocks = (a.n + kFp8Block - 1) / kFp8Block;
            const uint32_t row_dst = smem_u32(&ctl.row_scale[0][0][lane]);
            Ring<kScaleGroups> group;
            uint32_t tile_no = 0;
            bool ok = true;
            for (int t = first_tile<kSplit>(t0); ok && t < tiles; t += tile_step<kSplit>(tiles), ++tile_no) {
                const Tile tile = find_tile(t, cum, a);
                const int b0 = kGateUp ? tile.col_tile : 2 * tile.col_tile;
                const int b1 = kGateUp ? b0 + n_blocks / 2 : min(b0 + 1, n_blocks - 1);
                const int rows = tile.rows;
                const float* row = a.a_scale + (static_cast<int64_t>(tile.row0) + lane) * kb_count;
                const float* weight =
                    a.w_scale +
                    (static_cast<int64_t>(tile.expert) * n_blocks + ((lane & 1) == 0 ? b0 : b1)) * kb_count;
                for (int kb0 = kb_first; kb0 < kb_end; kb0 += kScaleGroup, group.next()) {
                    ok = warp_wait(scales_read + 8 * group.i, group.round ^ 1u, abort, a.status);
                    if (!ok) break;
                    const int count = min(kScaleGroup, kb_end - kb0);
                    uint32_t dst = row_dst + group.i * sizeof(ctl.row_scale[0]);
#pragma unroll 1
                    for (int i = lane; i < rows; i += 32, dst += 32 * 4) {
                        const float* src = row + static_cast<int64_t>(i - lane) * kb_count + kb0;
                        for (int j = 0; j < count; ++j) copy_async4(dst + j * (4 * kTileRows), src + j);
                    }
                    if (lane < 2 * count) {
                        const uint32_t j = lane >> 1;
                        copy_async4(smem_u32(&ctl.weight_scale[group.i][j][lane & 1]), weight + kb0 + j);
                    }
                    copy_async_arrive(scales + 8 * group.i);
                    if (lane == 0) {
                        if (kb0 == kb_first)
                            ctl.notes[tile_no % kTileNotes] = {tile.row0, tile.rows, tile.col_tile};
                        mbar_arrive(scales + 8 * group.i);  // (releases the note)
                    }
                }
            }
            copy_async_wait_all();
        }
        if (kSplit) {
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
    } else {
        // ---- scaled sums: thread = one row, columns [32 c, 32 c + 32) of both blocks ----
        set_max_registers_up<kAccRegs>();
        const int c = warp >> 2, quarter = warp & 3;
        const uint32_t row_scale = smem_u32(&ctl.row_scale[0][0][quarter * 32 + lane]);
        const uint32_t weight_scale = smem_u32(ctl.weight_scale);
        uint32_t sums = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c * kAccCols;
        uint32_t read = sums_read;
        Ring<kScaleGroups> group;
        Ring<kStages> st;
        uint32_t tile_no = 0;
        bool ok = true;
        if (kSplit && t0 >= tiles) {
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
        }
        for (int t = first_tile<kSplit>(t0); ok && t < tiles; t += tile_step<kSplit>(tiles), ++tile_no) {
            float acc[2][kAccCols];
#pragma unroll
            for (int i = 0; i < kAccCols; ++i) acc[0][i] = acc[1][i] = 0.0f;
            // The loop has no branch but the waits': warps whose rows the tile lacks
            // add along (with a branch around that, 32768 rows on 256 experts took
            // 1706 us instead of 1377), and after a wait that gave up the rest of
            // the tile runs on without waiting or arriving.
            for (int kb0 = kb_first; kb0 < kb_end; kb0 += kScaleGroup, group.next()) {
                ok = ok && warp_wait(scales + 8 * group.i, group.round, abort, a.status);
                uint32_t row_at = row_scale + group.i * sizeof(ctl.row_scale[0]);
                uint32_t weight_at = weight_scale + group.i * sizeof(ctl.weight_scale[0]);
                const int kb1 = min(kb0 + kScaleGroup, kb_end);
#pragma unroll 1
                for (int kb = kb0; kb < kb1; ++kb) {
                    const float sa = load_shared_f32(row_at);
                    const float2 sw = load_shared_f32x2(weight_at);
                    const float s0 = sa * sw.x, s1 = sa * sw.y;
                    ok = ok && warp_wait(done + 8 * st.i, st.round, abort, a.status);
                    st.next();
                    tcgen05_fence_after();
                    uint32_t v[16];
                    tmem_load16(sums, v);
                    tmem_load_wait16(v);
                    add_scaled(acc[0], 0, v, s0);
                    tmem_load16(sums + 16, v);
                    tmem_load_wait16(v);
                    add_scaled(acc[0], 16, v, s0);
                    tmem_load16(sums + kFp8Block, v);
                    tmem_load_wait16(v);
                    add_scaled(acc[1], 0, v, s1);
                    tmem_load16(sums + kFp8Block + 16, v);
                    tmem_load_wait16(v);
                    tcgen05_fence_before();
                    mbar_arrive_if(read, ok && lane == 0);
                    add_scaled(acc[1], 16, v, s1);
                    row_at += sizeof(ctl.row_scale[0][0]);
                    weight_at += sizeof(ctl.weight_scale[0][0]);
                    sums ^= kTileCols;  // the other place: tmem starts at a multiple of 512
                    read ^= 8u;         // sums_read is 16-byte aligned
                }
                __syncwarp();
                mbar_arrive_if(scales_read + 8 * group.i, ok && lane == 0);
            }
            const int row = quarter * 32 + lane;
            const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
            if (kSplit)
                join_parts(acc, base, ok ? ctl.notes[0].rows : 0, row, c * kAccCols * 4, rank, split);
            if (!ok) break;
            const TileNote tile = ctl.notes[tile_no % kTileNotes];
            const bool store = row < tile.rows && row % split == rank;
            const int64_t grow = static_cast<int64_t>(tile.row0) + row;
            if (kGateUp) {
                // silu(g) = g / (1 + e^-g) = g e^g / (1 + e^g): the one whose
                // exponential does not overflow, so that the divisor lies in
                // [1, 2] for every g and small values shrink into fp32's
                // subnormals. (As g / (1 + e^-g) alone an approximate division
                // gives 0 from g = -87.3 on, where the divisor passes 2^126.)
                // Approximate exponential and reciprocal: off by a few units of
                // 2^-24 (and |g| of them for the exponential), well inside what
                // the sums before and the e4m3 rounding after are off by; exact
                // ones took 2 us of a tile, and 8 us where lanes without a row
                // brought NaN into their slow paths.
                uint32_t top = 0;
                if (quarter * 32 < tile.rows) {
#pragma unroll
                    for (int i = 0; i < kAccCols; ++i) {
                        const float g = acc[0][i];
                        const float t = __expf(-fabsf(g));
                        acc[0][i] = (g < 0.0f ? g * t : g) * reciprocal(1.0f + t) * acc[1][i];
                        top = max(top, abs_bits(acc[0][i]));
                    }
                }
                // the block's other columns are in the other groups' warps
                uint32_t* amax = &ctl.amax[tile_no & 1][0][row];
                amax[c * kTileRows] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = warp_wait(joined, tile_no & 1, abort, a.status);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < kAccGroups; ++i) top = max(top, amax[i * kTileRows]);
                const BlockScale bs = block_scale(top);
                if (store) {
                    const int width = a.n / 2;
                    uint8_t* q = a.out_q + grow * width + tile.col_tile * kFp8Block + c * kAccCols;
#pragma unroll
                    for (int i = 0; i < kAccCols / 16; ++i) {
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* f = &acc[0][i * 16 + j * 4];
                            p[j] = pack_e4m3x4(f[0] * bs.inverse, f[1] * bs.inverse,
                                               f[2] * bs.inverse, f[3] * bs.inverse);
                        }
                        st_v4(q + i * 16, make_uint4(p[0], p[1], p[2], p[3]));
                    }
                    if (c == 0) a.out_scale[grow * (width / kFp8Block) + tile.col_tile] = bs.scale;
                }
            } else {
                // A lane holds 64 bytes of one row and block. Four lanes exchange
                // 16-byte pieces first, so that a store covers 64 contiguous
                // bytes of eight rows instead of 16 of 32: its cost goes by rows.
                const int piece = lane & 3;
                const int64_t col0 =
                    static_cast<int64_t>(tile.col_tile) * kTileCols + c * kAccCols + piece * 8;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint4 p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float* f = &acc[b][i * 8];
                        p[i] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                    }
                    transpose4(p, piece);
                    const int64_t col = col0 + b * kFp8Block;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = quarter * 32 + (lane & ~3) + i;
                        if (r < tile.rows && r % split == rank && col < a.n)
                            st_v4(a.out + (static_cast<int64_t>(tile.row0) + r) * a.n + col, p[i]);
                    }
                }
            }
            // (With the step alone the loop's state was kept over join_parts, and
            // 228 bytes of sums spilled: 5 % of a split call.)
            if (kSplit) break;
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    if (kSplit) cluster_wait();  // no CTA reads this one's sums any more
    // After a wait that gave up: no copy may land once the CTA has exited, and
    // no product may run once its tensor memory is released. (Otherwise every
    // copy and product has been waited for.)
    if (load_shared(abort) != 0) {
        if (warp == kCopyWarp && lane == 0)
            mbar_drain_bounded<kStages>(full, fills > kStages ? fills - kStages : 0u,
                                        static_cast<int64_t>(fills) - 1);
        if (warp == kProductWarp) {
            const uint32_t bar = smem_u32(&ctl.drained);
            if (elect_one()) mma_commit(bar);
            __syncwarp();
            mbar_wait_bounded(bar, 0);
        }
    }
    __syncwarp();
    if (warp == kProductWarp) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's, looked up once (a failure is not kept).
EncodeFn encode_fn() {
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

// A byte matrix [rows][width], read in boxes of box_rows x 128 bytes laid out
// with the 128-byte swizzle.
bool encode_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t width, int box_rows) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width)};
    const cuuint32_t box[2] = {kTileK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The warpgroups' registers come out of those of the launch; with fewer the
// ones that ask for more would wait forever.
template <bool kGateUp, bool kSplit>
cudaError_t check_registers(int device) {
    static PerDevice<bool> enough;
    bool ok = false;
    const cudaError_t err = enough.get(device, &ok, [](bool* found) {
        cudaFuncAttributes fa{};
        const cudaError_t e = cudaFuncGetAttributes(&fa, expert_kernel<kGateUp, kSplit>);
        *found = fa.numRegs >= kLaunchRegs;
        return e;
    });
    if (err != cudaSuccess) return err;
    return ok ? cudaSuccess : cudaErrorInvalidDeviceFunction;
}

template <bool kGateUp, bool kSplit>
cudaError_t launch(const ExpertArgs& a, const Maps& maps, int device, int grid, size_t smem,
                   cudaStream_t stream) {
    auto kern = expert_kernel<kGateUp, kSplit>;
    cudaError_t err = check_registers<kGateUp, kSplit>(device);
    if (err != cudaSuccess) return err;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_dependent_clusters(kern, grid, a.split, kThreads, smem, stream, a, maps);
}

// Clusters of 2, 4, 8 CTAs (n[2], n[4], n[8]) that a device holds at a time:
// fewer than SMs / size, because a cluster's lie in one part (GPC) of it.
struct ResidentClusters {
    int n[kMaxSplit + 1];
};

cudaError_t resident_clusters(int device, ResidentClusters* clusters) {
    static PerDevice<ResidentClusters> table;
    return table.get(device, clusters, [](ResidentClusters* found) {
        auto kern = expert_kernel<false, true>;
        const size_t smem = 1024 + kStages * kStageBytes;
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
        for (int split = 2; err == cudaSuccess && split <= kMaxSplit; split *= 2) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(split));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(split);
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            err = cudaOccupancyMaxActiveClusters(&found->n[split], kern, &cfg);
        }
        return err;
    });
}

// CTAs to share a tile's blocks along K, where `most` tiles leave SMs idle. A
// block takes a CTA 0.38 us then (the copies' latency over four stages); the
// cluster's launch, its barriers and the joining take 2-3.5 us for few rows
// and 4-5.5 us for 128, so at least 12 (16) blocks have to go to other CTAs:
// one row of 7168 x 2 x 2048 took 26.2 us with 16 CTAs, 17.4 with clusters of
// two, 13.6 of four; of 2048 x 7168 10.0, 9.6, 8.5; with two experts of those
// and clusters of two 11.9 instead of 11.4 (not split); with 128 rows to each
// of 16 tiles 56 blocks deep 27.2, 19.7, 15.7, but 14.1 instead of 11.9 16
// blocks deep (not split). Clusters of 3, 5, 6 and 7 were between these or, at
// 28 tiles, 30 % slower than four. A partition's SMs may not hold a cluster.
// (The split sets the order of the sums: a device that cannot be asked is an
// error, not a reason for another one.)
cudaError_t split_for(const ExpertArgs& a, int64_t most, int device, int num_sms, bool partition,
                      int* split) {
    *split = 1;
    if (partition || 2 * most > num_sms) return cudaSuccess;
    ResidentClusters clusters{};
    const cudaError_t err = resident_clusters(device, &clusters);
    if (err != cudaSuccess) return err;
    int n = 1;
    while (n < kMaxSplit && most <= clusters.n[2 * n]) n *= 2;
    const int rows = static_cast<int>(a.num_recv < kTileRows ? a.num_recv : kTileRows);
    const int passed_on = a.k_blocks - (a.k_blocks + n - 1) / n;
    if (passed_on >= 12 + rows / 32) *split = n;
    return cudaSuccess;
}

}  // namespace

int64_t expert_tiles_bound(int64_t num_recv, int E, int64_t n, bool gated) {
    const int64_t col_tiles = gated ? n / 2 / kFp8Block : (n + kTileCols - 1) / kTileCols;
    const int64_t row_tiles = num_recv / kTileRows + (num_recv < E ? num_recv : E);
    return row_tiles * col_tiles;
}

cudaError_t launch_expert(ExpertArgs a, int num_sms, bool partition, cudaStream_t stream) {
    const bool gated = a.out_q != nullptr;
    a.k_blocks = static_cast<int>((a.k + kFp8Block - 1) / kFp8Block);
    a.col_tiles = gated ? a.n / 2 / kFp8Block : (a.n + kTileCols - 1) / kTileCols;
    Maps maps;
    // no tile has more rows than there are: row boxes up to those are all it needs
    a.row_boxes = 1;
    while (a.row_boxes < kRowBoxes && (8 << a.row_boxes) < a.num_recv) ++a.row_boxes;
    for (int i = 0; i < a.row_boxes; ++i)
        if (!encode_map(&maps.rows[i], a.a, a.num_recv, a.k, 16 << i)) return cudaErrorInvalidValue;
    if (!encode_map(&maps.weights, a.w, static_cast<int64_t>(a.E) * a.n, a.k, kFp8Block))
        return cudaErrorInvalidValue;
    // at most this many tiles, checked against kMaxTiles by the caller
    const int64_t most = expert_tiles_bound(a.num_recv, a.E, a.n, gated);
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = split_for(a, most, device, num_sms, partition, &a.split);
    if (err != cudaSuccess) return err;
    const int grid = static_cast<int>(a.split > 1 ? most * a.split : most < num_sms ? most : num_sms);
    const size_t smem = 1024 + kStages * kStageBytes + sizeof(int32_t) * (a.E + 1);
    if (a.split > 1)
        return gated ? launch<true, true>(a, maps, device, grid, smem, stream)
                     : launch<false, true>(a, maps, device, grid, smem, stream);
    return gated ? launch<true, false>(a, maps, device, grid, smem, stream)
                 : launch<false, false>(a, maps, device, grid, smem, stream);
}

}  // namespace ep
