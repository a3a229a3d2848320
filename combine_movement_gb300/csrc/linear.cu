// linear.cu -- dense products in bf16 with fp32 sums,
//
//   v[m, n] = sum_k a[m, k] * b[n, k] + bias[n]
//   out[m, n] = act(v[m, n]) + residual[m, n]
//
// (gated: b's rows are a gate half and an up half, out = silu(gate) * up +
// residual), v kept in bf16 where asked for. Each operand has its rows along k
// or (its gradients' products) runs along m or n, k by k.
//
// Mapping. A stage of shared memory takes 64 values along k of a tile's rows of both
// operands (tensor copies, 128-byte swizzle; an operand that runs along m or n in
// groups of 64 by 64, which the product reads as it lies); one thread issues four
// tcgen05.mma, 16 values along k each, and a tile's sums stay in tensor memory, in one
// of two places, so that eight warps write a tile while the next one's products run.
// Three ways to make a tile, by what the sizes leave to do (plan_for):
//  - pairs of CTAs (cta_group::2) on 256 x 256, persistent: each brings in its 128 rows
//    of a and half of b, 32 KB for 512 cycles of products, which is what an SM
//    takes in (64 bytes a cycle; one CTA on 128 x 256 needs 96, and took 20 % longer);
//  - one CTA on 128 x 64, persistent: more tiles of small outputs;
//  - clusters of 2 to 16 CTAs on 128 x 64, 128 or 256 that share a tile's blocks along k
//    and add their sums through shared memory: few tiles, long k.
// A tensor core's fp32 sum loses more at each of its steps than rounding to nearest does,
// and to one side: 7168 products in a row are off by 8e-6 of their norm where their signs
// are mixed and by 4e-5 where they are alike, 131072 by 7e-4, a million by 6.5e-3. In parts of
// 1024 that are added in fp32 registers 7168 are off by 9e-7. So are all fp32
// results made, and bf16 results of more than 8192 products in a row (a step loses at
// most a unit of 2^-23 of the sum so far and takes at least 8 products: of 8192 at most 2^-14,
// a 64th of what a bf16 result loses at its end). Parts take 1-3 % longer.
//
// Results. Sums that are the result but for rounding leave by the copy engine, 32 x 32
// at a time. The others are turned around in shared memory, from a row to a lane to
// rows across lanes, for bias, activation and residual and for stores along rows.
//
// What bounds it. Large products: the tensor cores at 0.87 of their cycles (4096 x 4096 x
// 7168: 119-138 us for a few launches after a rest, 1.75-2.0 PFLOP/s by card; for seconds the
// board's power limit, 146 us, where the library's product takes 139-142). 16384 x 2048 x 7168
// with a residual 261 us after a rest, 300-317 for seconds (the library's 345). Few columns:
// 16384 x 7168 x 256 47-51 us, 0.8 of the copy rate: 64 pairs leave 24 SMs idle, and each
// reads all of b. Small ones:
// 128 x 7168 x 256 7.0 us: 0.2 us from launch to the first copy, 1.1 until it lands, 0.17 a
// block along k (what the copying and the product's warp take to wait for it and issue it, the
// same without the copies or without the products), 2 to join 16 parts, 0.7 to end
// together. A few rows: 8 x 7168 x 2048 8.7 us, of which 2.7 are a kernel with one block;
// 8 x 7168 x 4096 14 (4.3 TB/s).
// Measured and not kept: k begun at another block in each tile (nothing), rows brought
// into L2 ahead (2-30 % slower), more stages where few rows of a leave room (0.4 us slower on
// small calls, their number not being a constant), 128 values to a stage (0-10 % slower), a look
// at the next barrier before a block's issue (0.1-0.3 us slower on small calls), a warp's loop
// gone through by one lane alone (0.33 us a block).
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "kernels.cuh"
#include "linear_out.cuh"
#include "per_device.cuh"
#include "product.cuh"

namespace ep {
namespace {

// Who works on a tile: a CTA alone or the CTAs of a cluster that share its blocks
// along k, on 128 x 64 (gated: 32 columns of each half; kSharedMid 128 x 128, kSharedWide
// 128 x 256), or a pair of CTAs on 256 x 256 (gated: 128 of each half), 128 rows and
// half of b each.
enum Mode { kAlone, kShared, kSharedMid, kSharedWide, kPair };

constexpr unsigned kFullMask = 0xFFFFFFFFu;
constexpr int kRows = 128;                   // of the output, in one CTA
constexpr int kTileK = 64;                   // values of one stage along k
constexpr uint32_t kRowBytes = kTileK * 2;
constexpr uint32_t kGroupBytes = 64 * 128;   // 64 along k x 64 along m or n
constexpr uint32_t kStageA = kRows * kRowBytes;
constexpr int kSlots = 2;
constexpr int kOutWarps = 8;
constexpr int kProductWarp = kOutWarps, kCopyWarp = kOutWarps + 1;
constexpr int kThreads = (kOutWarps + 2) * 32;
constexpr int kChunk = 32;                   // columns turned around at a time
constexpr uint32_t kTurnBytes = 32 * kChunk * 4;
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 16;
constexpr int kRowGroup = 8;                 // row tiles that share a column tile's turn
// Blocks along k after which a tile's sums leave tensor memory, for fp32 results; and
// how many bf16 results may be of before they do the same.
constexpr int kExactBlocks = 16;
constexpr int kLongBlocks = 128;

template <Mode kMode>
struct Shape {
    static constexpr bool kParts = kMode == kShared || kMode == kSharedMid || kMode == kSharedWide;
    static constexpr int kCols =                                  // of the tile
        kMode == kPair || kMode == kSharedWide ? 256 : kMode == kSharedMid ? 128 : 64;
    static constexpr int kTileRows = kMode == kPair ? 2 * kRows : kRows;
    static constexpr int kOwnB = kMode == kPair ? kCols / 2 : kCols;  // rows of b in one CTA
    static constexpr uint32_t kStageBytes = kStageA + kOwnB * kRowBytes;
    // (shared tiles leave room for the next kernel's CTA beside theirs, so that it has
    // begun when they end)
    static constexpr int kStages = kMode == kShared ? 4 : 192 * 1024 / kStageBytes;
    static constexpr uint32_t kRingBytes = kStages * kStageBytes;
    static constexpr size_t kSmem = 1024 + kRingBytes + (kParts ? 0 : kOutWarps * kTurnBytes);
    static constexpr int kMine = kCols / 2;  // columns of sums that a warp takes
    // a shared tile's sums, [row][column] in fp32, in the stages' place
    static constexpr uint32_t kPitch = kCols * 4 + 16;
    static_assert(kStages <= kMaxStages && kRows * kPitch <= kRingBytes, "shared memory");
};

struct Maps {
    CUtensorMap a, b;
    CUtensorMap out;                         // where `plain`
    bool plain;                              // out is the rounded sums, in aligned rows
    int a_rows;                              // of a's box along m (not by_k)
};

struct Control {
    uint64_t full[kMaxStages];    // the copies have landed (a pair's: rank 0's)
    uint64_t done[kMaxStages];    // the stage's product is done
    uint64_t sums[kSlots];        // a tile's sums are complete
    uint64_t sums_read[kSlots];   // and have been read: the writing warps (rank 0's)
    uint64_t drained;             // after an abort: products still in flight
    uint32_t tmem;
    int32_t abort;
};

struct Tile {
    int64_t row0;
    int64_t col_tile;
};
// Groups of kRowGroup row tiles, column tiles outside of row tiles in each: the
// tiles that run at a time share their rows of both operands.
template <Mode kMode>
__device__ __forceinline__ Tile tile_at(int64_t t, const LinearArgs& a) {
    const int64_t per = kRowGroup * a.col_tiles;
    const int64_t group = t / per, r0 = group * kRowGroup;
    const int64_t rows = min(static_cast<int64_t>(kRowGroup), a.row_tiles - r0);
    const int64_t i = t - group * per;
    return {(r0 + i % rows) * Shape<kMode>::kTileRows, i / rows};
}

// 16-byte piece p of row r of a warp's turning place.
__device__ __forceinline__ uint32_t turn_at(uint32_t turn, int r, int p) {
    return turn + r * (kChunk * 4) + ((p ^ (r & 7)) << 4);
}

// A warp's part of out: 32 rows from row0 on, of which `rows` are there.
struct Part {
    int64_t row0;
    int rows;
};

// How a warp goes through the 32 rows of a chunk's columns of out, N of them to a
// lane: kRounds times kAtOnce rows.
template <int N, bool kGated>
struct Walk {
    static constexpr int kCols = kGated ? kChunk / 2 : kChunk;
    static constexpr int kPieces = kCols / N, kAtOnce = 32 / kPieces, kRounds = 32 / kAtOnce;
};

// N neighbouring sums of a row from shared memory.
template <int N>
__device__ __forceinline__ Values<N> load_sums(uint32_t at) {
    if constexpr (N == 4) {
        const float4 f = load_shared_v4(at);
        return {{f.x, f.y, f.z, f.w}};
    } else if constexpr (N == 2) {
        const float2 f = load_shared_f32x2(at);
        return {{f.x, f.y}};
    } else {
        return {{load_shared_f32(at)}};
    }
}
// Those of row r from value c of a chunk on, in its turning place.
template <int N>
__device__ __forceinline__ Values<N> turned(uint32_t turn, int r, int c) {
    return load_sums<N>(turn_at(turn, r, c / 4) + c % 4 * 4);
}

// What a lane adds to its values of a chunk, read ahead of them.
struct Ahead {
    uint32_t bits[32];
};
template <int N, bool kGated>
__device__ __forceinline__ void read_ahead(const LinearArgs& a, const Part& part, int64_t col,
                                           Ahead& ahead) {
    using W = Walk<N, kGated>;
    const int lane = threadIdx.x & 31, r0 = lane / W::kPieces;
    const int64_t c = col + lane % W::kPieces * N;
    if (c >= a.n) return;
    int64_t at = (part.row0 + r0) * a.n + c;
#pragma unroll
    for (int i = 0; i < W::kRounds; ++i, at += W::kAtOnce * a.n) {
        if (r0 + i * W::kAtOnce >= part.rows) continue;
        const Residual<N> v = load_residual<N>(a, at);
#pragma unroll
        for (int j = 0; j < N; ++j) ahead.bits[N * i + j] = v.bits[j];
    }
}
template <bool kGated>
__device__ __forceinline__ void read_ahead(const LinearArgs& a, const Part& part, int64_t col,
                                           Ahead& ahead) {
    if (a.residual != nullptr)
        by_width(a.n, [&](auto n) { read_ahead<decltype(n)::value, kGated>(a, part, col, ahead); });
}

// A chunk from its turning place to out, with all that may be asked for: `col` the
// column of its first sums (gated: of 16 of each half). kWhole: all of a lane's values
// at once, for CTAs that write many chunks: the instructions overlap (a tile of 256 x
// 256 with silu takes 2.5 us, in eights 9). Else eight values at a time: a small call
// goes through these instructions once, and its time is that of bringing them in (333 x
// 1075 with all of it 3 us, whole 4.7); the next ones' residual is on the way.
template <int N, bool kGated, bool kWhole>
__device__ __forceinline__ void write_chunk(const LinearArgs& a, uint32_t turn, const Part& part,
                                            int64_t col, const Ahead& ahead) {
    using W = Walk<N, kGated>;
    constexpr int kStep = kWhole ? W::kRounds : 8 / N;  // rounds at a time
    const int lane = threadIdx.x & 31, p = lane % W::kPieces * N, r0 = lane / W::kPieces;
    const int64_t c = col + p;
    if (c >= a.n) return;
    const Values<N> b0 = load_bias<N>(a.bias, c), b1 = load_bias<N>(a.bias, kGated ? a.n + c : c);
    auto residual = [&](int i) {
        const int r = r0 + i * W::kAtOnce;
        if (a.residual == nullptr || r >= part.rows) return Residual<N>{};
        return load_residual<N>(a, (part.row0 + r) * a.n + c);
    };
    Residual<N> now[kStep], next[kStep];
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
        if constexpr (kWhole) {
#pragma unroll
            for (int i = 0; i < N; ++i) now[j].bits[i] = ahead.bits[N * j + i];
        } else {
            next[j] = residual(j);
        }
    }
#pragma unroll 1
    for (int i = 0; i < W::kRounds; i += kStep) {
        if constexpr (!kWhole) {
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                now[j] = next[j];
                next[j] = residual(i + kStep + j);
            }
        }
        const int r = r0 + i * W::kAtOnce;
        Values<N> v[kStep], up[kStep];
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            v[j] = turned<N>(turn, r + j * W::kAtOnce, p) + b0;
            up[j] = kGated ? turned<N>(turn, r + j * W::kAtOnce, p + W::kCols) + b1 : v[j];
        }
        const int rows = (part.rows - r + W::kAtOnce - 1) / W::kAtOnce;
        finish<N, kGated>(a, part.row0 + r, c, W::kAtOnce, rows, v, up, now);
    }
}

// The sums of a tile that the cluster's CTAs took parts of k of: each has laid
// its own out in shared memory; CTA `rank` adds, in the parts' order, and writes
// those of the rows r = rank mod kParts. A thread takes N neighbouring columns
// of a few rows at a time, so that its loads overlap.
template <int N>
__device__ __forceinline__ Values<N> load_cluster(uint32_t at) {
    if constexpr (N == 4) {
        const float4 f = load_cluster_v4(at);
        return {{f.x, f.y, f.z, f.w}};
    } else {
        Values<N> r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = load_cluster_f32(at + 4 * i);
        return r;
    }
}
template <Mode kMode, int N, bool kGated, int kParts>
__device__ __forceinline__ void write_shared_tile(const LinearArgs& a, uint32_t sums, const Tile& tile,
                                                  int rank) {
    using S = Shape<kMode>;
    constexpr int kCols = kGated ? S::kCols / 2 : S::kCols, kPieces = kCols / N;
    constexpr int kStep = kOutWarps * 32 / kPieces;  // of this CTA's rows, by all threads
    constexpr int kMost = kRows / kParts / kStep;    // of them to a thread
    constexpr int kWant = kParts >= 8 ? 4 / N : 32 / kParts / N;  // loads in flight
    constexpr int kAtOnce = kMost < 1 || kWant < 1 ? 1 : kMost < kWant ? kMost : kWant;
    const int64_t rows_left = a.m - tile.row0;
    const int rows = static_cast<int>(rows_left < kRows ? rows_left : kRows);
    const int own = (rows + kParts - 1 - rank) / kParts;
    const int c = threadIdx.x % kPieces * N;
    const int64_t col = tile.col_tile * kCols + c;
    if (col >= a.n) return;
    const Values<N> b0 = load_bias<N>(a.bias, col), b1 = load_bias<N>(a.bias, kGated ? a.n + col : col);
#pragma unroll 1
    for (int i0 = threadIdx.x / kPieces; i0 < own; i0 += kAtOnce * kStep) {
        Values<N> v[kAtOnce][kParts], up[kAtOnce][kParts], vs[kAtOnce], us[kAtOnce];
        Residual<N> res[kAtOnce] = {};
        const int64_t row = tile.row0 + i0 * kParts + rank;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = min(i0 + j * kStep, own - 1);  // (rows past the last: it again)
            if (a.residual != nullptr)
                res[j] = load_residual<N>(a, (tile.row0 + i * kParts + rank) * a.n + col);
            const uint32_t at = sums + (i * kParts + rank) * S::kPitch + c * 4;
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const uint32_t from = cluster_map(at, p);
                v[j][p] = load_cluster<N>(from);
                if (kGated) up[j][p] = load_cluster<N>(from + kCols * 4);
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            vs[j] = v[j][0];
            us[j] = kGated ? up[j][0] : v[j][0];
#pragma unroll
            for (int p = 1; p < kParts; ++p) {
                vs[j] = vs[j] + v[j][p];
                if (kGated) us[j] = us[j] + up[j][p];
            }
            vs[j] = vs[j] + b0;
            if (kGated) us[j] = us[j] + b1;
        }
        finish<N, kGated>(a, row, col, kStep * kParts, (own - i0 + kStep - 1) / kStep, vs, us, res);
    }
}
template <Mode kMode, bool kGated>
__device__ __forceinline__ void write_shared_tile(const LinearArgs& a, uint32_t sums, const Tile& tile,
                                                  int rank) {
    by_width(a.n, [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (a.split == 2)
            write_shared_tile<kMode, N, kGated, 2>(a, sums, tile, rank);
        else if (a.split == 4)
            write_shared_tile<kMode, N, kGated, 4>(a, sums, tile, rank);
        else if (a.split == 8)
            write_shared_tile<kMode, N, kGated, 8>(a, sums, tile, rank);
        else if (kMode == kShared && a.split == 16)
            write_shared_tile<kMode, N, kGated, 16>(a, sums, tile, rank);
    });
}

// 32 x 32 sums of a warp into its turning place.
__device__ __forceinline__ void turn_chunk(uint32_t turn, const float* v0, const float* v1) {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // the chunk before has been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        store_shared_v4(turn_at(turn, lane, i),
                        make_float4(v0[4 * i], v0[4 * i + 1], v0[4 * i + 2], v0[4 * i + 3]));
        store_shared_v4(turn_at(turn, lane, 4 + i),
                        make_float4(v1[4 * i], v1[4 * i + 1], v1[4 * i + 2], v1[4 * i + 3]));
    }
    __syncwarp();
}

// A chunk that is out as it is: each lane lays its row's 32 sums out as the copy
// engine's swizzle has them (fp32 rows of 128 bytes: the turning place's own; bf16 rows
// of 64), which takes them out together. `second`: of two places that take turns.
__device__ __forceinline__ void send_chunk(const LinearArgs& a, const Maps& maps, uint32_t turn,
                                           const Part& part, int64_t col, bool second,
                                           const uint32_t (&v)[2][16]) {
    const int lane = threadIdx.x & 31;
    if (a.out_f32) {
        if (elect_one()) bulk_wait_read<0>();  // the chunk before has left
        turn_chunk(turn, reinterpret_cast<const float*>(v[0]), reinterpret_cast<const float*>(v[1]));
    } else {
        if (elect_one()) bulk_wait_read<1>();  // the one before that
        __syncwarp();
        turn += second ? kTurnBytes / 2 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t* w = &v[i / 2][i % 2 * 8];
            auto pack = [&](int j) {
                return pack_bf16x2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
            };
            const uint32_t at = turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4);
            store_shared_v4(at, make_float4(__uint_as_float(pack(0)), __uint_as_float(pack(2)),
                                            __uint_as_float(pack(4)), __uint_as_float(pack(6))));
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
        tensor_store_2d(&maps.out, static_cast<int>(col), static_cast<int>(part.row0), turn);
        bulk_commit();
    }
    __syncwarp();
}

// kExact: sums leave tensor memory every kExactBlocks blocks along k and are added
// in registers.
template <Mode kMode, bool kGated, bool kExact>
__global__ void __launch_bounds__(kThreads, kMode == kShared ? 2 : 1)
    linear_kernel(const LinearArgs a, const __grid_constant__ Maps maps) {
    using S = Shape<kMode>;
    constexpr bool kClusters = kMode != kAlone;
    constexpr uint32_t kTmemCols = kSlots * S::kCols;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // the swizzle's period
    // (from one lane: what the warps' loops go by is then known to be the same in all)
    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(ctl.full), done = smem_u32(ctl.done);
    const uint32_t sums = smem_u32(ctl.sums), sums_read = smem_u32(ctl.sums_read);
    const uint32_t abort = smem_u32(&ctl.abort);
    const int rank = kClusters ? __shfl_sync(kFullMask, static_cast<int>(cluster_rank()), 0) : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(sums + 8 * i, 1);
            mbar_init(sums_read + 8 * i, kMode == kPair ? 2 * kOutWarps : kOutWarps);
        }
        mbar_init(smem_u32(&ctl.drained), 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == kProductWarp) {
        if constexpr (kMode == kPair)
            tmem_alloc_pair(smem_u32(&ctl.tmem), kTmemCols);
        else
            tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensor_map(&maps.a);
        prefetch_tensor_map(&maps.b);
        if (maps.plain) prefetch_tensor_map(&maps.out);
    }
    tcgen05_fence_before();
    __syncthreads();
    if (kMode == kPair) {  // both CTAs' barriers and tensor memory are there
        cluster_arrive();
        cluster_wait();
    }
    tcgen05_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = __shfl_sync(kFullMask, ctl.tmem, 0);
    const int64_t tiles = a.row_tiles * a.col_tiles;
    const int size = kMode == kPair ? 2 : S::kParts ? a.split : 1;
    const int64_t t0 = blockIdx.x / size;
    const int64_t step = S::kParts ? tiles : gridDim.x / size;
    const int kb_first =
        S::kParts ? static_cast<int>(static_cast<int64_t>(a.k_blocks) * rank / size) : 0;
    const int kb_end = S::kParts
                           ? static_cast<int>(static_cast<int64_t>(a.k_blocks) * (rank + 1) / size)
                           : a.k_blocks;
    const int per_sum = kExact ? kExactBlocks : kb_end - kb_first;  // blocks
    int64_t fills = 0;  // stages filled so far (the copying warp's)

    if (warp == kCopyWarp) {
        // ---- copies: one lane fills the stages in order ----
        const int a_groups = kMode == kPair || a.m > 64 ? 2 : 1;
        const uint32_t bytes =
            S::kOwnB * kRowBytes +
            (a.a_by_k ? a_groups * kGroupBytes : static_cast<uint32_t>(maps.a_rows) * kRowBytes);
        auto load = [](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
            if constexpr (kMode == kPair)
                tensor_load_2d_pair(dst, map, x, y, bar);
            else
                tensor_load_2d(dst, map, x, y, bar);
        };
        Ring<S::kStages> st;
        bool ok = true;
        for (int64_t t = t0; ok && t < tiles; t += step) {
            const Tile tile = tile_at<kMode>(t, a);
            const int row0 = static_cast<int>(tile.row0) + (kMode == kPair ? rank * kRows : 0);
            const int col0 = static_cast<int>(tile.col_tile) * (kGated ? S::kCols / 2 : S::kCols);
            const int col1 = kGated ? static_cast<int>(a.n) + col0 : col0 + S::kCols / 2;
            for (int kb = kb_first; kb < kb_end; ++kb, st.next(), ++fills) {
                ok = warp_wait<kMode == kPair>(done + 8 * st.i, st.round ^ 1u, abort, a.status);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t dst_a = base + st.i * S::kStageBytes, dst_b = dst_a + kStageA;
                    const int k = kb * kTileK;
                    uint32_t bar = full + 8 * st.i;
                    if (kMode == kPair) {
                        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
                        bar = cluster_map(bar, 0);
                    } else {
                        mbar_arrive_expect_tx(bar, bytes);
                    }
                    if (a.a_by_k) {
                        for (int g = 0; g < a_groups; ++g)
                            load(dst_a + g * kGroupBytes, &maps.a, row0 + 64 * g, k, bar);
                    } else {
                        load(dst_a, &maps.a, k, row0, bar);
                    }
                    if (a.b_by_k) {
                        const int c = kMode == kPair && rank == 1 ? col1 : col0;
#pragma unroll
                        for (int g = 0; g < S::kOwnB / 64; ++g)
                            load(dst_b + g * kGroupBytes, &maps.b, c + 64 * g, k, bar);
                    } else {
                        load(dst_b, &maps.b, k, kMode == kPair && rank == 1 ? col1 : col0, bar);
                        if (kGated && kMode != kPair)
                            load(dst_b + S::kCols / 2 * kRowBytes, &maps.b, k, col1, bar);
                    }
                }
                __syncwarp();
            }
        }
        // the last products' arrivals, too, come before the CTA's end
        for (int i = 0; ok && i < S::kStages; ++i, st.next())
            ok = warp_wait<kMode == kPair>(done + 8 * st.i, st.round ^ 1u, abort, a.status);
    } else if (warp == kProductWarp) {
        // ---- products: one lane (of a pair, rank 0's) ----
        const uint32_t desc = mma_desc_bf16(S::kTileRows, S::kCols, a.a_by_k, a.b_by_k);
        const uint64_t desc_a = a.a_by_k ? operand_desc_by_k(base) : operand_desc(base);
        const uint64_t desc_b =
            a.b_by_k ? operand_desc_by_k(base + kStageA) : operand_desc(base + kStageA);
        const uint32_t step_a = (a.a_by_k ? 2048 : 32) >> 4, step_b = (a.b_by_k ? 2048 : 32) >> 4;
        Ring<S::kStages> st;
        Ring<kSlots> slot;
        bool ok = kMode != kPair || rank == 0;
        for (int64_t t = t0; ok && t < tiles; t += step) {
            for (int kb0 = kb_first; ok && kb0 < kb_end; kb0 += per_sum, slot.next()) {
                ok = warp_wait<kMode == kPair>(sums_read + 8 * slot.i, slot.round ^ 1u, abort, a.status);
                if (!ok) break;
                tcgen05_fence_after();
                const int kb1 = min(kb0 + per_sum, kb_end);
                for (int kb = kb0; kb < kb1; ++kb, st.next()) {
                    ok = warp_wait<kMode == kPair>(full + 8 * st.i, st.round, abort, a.status);
                    if (!ok) break;
                    tcgen05_fence_after();
                    if (elect_one()) {
                        const uint32_t at = st.i * (S::kStageBytes >> 4);
                        const uint32_t d = tmem + slot.i * S::kCols;
#pragma unroll
                        for (int k = 0; k < kTileK / 16; ++k) {
                            const uint64_t da = desc_a + at + k * step_a, db = desc_b + at + k * step_b;
                            const bool add = kb > kb0 || k > 0;
                            if constexpr (kMode == kPair)
                                mma_bf16_pair(d, da, db, desc, add);
                            else
                                mma_bf16(d, da, db, desc, add);
                        }
                        if constexpr (kMode == kPair)
                            mma_commit_pair(done + 8 * st.i);
                        else
                            mma_commit(done + 8 * st.i);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) {
                    if constexpr (kMode == kPair)
                        mma_commit_pair(sums + 8 * slot.i);
                    else
                        mma_commit(sums + 8 * slot.i);
                }
                __syncwarp();
            }
        }
    } else {
        // ---- results: warp = 32 rows (its quarter) and half of the columns ----
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t turn = base + S::kRingBytes + warp * kTurnBytes;
        const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t read = kMode == kPair ? cluster_map(sums_read, 0) : sums_read;
        // of out, in a chunk, and the warp's
        constexpr int kCols = kGated ? kChunk / 2 : kChunk, kMine = kGated ? S::kMine / 2 : S::kMine;
        // the second half of a chunk's sums: gated, the up half's
        constexpr int kSecond = kGated ? S::kCols / 2 : 16;
        const bool plain = !kGated && maps.plain;
        constexpr bool kWhole = kMode == kPair;
        auto release = [&](int i) {
            __syncwarp();
            tcgen05_fence_before();
            if (kMode == kPair) {
                if (lane == 0) mbar_arrive_cluster(read + 8 * i);
            } else {
                mbar_arrive_if(read + 8 * i, lane == 0);
            }
        };
        Ring<kSlots> slot;
        bool ok = true, second = false;
        for (int64_t t = t0; ok && t < tiles; t += step) {
            const Tile tile = tile_at<kMode>(t, a);
            Part part;
            part.row0 = tile.row0 + (kMode == kPair ? rank * kRows : 0) + quarter * 32;
            part.rows = static_cast<int>(min(static_cast<int64_t>(32), a.m - part.row0));
            const int64_t col0 = tile.col_tile * (2 * kMine) + half * kMine;
            Ahead ahead = {};
            if (kWhole && !kExact) read_ahead<kGated>(a, part, col0, ahead);
            if constexpr (kExact) {
                // all but the last of the tile's sums into registers, which the last ones
                // are then added to, in their place
                float acc[S::kMine / 16][16] = {};
                for (int kb = kb_first; kb < kb_end; kb += per_sum) {
                    ok = warp_wait<kMode == kPair>(sums + 8 * slot.i, slot.round, abort, a.status);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const bool last = kb + per_sum >= kb_end;
#pragma unroll
                    for (int c = 0; c < S::kMine / 16; ++c) {
                        // gated, half of each half: the columns that it writes (of a shared
                        // tile it lays out neighbouring ones)
                        const uint32_t at =
                            from + slot.i * S::kCols + 16 * c +
                            (S::kParts ? half * S::kMine
                                       : half * kMine + (16 * c >= kMine ? S::kCols / 2 - kMine : 0));
                        uint32_t v[16];
                        tmem_load16(at, v);
                        tmem_load_wait16(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            acc[c][i] += __uint_as_float(v[i]);
                            v[i] = __float_as_uint(acc[c][i]);
                        }
                        if (last) tmem_store16(at, v);
                    }
                    if (last) break;
                    release(slot.i);
                    slot.next();
                }
                if (!ok) break;
                tmem_store_wait();
                if (kWhole) read_ahead<kGated>(a, part, col0, ahead);
            } else {
                ok = warp_wait<kMode == kPair>(sums + 8 * slot.i, slot.round, abort, a.status);
                if (!ok) break;
                tcgen05_fence_after();
            }
            const uint32_t slot_at = from + slot.i * S::kCols;
            if constexpr (S::kParts) {
                const uint32_t own = base + (quarter * 32 + lane) * S::kPitch + half * S::kMine * 4;
#pragma unroll 2
                for (int c = 0; c < S::kMine; c += 16) {
                    uint32_t v[16];
                    tmem_load16(slot_at + half * S::kMine + c, v);
                    tmem_load_wait16(v);
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        store_shared_v4(own + (c + i) * 4,
                                        make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                    __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])));
                }
                break;
            } else {
                if (part.rows > 0) {
#pragma unroll 1
                    for (int c = 0; c < kMine && col0 + c < a.n; c += kCols) {
                        const uint32_t at = slot_at + half * kMine + c;
                        uint32_t v[2][16];
                        tmem_load16(at, v[0]);
                        tmem_load16(at + kSecond, v[1]);
                        tmem_load_wait16(v[0]);
                        tmem_load_wait16(v[1]);
                        if (plain) {
                            send_chunk(a, maps, turn, part, col0 + c, second, v);
                            second = !second;
                            continue;
                        }
                        turn_chunk(turn, reinterpret_cast<const float*>(v[0]),
                                   reinterpret_cast<const float*>(v[1]));
                        const Ahead now = ahead;
                        if (kWhole && c + kCols < kMine) read_ahead<kGated>(a, part, col0 + c + kCols, ahead);
                        by_width(a.n, [&](auto n) {
                            write_chunk<decltype(n)::value, kGated, kWhole>(a, turn, part, col0 + c, now);
                        });
                    }
                }
                release(slot.i);
                slot.next();
            }
        }
        if (elect_one()) bulk_wait<0>();  // what was sent has been written
        __syncwarp();
    }
    if (S::kParts) {
        // Every thread passes both barriers, whatever its CTA found to do.
        cluster_arrive();
        cluster_wait();
        if (warp < kOutWarps && t0 < tiles && load_shared(abort) == 0) {
            const Tile tile = tile_at<kMode>(t0, a);
            write_shared_tile<kMode, kGated>(a, base, tile, rank);
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    // After a wait that gave up: no copy may land once the CTA has exited, and
    // no product may run once its tensor memory is released. (Otherwise every
    // copy and product has been waited for.)
    if (load_shared(abort) != 0) {
        if (warp == kCopyWarp && lane == 0)
            mbar_drain_bounded<S::kStages>(full, fills > S::kStages ? fills - S::kStages : 0, fills - 1);
        if (warp == kProductWarp) {
            const uint32_t bar = smem_u32(&ctl.drained);
            if (elect_one()) {
                if constexpr (kMode != kPair)
                    mma_commit(bar);
                else if (rank == 0)
                    mma_commit_pair(bar);
            }
            __syncwarp();
            mbar_wait_bounded(bar, 0);
        }
    }
    if (kClusters) {  // no CTA reads this one's sums, or arrives at its barriers, any more
        cluster_arrive();
        cluster_wait();
    }
    __syncwarp();
    if (warp == kProductWarp) {
        tcgen05_fence_after();
        if constexpr (kMode == kPair)
            tmem_dealloc_pair(tmem, kTmemCols);
        else
            tmem_dealloc(tmem, kTmemCols);
    }
}

// A bf16 matrix [rows][width] of this pitch, read in boxes of box_rows x 64 with
// the 128-byte swizzle.
bool encode_map(CUtensorMap* map, const uint16_t* p, int64_t rows, int64_t width, int64_t pitch,
                int box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, rows, width, pitch * 2, box_rows, 64,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// out, written in boxes of 32 x 32.
bool encode_out(CUtensorMap* map, const LinearArgs& a) {
    return encode_2d(map,
                     a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     a.out, a.m, a.n, a.n * (a.out_f32 ? 4 : 2), 32, kChunk,
                     a.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// What a kernel's launches need beyond the defaults: its shared memory, and for narrow
// shared tiles clusters of up to 16 CTAs.
template <Mode kMode>
cudaError_t allow(void (*kern)(LinearArgs, Maps)) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(Shape<kMode>::kSmem));
    if (err != cudaSuccess || kMode != kShared) return err;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <Mode kMode, bool kGated, bool kExact>
cudaError_t launch(const LinearArgs& a, const Maps& maps, int grid, int cluster, cudaStream_t stream) {
    auto kern = linear_kernel<kMode, kGated, kExact>;
    constexpr size_t kSmem = Shape<kMode>::kSmem;
    const cudaError_t err = allow<kMode>(kern);
    if (err != cudaSuccess) return err;
    return launch_dependent_clusters(kern, grid, cluster, kThreads, kSmem, stream, a, maps);
}

template <Mode kMode>
cudaError_t launch_shared(const LinearArgs& a, const Maps& maps, bool gated, bool exact, int64_t tiles,
                          cudaStream_t stream) {
    const int grid = static_cast<int>(tiles) * a.split;
    if (exact)
        return gated ? launch<kMode, true, true>(a, maps, grid, a.split, stream)
                     : launch<kMode, false, true>(a, maps, grid, a.split, stream);
    return gated ? launch<kMode, true, false>(a, maps, grid, a.split, stream)
                 : launch<kMode, false, false>(a, maps, grid, a.split, stream);
}

// Pairs, and clusters of 2, 4, 8, 16 CTAs that share a tile (wide ones at most 8), that a device holds at a
// time: fewer than SMs / size, because a cluster's lie in one part (GPC) of it.
struct ResidentClusters {
    int pairs;
    int n[kMaxSplit + 1];
    int mid[kMaxSplit + 1];
    int wide[kMaxSplit + 1];
};

template <Mode kMode>
cudaError_t count_clusters(int size, int* n) {
    auto kern = linear_kernel<kMode, false, false>;
    constexpr size_t kSmem = Shape<kMode>::kSmem;
    const cudaError_t err = allow<kMode>(kern);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kern, &cfg);
}

cudaError_t resident_clusters(int device, ResidentClusters* clusters) {
    static PerDevice<ResidentClusters> table;
    return table.get(device, clusters, [](ResidentClusters* found) {
        cudaError_t err = count_clusters<kPair>(2, &found->pairs);
        for (int split = 2; err == cudaSuccess && split <= kMaxSplit; split *= 2)
            err = count_clusters<kShared>(split, &found->n[split]);
        for (int split = 2; err == cudaSuccess && split <= 8; split *= 2)
            err = count_clusters<kSharedMid>(split, &found->mid[split]);
        for (int split = 2; err == cudaSuccess && split <= 8; split *= 2)
            err = count_clusters<kSharedWide>(split, &found->wide[split]);
        return err;
    });
}

int64_t up(int64_t v, int64_t by) { return (v + by - 1) / by; }

// Who works on a tile, and how many CTAs share one: what takes least by a model of the
// times (us; fitted to 1231 shapes of 2 to 8000 rows, 32 to 16384 columns and k, each in
// all ways: what it takes is on average 1 % slower than the best of them, for 36 of them by
// more than 10 %, for 13 by more than 20 and at worst by 53. Those 13 have sums of 32 to 704
// products, most of them for more results than a round of CTAs makes: 3007 x 192 x 2112, 293 x
// 64 x 13120. There CTAs alone and pairs take nearly the same by the model, and not in fact). A
// block along k takes its issue or a stage's latency by the stages that are on their way, all
// of them what L2 and memory give; then come the results, by what a tile's CTAs have to join
// and by how many values of a row are stored at once. A partition's SMs may not hold a cluster.
struct Times {
    float block;      // along k
    float end, rows;  // what follows, in any tile and in one of 128 rows besides
};
constexpr Times kSharedTimes{0.17f, 0.7f, 1.5f}, kMidTimes{0.17f, 1.5f, 2.1f}, kWideTimes{0.29f, 2.0f, 3.7f};
constexpr float kAloneBlock = 0.19f, kPairBlock = 0.31f, kPairEnd = 2.1f;
constexpr float kAloneTurn = 0.25f, kPairTurn = 0.5f;  // from a tile to the next
constexpr float kWideGated = 1.0f;                     // after a gated wide tile
constexpr float kLatency = 0.89f;                      // from asking for a stage to its product
constexpr float kMemory = 8.2e6f, kL2 = 20e6f;         // bytes
struct Results {
    float narrow, pair;  // of a tile of 128 x 64 by one CTA, of a pair's
};
constexpr Results kPlainResults{0.6f, 2.3f}, kFours{1.1f, 2.6f}, kTwos{1.3f, 3.6f}, kOnes{2.5f, 5.2f};
struct Plan {
    Mode mode;
    int split;
    int clusters;  // pairs at a time
};
cudaError_t plan_for(const LinearArgs& a, bool gated, bool plain, int a_rows, int device,
                     int num_sms, bool partition, Plan* plan) {
    *plan = {kAlone, 1, 0};
    if (partition) return cudaSuccess;
    ResidentClusters clusters{};
    const cudaError_t err = resident_clusters(device, &clusters);
    if (err != cudaSuccess) return err;
    const int half = gated ? 2 : 1;
    const float a_bytes = a.a_by_k ? (a.m > 64 ? 2 : 1) * kGroupBytes : a_rows * kRowBytes;
    auto part = [&](int rows) { return a.m < rows ? static_cast<float>(a.m) / rows : 1.0f; };
    const Results results = plain ? kPlainResults : a.n % 4 == 0 ? kFours : a.n % 2 == 0 ? kTwos : kOnes;
    const float memory = 2.0f * a.k * (a.m + static_cast<float>(half) * a.n) / kMemory;
    auto tiles = [&](int cols) { return up(a.m, kRows) * up(a.n, cols / half); };
    auto from_l2 = [&](int64_t blocks, int cols) { return blocks * (a_bytes + cols * kRowBytes) / kL2; };
    float best;
    auto take = [&](float time, Plan p) {
        if (time < best) best = time, *plan = p;
    };
    // CTAs that take several tiles: a tile takes its products' time, or its results' where
    // those take longer
    auto persistent = [&](int64_t turns, float block, float result, float turn) {
        return turns * fmaxf(a.k_blocks * block, turns > 1 ? result : 0.0f) + (turns - 1) * turn;
    };
    const int64_t narrow = tiles(64);
    best = fmaxf(fmaxf(persistent(up(narrow, num_sms), kAloneBlock, results.narrow, kAloneTurn), memory),
                 from_l2(narrow * a.k_blocks, 64)) +
           results.narrow * part(kRows);
    if (clusters.pairs > 0) {
        constexpr int kRowsEach = Shape<kPair>::kTileRows;
        const int64_t n = up(a.m, kRowsEach) * up(a.n, Shape<kPair>::kCols / half);
        take(fmaxf(persistent(up(n, clusters.pairs), kPairBlock, results.pair, kPairTurn), memory) + kPairEnd +
                 results.pair * part(kRowsEach),
             {kPair, 1, clusters.pairs});
    }
    auto shared = [&](Mode mode, int split, int cols, int stages, int resident, const Times& t) {
        const int64_t n = tiles(cols), blocks = up(a.k_blocks, split);
        if (n > resident) return;
        const float in = fmaxf(blocks * fmaxf(t.block, kLatency / stages), memory);
        const float out = t.end + part(kRows) * (t.rows + results.narrow * cols / (128 * split)) +
                          (mode == kSharedWide && gated ? kWideGated : 0.0f);
        take(fmaxf(in, from_l2(n * split * blocks, cols)) + out, {mode, split, 0});
    };
    for (int n = 2; n <= kMaxSplit && n <= a.k_blocks; n *= 2) {
        shared(kShared, n, 64, Shape<kShared>::kStages, clusters.n[n], kSharedTimes);
        if (n > 8) continue;
        shared(kSharedMid, n, 128, Shape<kSharedMid>::kStages, clusters.mid[n], kMidTimes);
        shared(kSharedWide, n, 256, Shape<kSharedWide>::kStages, clusters.wide[n], kWideTimes);
    }
    return cudaSuccess;
}

// A call's way: the rule's plan, and what it went by. `epilogue`: more than rounding the sums.
struct Way {
    Plan plan;
    int a_rows;   // of a's box along k: no more than there are
    bool plain;   // out is the rounded sums, in aligned rows
    bool exact;   // sums leave tensor memory in parts
};
cudaError_t way_of(LinearArgs& a, bool epilogue, int num_sms, bool partition, Way* way) {
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    a.k_blocks = static_cast<int>(up(a.k, kTileK));
    way->a_rows = 16;
    while (way->a_rows < kRows && way->a_rows < a.m) way->a_rows *= 2;
    way->plain = !epilogue && a.act == EP_ACT_NONE && a.n % (a.out_f32 ? 4 : 8) == 0;
    if (err == cudaSuccess)
        err = plan_for(a, a.act == EP_ACT_SWIGLU, way->plain, way->a_rows, device, num_sms, partition,
                       &way->plan);
    if (err != cudaSuccess) return err;
    a.split = way->plan.split;
    const int64_t sum_blocks = up(a.k_blocks, a.split);
    way->exact = sum_blocks > kExactBlocks && (a.out_f32 || sum_blocks > kLongBlocks);
    return cudaSuccess;
}

}  // namespace

cudaError_t linear_tiles(LinearArgs a, bool epilogue, int num_sms, bool partition, LinearTiles* tiles) {
    *tiles = {EP_TILES_FEW_ROWS, 1, false};
    if (linear_few_takes(a)) return cudaSuccess;
    Way way{};
    const cudaError_t err = way_of(a, epilogue, num_sms, partition, &way);
    if (err != cudaSuccess) return err;
    switch (way.plan.mode) {
        case kAlone: tiles->kind = EP_TILES_ALONE; break;
        case kShared: tiles->kind = EP_TILES_SHARED_64; break;
        case kSharedMid: tiles->kind = EP_TILES_SHARED_128; break;
        case kSharedWide: tiles->kind = EP_TILES_SHARED_256; break;
        case kPair: tiles->kind = EP_TILES_PAIR; break;
    }
    tiles->shared_by = way.plan.mode == kPair ? 2 : way.plan.split;
    tiles->in_parts = way.exact;
    return cudaSuccess;
}

cudaError_t launch_linear(LinearArgs a, int num_sms, bool partition, cudaStream_t stream) {
    const bool gated = a.act == EP_ACT_SWIGLU;
    const int half = gated ? 2 : 1;
    if (linear_few_takes(a)) return launch_linear_few(a, stream);
    Way way{};
    const bool epilogue = a.bias != nullptr || a.z != nullptr || a.residual != nullptr;
    const cudaError_t err = way_of(a, epilogue, num_sms, partition, &way);
    if (err != cudaSuccess) return err;
    const Plan& plan = way.plan;
    const bool exact = way.exact;
    const bool pair = plan.mode == kPair;
    const int cols = pair || plan.mode == kSharedWide ? 256 : plan.mode == kSharedMid ? 128 : 64;
    a.row_tiles = up(a.m, pair ? Shape<kPair>::kTileRows : kRows);
    a.col_tiles = up(a.n, cols / half);
    Maps maps;
    maps.a_rows = pair ? kRows : way.a_rows;
    const int64_t b_rows = half * a.n;
    const bool ok =
        (a.a_by_k ? encode_map(&maps.a, a.a, a.k, a.m, a.a_pitch, kTileK)
                  : encode_map(&maps.a, a.a, a.m, a.k, a.a_pitch, maps.a_rows)) &&
        (a.b_by_k ? encode_map(&maps.b, a.b, a.k, b_rows, a.b_pitch, kTileK)
                  : encode_map(&maps.b, a.b, b_rows, a.k, a.b_pitch, gated || pair ? cols / 2 : cols));
    maps.plain = way.plain && (pair || plan.mode == kAlone);
    if (!ok || (maps.plain && !encode_out(&maps.out, a))) return cudaErrorInvalidValue;
    const int64_t tiles = a.row_tiles * a.col_tiles;
    if (pair) {
        const int grid = 2 * static_cast<int>(tiles < plan.clusters ? tiles : plan.clusters);
        if (exact)
            return gated ? launch<kPair, true, true>(a, maps, grid, 2, stream)
                         : launch<kPair, false, true>(a, maps, grid, 2, stream);
        return gated ? launch<kPair, true, false>(a, maps, grid, 2, stream)
                     : launch<kPair, false, false>(a, maps, grid, 2, stream);
    }
    if (plan.mode == kSharedMid) return launch_shared<kSharedMid>(a, maps, gated, exact, tiles, stream);
    if (plan.mode == kSharedWide) return launch_shared<kSharedWide>(a, maps, gated, exact, tiles, stream);
    if (plan.mode == kShared) return launch_shared<kShared>(a, maps, gated, exact, tiles, stream);
    const int grid = static_cast<int>(tiles < num_sms ? tiles : num_sms);
    if (exact)
        return gated ? launch<kAlone, true, true>(a, maps, grid, 1, stream)
                     : launch<kAlone, false, true>(a, maps, grid, 1, stream);
    return gated ? launch<kAlone, true, false>(a, maps, grid, 1, stream)
                 : launch<kAlone, false, false>(a, maps, grid, 1, stream);
}

}  // namespace ep
