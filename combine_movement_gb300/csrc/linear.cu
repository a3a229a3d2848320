// linear.cu -- dense products in bf16 with fp32 sums,
//
//   v[m, n] = sum_k a[m, k] * b[n, k] + bias[n]
//   out[m, n] = act(v[m, n]) + residual[m, n]
//
// (gated: b's rows are a gate half and an up half, out = silu(gate) * up +
// residual), v kept in bf16 where asked for. Each operand has its rows along k
// or (its gradients' products) runs along m or n, k by k.
//
// Mapping: a persistent grid, one CTA per SM, tiles of 128 x 256 of the output
// (gated: 128 columns of each half). Four stages of shared memory take 64
// values along k of both operands (tensor copies, 128-byte swizzle; an operand
// that runs along m or n in groups of 64 by 64); one thread issues four
// tcgen05.mma of 128 x 256 x 16 for each. A tile's sums stay in tensor memory,
// in one of two places, so that eight warps write a tile while the next one's
// products run. They read 32 columns of 32 rows at a time and turn them around in
// shared memory, so that eight lanes write 128 bytes of a row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "kernels.cuh"
#include "linear_math.cuh"
#include "per_device.cuh"
#include "product.cuh"

namespace ep {
namespace {

constexpr int kTileRows = 128;
constexpr int kBlock = 128;                  // columns of one of the tile's two blocks
constexpr int kTileCols = 2 * kBlock;
constexpr int kTileK = 64;                   // values of one stage along k
constexpr uint32_t kRowBytes = kTileK * 2;
constexpr uint32_t kGroupBytes = 64 * 128;   // 64 along k x 64 along m or n
constexpr uint32_t kStageA = kTileRows * kRowBytes;
constexpr uint32_t kStageB = kTileCols * kRowBytes;
constexpr uint32_t kStageBytes = kStageA + kStageB;
constexpr int kStages = 4;
constexpr int kSlots = 2;
constexpr int kOutWarps = 8;
constexpr int kProductWarp = kOutWarps, kCopyWarp = kOutWarps + 1;
constexpr int kThreads = (kOutWarps + 2) * 32;
constexpr uint32_t kTmemCols = kSlots * kTileCols;
constexpr int kChunk = 32;                   // columns turned around at a time
constexpr uint32_t kTurnBytes = 32 * kChunk * 4;
constexpr size_t kSmem = 1024 + kStages * kStageBytes + kOutWarps * kTurnBytes;
// A shared tile's sums, [row][column] in fp32, in the stages' place.
constexpr uint32_t kSharedPitch = kTileCols * 4 + 16;
static_assert(kTileRows * kSharedPitch <= kStages * kStageBytes, "shared sums");
constexpr int kMaxSplit = 8;
constexpr int kRowGroup = 8;                 // row tiles that share a column tile's turn

struct Maps {
    CUtensorMap a, b;
    int a_rows;                              // of a's box along m (not by_k)
};

struct Control {
    uint64_t full[kStages];       // the copies have landed
    uint64_t done[kStages];       // the stage's product is done
    uint64_t sums[kSlots];        // a tile's sums are complete
    uint64_t sums_read[kSlots];   // and have been read: the writing warps
    uint64_t drained;             // after an abort: products still in flight
    uint32_t tmem;
    int32_t abort;
};

struct Tile {
    int64_t row0, col0;
};
// Groups of kRowGroup row tiles, column tiles outside of row tiles in each: the
// tiles that run at a time share their rows of both operands.
__device__ __forceinline__ Tile tile_at(int64_t t, const LinearArgs& a) {
    const int64_t per = kRowGroup * a.col_tiles;
    const int64_t group = t / per, r0 = group * kRowGroup;
    const int64_t rows = min(static_cast<int64_t>(kRowGroup), a.row_tiles - r0);
    const int64_t i = t - group * per;
    return {(r0 + i % rows) * kTileRows, i / rows};
}

__device__ __forceinline__ float bf16_low(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_high(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// N (4 or 1) neighbouring values of a row.
template <int N>
struct Values {
    float v[N];
};
template <int N>
__device__ __forceinline__ Values<N> load_f32(const float* p) {
    Values<N> r;
    if constexpr (N == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        r.v[0] = f.x, r.v[1] = f.y, r.v[2] = f.z, r.v[3] = f.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}
template <int N>
__device__ __forceinline__ Values<N> load_bf16(const uint16_t* p) {
    Values<N> r;
    if constexpr (N == 4) {
        const uint2 f = *reinterpret_cast<const uint2*>(p);
        r.v[0] = bf16_low(f.x), r.v[1] = bf16_high(f.x), r.v[2] = bf16_low(f.y), r.v[3] = bf16_high(f.y);
    } else {
        r.v[0] = bf16_low(*p);
    }
    return r;
}
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]));
    else
        *p = __bfloat16_as_ushort(__float2bfloat16_rn(r.v[0]));
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const Values<N>& r) {
    if constexpr (N == 4)
        *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    else
        *p = r.v[0];
}

template <int N>
__device__ __forceinline__ Values<N> load_residual(const LinearArgs& a, int64_t at) {
    return a.out_f32 ? load_f32<N>(static_cast<const float*>(a.residual) + at)
                     : load_bf16<N>(static_cast<const uint16_t*>(a.residual) + at);
}

// The end of N values of out's row `row` from column `col` on: sums in `v`
// (gated: the up half's in `up`), `res` what is added.
template <int N, bool kGated>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t row, int64_t col, Values<N> v,
                                       Values<N> up, const Values<N>& res) {
    if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v.v[i] += __ldg(a.bias + col + i);
        if (kGated) {
#pragma unroll
            for (int i = 0; i < N; ++i) up.v[i] += __ldg(a.bias + a.n + col + i);
        }
    }
    if (a.z != nullptr) {
        uint16_t* z = a.z + row * (kGated ? 2 * a.n : a.n) + col;
        store_bf16<N>(z, v);
        if (kGated) store_bf16<N>(z + a.n, up);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v.v[i] = kGated ? silu(v.v[i]) * up.v[i] : activate(v.v[i], a.act);
        v.v[i] += res.v[i];
    }
    const int64_t at = row * a.n + col;
    if (a.out_f32)
        store_f32<N>(static_cast<float*>(a.out) + at, v);
    else
        store_bf16<N>(static_cast<uint16_t*>(a.out) + at, v);
}

// 16-byte piece p of row r of a warp's turning place.
__device__ __forceinline__ uint32_t turn_at(uint32_t turn, int r, int p) {
    return turn + r * (kChunk * 4) + ((p ^ (r & 7)) << 4);
}

// 32 x 32 sums from the turning place: `col` the column of the first (gated:
// of 16 of each half), `rows` how many rows are the tile's.
template <bool kGated>
__device__ __forceinline__ void write_chunk(const LinearArgs& a, uint32_t turn, int64_t row0,
                                            int rows, int64_t col) {
    constexpr int kCols = kGated ? kChunk / 2 : kChunk;  // of out
    const int lane = threadIdx.x & 31;
    if (a.n % 4 == 0) {
        constexpr int kPieces = kCols / 4, kAtOnce = 32 / kPieces, kRounds = 32 / kAtOnce;
        const int p = lane % kPieces, r0 = lane / kPieces;
        const int64_t c = col + 4 * p;
        Values<4> res[kRounds] = {};
        if (a.residual != nullptr) {
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (r0 + i * kAtOnce < rows && c < a.n)
                    res[i] = load_residual<4>(a, (row0 + r0 + i * kAtOnce) * a.n + c);
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = r0 + i * kAtOnce;
            if (r >= rows || c >= a.n) continue;
            const float4 f = load_shared_v4(turn_at(turn, r, p));
            const float4 u = kGated ? load_shared_v4(turn_at(turn, r, p + kPieces)) : f;
            finish<4, kGated>(a, row0 + r, c, {{f.x, f.y, f.z, f.w}}, {{u.x, u.y, u.z, u.w}}, res[i]);
        }
    } else {  // rows that do not start on 16 bytes: value by value
        constexpr int kAtOnce = 32 / kCols;
        const int cl = lane % kCols;
        const int64_t c = col + cl;
        for (int r = lane / kCols; r < rows; r += kAtOnce) {
            if (c >= a.n) break;
            Values<1> res = {};
            if (a.residual != nullptr) res = load_residual<1>(a, (row0 + r) * a.n + c);
            const float f = load_shared_f32(turn_at(turn, r, cl / 4) + cl % 4 * 4);
            const float u =
                kGated ? load_shared_f32(turn_at(turn, r, (cl + kCols) / 4) + cl % 4 * 4) : f;
            finish<1, kGated>(a, row0 + r, c, {{f}}, {{u}}, res);
        }
    }
}

// The sums of a tile that the cluster's CTAs took parts of k of: each has laid
// its own out in shared memory; CTA `rank` adds, in the parts' order, and writes
// those of the rows r = rank mod split.
template <int N, bool kGated>
__device__ __forceinline__ void write_shared_tile(const LinearArgs& a, uint32_t sums, const Tile& tile,
                                                  int rank) {
    constexpr int kCols = kGated ? kBlock : kTileCols, kPieces = kCols / N;
    const int64_t left = a.m - tile.row0;
    const int rows = static_cast<int>(left < kTileRows ? left : kTileRows);
    const int pieces = (rows + a.split - 1 - rank) / a.split * kPieces;
    const int64_t col0 = tile.col0 * kCols;
    for (int i = threadIdx.x; i < pieces; i += kOutWarps * 32) {
        const int r = i / kPieces * a.split + rank, c = i % kPieces * N;
        if (col0 + c >= a.n) continue;
        const int64_t row = tile.row0 + r, col = col0 + c;
        Values<N> res = {}, v = {}, up = {};
        if (a.residual != nullptr) res = load_residual<N>(a, row * a.n + col);
        const uint32_t at = sums + r * kSharedPitch + c * 4;
        for (int p = 0; p < a.split; ++p) {
            const uint32_t from = cluster_map(at, p);
            if constexpr (N == 4) {
                const float4 f = load_cluster_v4(from);
                v.v[0] += f.x, v.v[1] += f.y, v.v[2] += f.z, v.v[3] += f.w;
                if (kGated) {
                    const float4 u = load_cluster_v4(from + kBlock * 4);
                    up.v[0] += u.x, up.v[1] += u.y, up.v[2] += u.z, up.v[3] += u.w;
                }
            } else {
                v.v[0] += load_cluster_f32(from);
                if (kGated) up.v[0] += load_cluster_f32(from + kBlock * 4);
            }
        }
        finish<N, kGated>(a, row, col, v, up, res);
    }
}

// kSplit: a tile's blocks along k go to the CTAs of a cluster, a tile to a
// cluster; else a CTA takes whole tiles, one after the other.
template <bool kGated, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const LinearArgs a, const __grid_constant__ Maps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // the swizzle's period
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(ctl.full), done = smem_u32(ctl.done);
    const uint32_t sums = smem_u32(ctl.sums), sums_read = smem_u32(ctl.sums_read);
    const uint32_t abort = smem_u32(&ctl.abort);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(sums + 8 * i, 1);
            mbar_init(sums_read + 8 * i, kOutWarps);
        }
        mbar_init(smem_u32(&ctl.drained), 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == kProductWarp) tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensor_map(&maps.a);
        prefetch_tensor_map(&maps.b);
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = ctl.tmem;
    const int64_t tiles = a.row_tiles * a.col_tiles;
    const int split = kSplit ? a.split : 1;
    const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
    const int64_t t0 = kSplit ? blockIdx.x / split : blockIdx.x;
    const int64_t step = kSplit ? tiles : gridDim.x;
    const int kb_first = static_cast<int>(static_cast<int64_t>(a.k_blocks) * rank / split);
    const int kb_end = static_cast<int>(static_cast<int64_t>(a.k_blocks) * (rank + 1) / split);
    int64_t fills = 0;  // stages filled so far (the copying warp's)

    if (warp == kCopyWarp) {
        // ---- copies: one lane fills the stages in order ----
        const int a_groups = a.m > 64 ? 2 : 1;
        const uint32_t bytes =
            kStageB + (a.a_by_k ? a_groups * kGroupBytes : static_cast<uint32_t>(maps.a_rows) * kRowBytes);
        Ring<kStages> st;
        bool ok = true;
        for (int64_t t = t0; ok && t < tiles; t += step) {
            const Tile tile = tile_at(t, a);
            const int row0 = static_cast<int>(tile.row0);
            const int col0 = static_cast<int>(tile.col0) * (kGated ? kBlock : kTileCols);
            const int col1 = kGated ? static_cast<int>(a.n) + col0 : col0 + kBlock;
            for (int kb = kb_first; kb < kb_end; ++kb, st.next(), ++fills) {
                ok = warp_wait(done + 8 * st.i, st.round ^ 1u, abort, a.status);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t dst_a = base + st.i * kStageBytes, dst_b = dst_a + kStageA;
                    const uint32_t bar = full + 8 * st.i;
                    const int k = kb * kTileK;
                    mbar_arrive_expect_tx(bar, bytes);
                    if (a.a_by_k) {
                        for (int g = 0; g < a_groups; ++g)
                            tensor_load_2d(dst_a + g * kGroupBytes, &maps.a, row0 + 64 * g, k, bar);
                    } else {
                        tensor_load_2d(dst_a, &maps.a, k, row0, bar);
                    }
                    if (a.b_by_k) {
                        for (int g = 0; g < kTileCols / 64; ++g)
                            tensor_load_2d(dst_b + g * kGroupBytes, &maps.b, col0 + 64 * g, k, bar);
                    } else {
                        tensor_load_2d(dst_b, &maps.b, k, col0, bar);
                        tensor_load_2d(dst_b + kBlock * kRowBytes, &maps.b, k, col1, bar);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == kProductWarp) {
        // ---- products: one lane ----
        const uint32_t desc = mma_desc_bf16(kTileRows, kTileCols, a.a_by_k, a.b_by_k);
        const uint64_t desc_a = a.a_by_k ? operand_desc_by_k(base) : operand_desc(base);
        const uint64_t desc_b =
            a.b_by_k ? operand_desc_by_k(base + kStageA) : operand_desc(base + kStageA);
        const uint32_t step_a = (a.a_by_k ? 2048 : 32) >> 4, step_b = (a.b_by_k ? 2048 : 32) >> 4;
        Ring<kStages> st;
        Ring<kSlots> slot;
        bool ok = true;
        for (int64_t t = t0; ok && t < tiles; t += step, slot.next()) {
            ok = warp_wait(sums_read + 8 * slot.i, slot.round ^ 1u, abort, a.status);
            if (!ok) break;
            tcgen05_fence_after();
            for (int kb = kb_first; kb < kb_end; ++kb, st.next()) {
                ok = warp_wait(full + 8 * st.i, st.round, abort, a.status);
                if (!ok) break;
                tcgen05_fence_after();
                if (elect_one()) {
                    const uint32_t at = st.i * (kStageBytes >> 4);
#pragma unroll
                    for (int k = 0; k < kTileK / 16; ++k)
                        mma_bf16(tmem + slot.i * kTileCols, desc_a + at + k * step_a,
                                 desc_b + at + k * step_b, desc, kb > kb_first || k > 0);
                    mma_commit(done + 8 * st.i);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) mma_commit(sums + 8 * slot.i);
            __syncwarp();
        }
    } else {
        // ---- results: warp = 32 rows (its quarter) and half of the columns ----
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t turn = base + kStages * kStageBytes + warp * kTurnBytes;
        const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        Ring<kSlots> slot;
        bool ok = true;
        for (int64_t t = t0; ok && t < tiles; t += step, slot.next()) {
            const Tile tile = tile_at(t, a);
            ok = warp_wait(sums + 8 * slot.i, slot.round, abort, a.status);
            if (!ok) break;
            tcgen05_fence_after();
            const uint32_t slot_at = from + slot.i * kTileCols;
            if (kSplit) {
                const uint32_t own = base + (quarter * 32 + lane) * kSharedPitch + half * kBlock * 4;
#pragma unroll 1
                for (int c = 0; c < kBlock; c += 16) {
                    uint32_t v[16];
                    tmem_load16(slot_at + half * kBlock + c, v);
                    tmem_load_wait16(v);
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        store_shared_v4(own + (c + i) * 4,
                                        make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                    __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])));
                }
                break;
            }
            const int64_t row0 = tile.row0 + quarter * 32;
            const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.m - row0));
            constexpr int kCols = kGated ? kChunk / 2 : kChunk;     // of out, in a chunk
            constexpr int kMine = kGated ? kBlock / 2 : kBlock;     // of out, the warp's
            const int64_t col0 = tile.col0 * (2 * kMine) + half * kMine;
            if (rows > 0) {
#pragma unroll 1
                for (int c = 0; c < kMine && col0 + c < a.n; c += kCols) {
                    const uint32_t at = slot_at + half * kMine + c;
                    uint32_t v[2][16];
                    tmem_load16(at, v[0]);
                    tmem_load16(at + (kGated ? kBlock : 16), v[1]);
                    tmem_load_wait16(v[0]);
                    tmem_load_wait16(v[1]);
                    __syncwarp();  // the chunk before has been read
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            store_shared_v4(turn_at(turn, lane, h * 4 + i / 4),
                                            make_float4(__uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1]),
                                                        __uint_as_float(v[h][i + 2]),
                                                        __uint_as_float(v[h][i + 3])));
                    __syncwarp();
                    write_chunk<kGated>(a, turn, row0, rows, col0 + c);
                }
            }
            __syncwarp();
            tcgen05_fence_before();
            mbar_arrive_if(sums_read + 8 * slot.i, lane == 0);
        }
    }
    if (kSplit) {
        // Every thread passes both barriers, whatever its CTA found to do.
        cluster_arrive();
        cluster_wait();
        if (warp < kOutWarps && t0 < tiles && load_shared(abort) == 0) {
            const Tile tile = tile_at(t0, a);
            if (a.n % 4 == 0)
                write_shared_tile<4, kGated>(a, base, tile, rank);
            else
                write_shared_tile<1, kGated>(a, base, tile, rank);
        }
        cluster_arrive();
        cluster_wait();  // no CTA reads this one's sums any more
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    // After a wait that gave up: no copy may land once the CTA has exited, and
    // no product may run once its tensor memory is released. (Otherwise every
    // copy and product has been waited for.)
    if (load_shared(abort) != 0) {
        if (warp == kCopyWarp && lane == 0)
            mbar_drain_bounded<kStages>(full, fills > kStages ? fills - kStages : 0, fills - 1);
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

// A bf16 matrix [rows][width] of this pitch, read in boxes of box_rows x 64 with
// the 128-byte swizzle.
bool encode_map(CUtensorMap* map, const uint16_t* p, int64_t rows, int64_t width, int64_t pitch,
                int box_rows) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p), dims, strides, box,
              step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kGated, bool kSplit>
cudaError_t launch(const LinearArgs& a, const Maps& maps, int grid, cudaStream_t stream) {
    auto kern = linear_kernel<kGated, kSplit>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    return launch_dependent_clusters(kern, grid, a.split, kThreads, kSmem, stream, a, maps);
}

// Clusters of 2, 4, 8 CTAs that a device holds at a time: fewer than SMs / size,
// because a cluster's lie in one part (GPC) of it.
struct ResidentClusters {
    int n[kMaxSplit + 1];
};

cudaError_t resident_clusters(int device, ResidentClusters* clusters) {
    static PerDevice<ResidentClusters> table;
    return table.get(device, clusters, [](ResidentClusters* found) {
        auto kern = linear_kernel<false, true>;
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmem));
        for (int split = 2; err == cudaSuccess && split <= kMaxSplit; split *= 2) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(split));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmem;
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

// CTAs to share a tile's blocks along k, where the tiles leave SMs idle. A
// partition's SMs may not hold a cluster.
cudaError_t split_for(const LinearArgs& a, int device, int num_sms, bool partition, int* split) {
    *split = 1;
    const int64_t tiles = a.row_tiles * a.col_tiles;
    if (partition || 2 * tiles > num_sms) return cudaSuccess;
    ResidentClusters clusters{};
    const cudaError_t err = resident_clusters(device, &clusters);
    if (err != cudaSuccess) return err;
    int n = 1;
    while (n < kMaxSplit && tiles <= clusters.n[2 * n] && a.k_blocks >= 4 * n) n *= 2;
    *split = n;
    return cudaSuccess;
}

}  // namespace

int64_t linear_tiles(int64_t m, int64_t n, bool gated) {
    const int cols = gated ? kBlock : kTileCols;
    return ((m + kTileRows - 1) / kTileRows) * ((n + cols - 1) / cols);
}

cudaError_t launch_linear(LinearArgs a, int num_sms, bool partition, cudaStream_t stream) {
    const bool gated = a.act == EP_ACT_SWIGLU;
    const int cols = gated ? kBlock : kTileCols;
    a.k_blocks = static_cast<int>((a.k + kTileK - 1) / kTileK);
    a.row_tiles = (a.m + kTileRows - 1) / kTileRows;
    a.col_tiles = (a.n + cols - 1) / cols;
    Maps maps;
    maps.a_rows = 16;  // no more than there are
    while (maps.a_rows < kTileRows && maps.a_rows < a.m) maps.a_rows *= 2;
    const int64_t b_rows = gated ? 2 * a.n : a.n;
    const bool ok =
        (a.a_by_k ? encode_map(&maps.a, a.a, a.k, a.m, a.a_pitch, kTileK)
                  : encode_map(&maps.a, a.a, a.m, a.k, a.a_pitch, maps.a_rows)) &&
        (a.b_by_k ? encode_map(&maps.b, a.b, a.k, b_rows, a.b_pitch, kTileK)
                  : encode_map(&maps.b, a.b, b_rows, a.k, a.b_pitch, kBlock));
    if (!ok) return cudaErrorInvalidValue;
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err == cudaSuccess) err = split_for(a, device, num_sms, partition, &a.split);
    if (err != cudaSuccess) return err;
    const int64_t tiles = a.row_tiles * a.col_tiles;
    const int grid = static_cast<int>(a.split > 1 ? tiles * a.split : tiles < num_sms ? tiles : num_sms);
    if (a.split > 1)
        return gated ? launch<true, true>(a, maps, grid, stream) : launch<false, true>(a, maps, grid, stream);
    return gated ? launch<true, false>(a, maps, grid, stream) : launch<false, false>(a, maps, grid, stream);
}

}  // namespace ep
