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
// Mapping: a persistent grid, one CTA per SM. A tile is 128 rows of one
// expert times two blocks of 128 weight rows (neighbours; for the gated form
// block j of the gate half and block j of the up half, so that the tile holds
// a whole quantisation block of h). Per 128 values along K one stage of
// shared memory takes the operands (tensor copies, 128-byte swizzle) and four
// tcgen05.mma of 128 x 256 x 32 leave that block's plain sums in one of two
// halves of tensor memory. The scales differ between rows and between blocks
// along K, so they cannot ride in the tensor core's sum: eight warps read each
// block's sums back and add them, scaled, into fp32 registers (a thread holds
// 64 + 64 columns of one row), while the tensor core works on the next
// block. One warp issues the copies, one the products, one the scales' copies.
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/ep.h"
#include "combine_math.cuh"
#include "fp8_math.cuh"
#include "kernels.cuh"
#include "tcgen05.cuh"

namespace ep {
namespace {

constexpr int kTileRows = 128;
constexpr int kTileK = 128;                    // bytes and values of one stage row
constexpr int kTileCols = 2 * kFp8Block;       // weight rows of a tile
constexpr uint32_t kStageA = kTileRows * kTileK;
constexpr uint32_t kStageB = kTileCols * kTileK;
constexpr uint32_t kStageBytes = kStageA + kStageB;
constexpr int kStages = 4;
constexpr int kAccWarps = 8;
constexpr int kCopyWarp = kAccWarps, kProductWarp = kAccWarps + 1, kScaleWarp = kAccWarps + 2;
constexpr int kThreads = (kAccWarps + 3) * 32;
constexpr uint32_t kTmemCols = 512;            // two halves of 256 columns
constexpr int kRowBoxes = 4;                   // row boxes of 16, 32, 64, 128

// Scales of one stage: of the tile's 128 rows, then of its two weight blocks.
// The scales of fill i overwrite those of fill i - kScaleSlots. A stage is
// refilled once its product is done (fill i - kStages), and that product
// began after the sums of fill i - kStages - 2 were read, with their scales:
// so kStages + 2 slots suffice.
constexpr int kScaleSlots = 8;
static_assert(kScaleSlots >= kStages + 2, "scales in use would be overwritten");

struct Maps {
    CUtensorMap rows[kRowBoxes];
    CUtensorMap weights;
};

struct Control {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t sums_full[2];
    uint64_t sums_empty[2];
    uint64_t joined;       // accumulating warps, once per tile
    uint64_t drained;      // after an abort: products still in flight
    uint32_t tmem;
    int32_t abort;
    int32_t warp_sum[32];
    uint32_t amax[2][2][kTileRows];
    float row_scale[kScaleSlots][kTileRows];
    float weight_scale[kScaleSlots][2];
};

// Wait on a barrier; false once it gave up after kWaitLimitNs or another
// warp did.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                              int32_t* status) {
    if (mbar_try_wait(bar, parity)) return true;
    for (int i = 0; i < 64; ++i)  // the timer is slow to read
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort != 0) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            set_status(status, EP_ERR_TIMEOUT);
            return false;
        }
    }
}

// One tile: 128 rows of an expert times two blocks of its weight rows.
struct Tile {
    int expert;
    int col_tile;
    int row0;   // first row
    int rows;   // valid rows, 1 .. 128
};

// The tiles of expert e are [cum[e], cum[e + 1]) * col_tiles, row tiles
// innermost: tiles that read the same weights run at the same time.
__device__ __forceinline__ Tile find_tile(int64_t t, const int32_t* cum, const ExpertArgs& a) {
    int lo = 0, hi = a.E;  // cum[lo] * col_tiles <= t < cum[hi] * col_tiles
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(cum[mid]) * a.col_tiles <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int row_tiles = cum[lo + 1] - cum[lo];
    const uint32_t local = static_cast<uint32_t>(t - static_cast<int64_t>(cum[lo]) * a.col_tiles);
    Tile tile;
    tile.expert = lo;
    tile.col_tile = static_cast<int>(local / row_tiles);
    const int rt = static_cast<int>(local - static_cast<uint32_t>(tile.col_tile) * row_tiles);
    const int begin = __ldg(a.offsets + lo), end = __ldg(a.offsets + lo + 1);
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

template <bool kGateUp>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const ExpertArgs a, const __grid_constant__ Maps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;
    // stages on a 1024-byte boundary (the swizzle's period), then cum[E + 1]
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int32_t* cum = reinterpret_cast<int32_t*>(smem_raw + (base - smem_u32(smem_raw)) +
                                              kStages * kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(ctl.full), empty = smem_u32(ctl.empty);
    const uint32_t sums_full = smem_u32(ctl.sums_full), sums_empty = smem_u32(ctl.sums_empty);
    const uint32_t joined = smem_u32(&ctl.joined);
    volatile int32_t* abort = &ctl.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1 + 32);  // the copies' bytes, the scale warp's lanes
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sums_full + 8 * i, 1);
            mbar_init(sums_empty + 8 * i, kAccWarps);
        }
        mbar_init(joined, kAccWarps);
        mbar_init(smem_u32(&ctl.drained), 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == kProductWarp) tmem_alloc(smem_u32(&ctl.tmem), kTmemCols);
    if (warp == kCopyWarp && lane == 0) {
        for (int i = 0; i < kRowBoxes; ++i) prefetch_tensor_map(&maps.rows[i]);
        prefetch_tensor_map(&maps.weights);
    }
    griddep_wait();
    griddep_launch_dependents();

    // cum[e] = row tiles of the experts before e
    {
        const int per = (a.E + kThreads - 1) / kThreads;
        const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
        int mine = 0;
        for (int e = e0; e < e1; ++e) mine += (expert_rows(e, a) + kTileRows - 1) / kTileRows;
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) ctl.warp_sum[warp] = incl;
        __syncthreads();
        int run = incl - mine;
        for (int w = 0; w < warp; ++w) run += ctl.warp_sum[w];
        for (int e = e0; e < e1; ++e) {
            cum[e] = run;
            run += (expert_rows(e, a) + kTileRows - 1) / kTileRows;
        }
        if (threadIdx.x == kThreads - 1) cum[a.E] = run;
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = ctl.tmem;
    const int64_t tiles = static_cast<int64_t>(cum[a.E]) * a.col_tiles;
    const int kb_count = a.k_blocks;
    int64_t fills = 0;  // stages filled so far (the copying lane's)

    if (warp == kCopyWarp) {
        // ---- copies: one lane fills the stages in order ----
        if (lane == 0) {
            const uint64_t keep = policy_evict_last(), stream = policy_evict_normal();
            int64_t it = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile tile = find_tile(t, cum, a);
                const int box = tile.rows > 64 ? 3 : tile.rows > 32 ? 2 : tile.rows > 16 ? 1 : 0;
                const uint32_t bytes = (16u << box) * kTileK + kStageB;
                const int w0 = tile.expert * a.n + tile.col_tile * (kGateUp ? kFp8Block : kTileCols);
                const int w1 = w0 + (kGateUp ? a.n / 2 : kFp8Block);
                for (int kb = 0; kb < kb_count; ++kb, ++it) {
                    const uint32_t s = static_cast<uint32_t>(it % kStages);
                    ok = wait_or_abort(empty + 8 * s, static_cast<uint32_t>((it / kStages) & 1) ^ 1u,
                                       abort, a.status);
                    if (!ok) break;
                    const uint32_t dst = base + s * kStageBytes, bar = full + 8 * s;
                    mbar_arrive_expect_tx(bar, bytes);
                    tensor_load_2d(dst, &maps.rows[box], kb * kTileK, tile.row0, bar, keep);
                    tensor_load_2d(dst + kStageA, &maps.weights, kb * kTileK, w0, bar, stream);
                    tensor_load_2d(dst + kStageA + kStageB / 2, &maps.weights, kb * kTileK, w1, bar,
                                   stream);
                }
            }
            fills = it;
        }
    } else if (warp == kProductWarp) {
        // ---- products: one lane ----
        if (lane == 0) {
            constexpr uint32_t kDesc = mma_desc_e4m3(kTileRows, kTileCols);
            int64_t it = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                for (int kb = 0; kb < kb_count; ++kb, ++it) {
                    const uint32_t s = static_cast<uint32_t>(it % kStages), half = it & 1;
                    ok = wait_or_abort(sums_empty + 8 * half, static_cast<uint32_t>((it >> 1) & 1) ^ 1u,
                                       abort, a.status) &&
                         wait_or_abort(full + 8 * s, static_cast<uint32_t>((it / kStages) & 1), abort,
                                       a.status);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint64_t da = operand_desc(base + s * kStageBytes);
                    const uint64_t db = operand_desc(base + s * kStageBytes + kStageA);
#pragma unroll
                    for (int k = 0; k < kTileK / 32; ++k)
                        mma_e4m3(tmem + half * kTileCols, da + 2 * k, db + 2 * k, kDesc, k > 0);
                    mma_commit(empty + 8 * s);
                    mma_commit(sums_full + 8 * half);
                }
            }
        }
    } else if (warp == kScaleWarp) {
        // ---- scales: small copies that arrive on the stage's barrier too ----
        const int n_blocks = (a.n + kFp8Block - 1) / kFp8Block;
        int64_t it = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tile = find_tile(t, cum, a);
            const int b0 = kGateUp ? tile.col_tile : 2 * tile.col_tile;
            const int b1 = kGateUp ? b0 + n_blocks / 2 : min(b0 + 1, n_blocks - 1);
            const float* row[kTileRows / 32];
#pragma unroll
            for (int i = 0; i < kTileRows / 32; ++i)
                row[i] = a.a_scale +
                         static_cast<int64_t>(tile.row0 + min(i * 32 + lane, tile.rows - 1)) * kb_count;
            const float* weight =
                a.w_scale +
                (static_cast<int64_t>(tile.expert) * n_blocks + (lane == 0 ? b0 : b1)) * kb_count;
            for (int kb = 0; kb < kb_count; ++kb, ++it) {
                const uint32_t s = static_cast<uint32_t>(it % kStages), slot = it % kScaleSlots;
                ok = wait_or_abort(empty + 8 * s, static_cast<uint32_t>((it / kStages) & 1) ^ 1u, abort,
                                   a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < kTileRows / 32; ++i)
                    if (i * 32 < tile.rows)
                        copy_async4(smem_u32(&ctl.row_scale[slot][i * 32 + lane]), row[i] + kb);
                if (lane < 2) copy_async4(smem_u32(&ctl.weight_scale[slot][lane]), weight + kb);
                copy_async_arrive(full + 8 * s);
            }
        }
        copy_async_wait_all();
    } else {
        // ---- scaled sums: thread = one row, columns [64 h, 64 h + 64) of both blocks ----
        const int h = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t sums = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + h * 64;
        int64_t it = 0;
        uint32_t tile_no = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++tile_no) {
            const Tile tile = find_tile(t, cum, a);
            const bool live = quarter * 32 < tile.rows;  // warp-uniform
            const int64_t grow = tile.row0 + row;
            uint64_t acc[2][32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i] = 0ull;
            for (int kb = 0; kb < kb_count; ++kb, ++it) {
                const uint32_t half = it & 1, slot = it % kScaleSlots;
                ok = wait_or_abort(sums_full + 8 * half, static_cast<uint32_t>((it >> 1) & 1), abort,
                                   a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tcgen05_fence_after();
                if (live) {
                    const uint32_t src = sums + half * kTileCols;
                    const float sa = ctl.row_scale[slot][row];
                    const float s0 = sa * ctl.weight_scale[slot][0];
                    const float s1 = sa * ctl.weight_scale[slot][1];
                    uint64_t s2[2];
                    asm("mov.b64 %0, {%1, %1};" : "=l"(s2[0]) : "f"(s0));
                    asm("mov.b64 %0, {%1, %1};" : "=l"(s2[1]) : "f"(s1));
                    uint32_t v[2][16];
                    tmem_load16(src, v[0]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        tmem_load_wait16(v[c & 1]);
                        if (c < 7)
                            tmem_load16(src + ((c + 1) >> 2) * kFp8Block + ((c + 1) & 3) * 16,
                                        v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint64_t d;
                            asm("mov.b64 %0, {%1, %2};"
                                : "=l"(d)
                                : "r"(v[c & 1][2 * i]), "r"(v[c & 1][2 * i + 1]));
                            asm("fma.rn.f32x2 %0, %1, %2, %0;"
                                : "+l"(acc[c >> 2][(c & 3) * 8 + i])
                                : "l"(d), "l"(s2[c >> 2]));
                        }
                    }
                    tcgen05_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sums_empty + 8 * half);
            }
            if (!ok) break;
            const bool store = row < tile.rows;
            if (kGateUp) {
                float v[64];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float g[2], u[2];
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(g[0]), "=f"(g[1]) : "l"(acc[0][i]));
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(u[0]), "=f"(u[1]) : "l"(acc[1][i]));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float y = g[j] / (1.0f + expf(-g[j])) * u[j];
                        v[2 * i + j] = y;
                        top = max(top, abs_bits(y));
                    }
                }
                // the block's other 64 columns are in the other half's warps
                uint32_t* amax = &ctl.amax[tile_no & 1][0][0];
                amax[h * kTileRows + row] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = wait_or_abort(joined, tile_no & 1, abort, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                top = max(top, amax[(h ^ 1) * kTileRows + row]);
                const BlockScale bs = block_scale(top);
                if (store) {
                    const int width = a.n / 2;
                    uint8_t* q = a.out_q + grow * width + tile.col_tile * kFp8Block + h * 64;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* f = v + i * 16 + j * 4;
                            p[j] = pack_e4m3x4(f[0] * bs.inverse, f[1] * bs.inverse,
                                               f[2] * bs.inverse, f[3] * bs.inverse);
                        }
                        st_v4(q + i * 16, make_uint4(p[0], p[1], p[2], p[3]));
                    }
                    if (h == 0) a.out_scale[grow * (width / kFp8Block) + tile.col_tile] = bs.scale;
                }
            } else if (store) {
                const int64_t col0 = static_cast<int64_t>(tile.col_tile) * kTileCols + h * 64;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t col = col0 + b * kFp8Block + i * 8;
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float lo, hi;
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc[b][i * 4 + j]));
                            p[j] = pack_bf16x2(lo, hi);
                        }
                        if (col < a.n)
                            st_v4(a.out + grow * a.n + col, make_uint4(p[0], p[1], p[2], p[3]));
                    }
            }
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    // After a wait that gave up: no copy may land once the CTA has exited, and
    // no product may run once its tensor memory is released. (Otherwise every
    // copy and product has been waited for.)
    if (*abort != 0) {
        if (warp == kCopyWarp && lane == 0)
            mbar_drain_bounded<kStages>(full, fills > kStages ? fills - kStages : 0, fills - 1);
        if (warp == kProductWarp && lane == 0) {
            mma_commit(smem_u32(&ctl.drained));
            mbar_wait_bounded(smem_u32(&ctl.drained), 0);
        }
        __syncwarp();
    }
    if (warp == kProductWarp) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeFn>(nullptr);
        return reinterpret_cast<EncodeFn>(p);
    }();
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

}  // namespace

cudaError_t launch_expert(ExpertArgs a, int num_sms, cudaStream_t stream) {
    const bool gated = a.out_q != nullptr;
    a.k_blocks = static_cast<int>((a.k + kFp8Block - 1) / kFp8Block);
    a.col_tiles = gated ? a.n / 2 / kFp8Block : (a.n + kTileCols - 1) / kTileCols;
    Maps maps;
    for (int i = 0; i < kRowBoxes; ++i)
        if (!encode_map(&maps.rows[i], a.a, a.num_recv, a.k, 16 << i)) return cudaErrorInvalidValue;
    if (!encode_map(&maps.weights, a.w, static_cast<int64_t>(a.E) * a.n, a.k, kFp8Block))
        return cudaErrorInvalidValue;
    // at most this many tiles, whatever the offsets say
    const int64_t row_tiles =
        a.num_recv / kTileRows + (a.num_recv < a.E ? a.num_recv : static_cast<int64_t>(a.E));
    const int64_t most = row_tiles * a.col_tiles;
    const int grid = static_cast<int>(most < num_sms ? most : num_sms);
    const size_t smem = 1024 + kStages * kStageBytes + sizeof(int32_t) * (a.E + 1);
    auto kern = gated ? expert_kernel<true> : expert_kernel<false>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_dependent(kern, grid, kThreads, smem, stream, a, maps);
}

}  // namespace ep
