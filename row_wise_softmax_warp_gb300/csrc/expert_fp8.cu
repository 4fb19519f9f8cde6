// expert_fp8.cu - the experts' product on e4m3 operands with a scale for each
// block of 128 (tcgen05, clusters of two CTAs).
//
//   y[s][n] = sum_b xs[s][b] ws[e][n / 128][b] P_b,  P_b = sum_{k in block b} xq[s][k] wq[e][n][k]
//
// A cluster computes up to 256 rows of a group (128 a CTA) by 128 output columns;
// a stage of 128 bytes along the sum is one block.  Warps 8, 9 and 10 copy, issue
// products and prepare scales, otherwise as in expert_matmul.cu.  The tensor cores
// add up P_b alone; what they cannot do is the pair of scales, which differs from
// block to block.  So each block's products go to one of four tensor-memory
// buffers, and eight warps a CTA add scale * P_b to sums that stay in registers (64
// a thread) while the next blocks' products run into the others.
//
// Rows lie on the lanes of tensor memory here (in expert_matmul.cu the output
// columns do): a thread's sums then share one scale, read once a block.  With the
// rows along the columns every value needs its own scale from shared memory, 1024
// clocks of its bandwidth a block of 256 x 256 against the 512 clocks of the
// products: that way measured 788 TFLOP/s (16384 x 4096 x 4096).  A row tile is
// 256 rows whatever the group; groups of fewer rows copy only what they have.
//
// What bounds it: a block takes 0.20 us (some 400 clocks) where its products take 256,
// and each tile 1.2 to 1.6 us on top, in which the eight warps write their sums and add
// nothing while the products run only four blocks ahead (from 8192 rows, 768 and 1536 ->
// 2048: 22 and 30 us in 7 rounds of tiles; 16384 rows, 1024, 2048 and 4096 -> 4096: 77, 120
// and 210 us in 27).  Sums of 768 are six blocks, so more than half of their time is
// that fixed part: 32 rows of 64 experts take as long as in bf16.  Within a block, a
// buffer's way from the products to the adding warps and back takes about 1300 clocks,
// most of them looks at barriers in shared memory, which the operands keep busy.  Two
// buffers of 256 columns cover less of that way than four of 128 (1970 against 2150
// TFLOP/s when that was chosen), though
// these read the rows' operand twice as often.  Scales read one by one instead of
// four at once cost 6%.
#include <cuda_fp8.h>

#include "groups.cuh"
#include "row_store.cuh"
#include "tensor_core.cuh"
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kBlock = 128;                  // values of the sum per scale, and per stage
constexpr int kTileRows = 256, kTileCols = 128;
constexpr int kStages = 6;
constexpr uint32_t kXBytes = 128 * 128, kWBytes = 64 * 128;  // a CTA's share of a stage
constexpr uint32_t kStageBytes = kXBytes + kWBytes;
constexpr int kBuffers = 4;                  // of a block's products in tensor memory
constexpr int kScaleSlots = 3;               // of the scales of kAhead blocks
constexpr int kAhead = 4;
constexpr int kAddWarps = 8;
constexpr int kWarpColumns = kTileCols / (kAddWarps / 4);  // columns that an adding warp holds
constexpr int kCopyWarp = 8, kProductWarp = 9, kScaleWarp = 10;
constexpr int kThreads = 384;  // 168 registers a thread
constexpr uint32_t kTmemColumns = 512;

struct Fp8Args {
    CUtensorMap x;        // boxes of 64 rows
    CUtensorMap x_small;  // boxes of 16 rows
    CUtensorMap w;        // boxes of 64 output columns
    const float* xs;
    const float* ws;
    const int32_t* offsets;
    void* y;
    int slots, experts;
    int in, out;
    bool vec;        // rows of y allow 16-byte stores
    bool scale_vec;  // rows of scales allow 16-byte loads
};

struct Fp8Shared {
    float scale[kScaleSlots][kAhead][128];  // of this CTA's rows
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[kBuffers], acc_empty[kBuffers], peer_empty[kBuffers];
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    int warp_tiles[kThreads / 32];
    uint32_t tmem;
    int abort;
};

struct Fp8Tile {
    int expert = 0;
    int row0, rows;  // of the pair
    int col0;
};

__device__ __forceinline__ bool tile_at(const Fp8Args& g, const int* table, int t, int tiles, Fp8Tile& w) {
    if (t >= tiles) return false;
    const int across = (g.out + kTileCols - 1) / kTileCols;
    const int row = t / across;
    w.expert = uniform(tile_expert(table, g.experts, row, w.expert));
    const RowRange r = group_rows(g.offsets, w.expert, g.slots);
    const int at = (row - table[w.expert]) * kTileRows;
    w.row0 = uniform(r.first + at);
    w.rows = uniform(min(kTileRows, r.count - at));
    w.col0 = t % across * kTileCols;
    return true;
}

// Rows of the tile that CTA `rank` copies: its share in whole boxes of 16.
__device__ __forceinline__ int rows_of(const Fp8Tile& w, int rank) {
    return min(128, (max(0, w.rows - rank * 128) + 15) & ~15);
}

// acc += s * p, two at a time.
__device__ __forceinline__ void add_scaled(float2& acc, uint32_t p0, uint32_t p1, float s) {
    asm("{\n\t.reg .b64 a, p, s;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\t"
        "fma.rn.f32x2 a, p, s, a;\n\tmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(p0), "r"(p1), "f"(s));
}

template <typename O>
__global__ void __launch_bounds__(kThreads, 1) expert_product_fp8(const __grid_constant__ Fp8Args g) {
    extern __shared__ unsigned char raw[];
    unsigned char* stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char* turn = stages + kStages * kStageBytes;
    int* table = reinterpret_cast<int*>(turn + kAddWarps * kTurnBytes);
    __shared__ Fp8Shared sh;
    volatile int* abort_flag = &sh.abort;

    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cluster_rank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], kAddWarps);
            mbar_init(&sh.peer_empty[i], kAddWarps);  // in CTA 0: CTA 1's adding warps are done
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.scale_full[i], 1);
            mbar_init(&sh.scale_empty[i], kAddWarps);
        }
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_map(&g.w);
        prefetch_map(&g.x);
        prefetch_map(&g.x_small);
    }
    if (warp == kProductWarp) tmem_alloc_pair(&sh.tmem, kTmemColumns);
    build_tile_table<kTileRows, kThreads>(g.offsets, g.experts, g.slots, table, sh.warp_tiles);
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();
    tcgen05_fence_after();
    const uint32_t tmem = uniform(sh.tmem), stage0 = uniform(smem_addr(stages));

    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int tiles = uniform(all_tiles(table[g.experts], (g.out + kTileCols - 1) / kTileCols));
    const int blocks = (g.in + kBlock - 1) / kBlock;
    bool ok = true;
    if (warp == kCopyWarp) {
        const uint32_t full0 = map_to_rank(sh.full, 0);
        uint32_t s = 0, phase = 1;  // the stage, and the parity of its release
        Fp8Tile w;
        for (int t = first; ok && tile_at(g, table, t, tiles, w); t += step) {
            const int mine = rows_of(w, int(rank)), both = rows_of(w, 0) + rows_of(w, 1);
            const int row0 = w.row0 + int(rank) * 128;
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&sh.empty[s], phase, abort_flag);
                if (!ok) break;
                const uint32_t bar = full0 + s * 8;
                if (rank == 0) elect_arrive_expect_tx(&sh.full[s], 2 * kWBytes + uint32_t(both) * 128);
                const uint32_t a = stage0 + s * kStageBytes;
                tma_load_3d(a + kXBytes, &g.w, kb * kBlock, w.col0 + int(rank) * 64, w.expert, bar);
                load_rows(a, &g.x, &g.x_small, kb * kBlock, row0, mine, bar);
                next_stage<kStages>(s, phase);
            }
        }
        // every stage is released in this CTA too before it may leave
        for (int i = 0; ok && i < kStages; ++i) {
            ok = warp_wait(&sh.empty[s], phase, abort_flag);
            next_stage<kStages>(s, phase);
        }
    } else if (warp == kProductWarp) {
        if (rank == 0) {
            const uint64_t a0 = operand_desc(stage0, 16, 1024), b0 = operand_desc(stage0 + kXBytes, 16, 1024);
            constexpr uint32_t desc = instr_desc(0, false, false) | ((kTileCols >> 3) << 17);  // 0: e4m3
            uint32_t s = 0, phase = 0, buf = 0, free = 1;  // the stage and the buffer, with their parities
            bool ready = false;                            // they are full and free
            Fp8Tile w;
            for (int t = first; ok && tile_at(g, table, t, tiles, w); t += step) {
                for (int kb = 0; kb < blocks; ++kb) {
                    ok = ready || (warp_wait(&sh.full[s], phase, abort_flag) &&
                                   warp_wait(&sh.acc_empty[buf], free, abort_flag) &&
                                   warp_wait(&sh.peer_empty[buf], free, abort_flag));
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t here = s, into = buf;
                    next_stage<kStages>(s, phase);
                    next_stage<kBuffers>(buf, free);
                    const uint32_t looks = look(&sh.full[s], phase) & look(&sh.acc_empty[buf], free) &
                                           look(&sh.peer_empty[buf], free);
                    const uint32_t at = here * (kStageBytes >> 4);
                    mma_pair_8bit_4<32 / 16, 32 / 16>(tmem + into * kTileCols, a0 + at, b0 + at, desc, false);
                    mma_commit_pair(&sh.acc_full[into]);
                    mma_commit_pair(&sh.empty[here]);
                    ready = saw(looks);
                }
            }
        }
    } else if (warp == kScaleWarp) {
        uint32_t s = 0, phase = 1;  // the slot, and the parity of its release
        const int out_blocks = (g.out + kBlock - 1) / kBlock;
        Fp8Tile w;
        for (int t = first; ok && tile_at(g, table, t, tiles, w); t += step) {
            const int rows = min(128, w.rows - int(rank) * 128);
            const float* ws = g.ws + (int64_t(w.expert) * out_blocks + w.col0 / kBlock) * blocks;
            const float* xs = g.xs + (int64_t(w.row0) + rank * 128) * blocks;
            for (int k0 = 0; ok && k0 < blocks; k0 += kAhead) {
                float x[4][kAhead], wv[kAhead];
                if (g.scale_vec) {
                    ld_chunk<kAhead>(ws + k0, wv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i * 32 + lane < rows) ld_chunk<kAhead>(xs + int64_t(i * 32 + lane) * blocks + k0, x[i]);
                        else
#pragma unroll
                            for (int j = 0; j < kAhead; ++j) x[i][j] = 0.f;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) {
                        const int kb = min(k0 + j, blocks - 1);
                        wv[j] = __ldg(ws + kb);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i][j] = i * 32 + lane < rows ? __ldg(xs + int64_t(i * 32 + lane) * blocks + kb) : 0.f;
                    }
                }
                ok = warp_wait(&sh.scale_empty[s], phase, abort_flag);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sh.scale[s][j][i * 32 + lane] = x[i][j] * wv[j];
                __syncwarp();
                elect_arrive(&sh.scale_full[s]);
                next_stage<kScaleSlots>(s, phase);
            }
        }
    } else if (warp < kAddWarps) {
        const int c0 = warp / 4 * kWarpColumns, row = (warp & 3) * 32 + lane;
        const uint32_t from = tmem + (uint32_t(warp & 3) << 21) + uint32_t(c0);  // lane 32 * (warp % 4)
        const uint32_t freed = map_to_rank(rank == 0 ? sh.acc_empty : sh.peer_empty, 0);  // CTA 0's, of buffer 0
        uint32_t buf = 0, full = 0, group = 0, group_full = 0;  // the buffer and the scales, with their parities
        bool ready = false;                                     // the next block's products are there
        Fp8Tile w;
        for (int t = first; ok && tile_at(g, table, t, tiles, w); t += step) {
            float2 acc[kWarpColumns / 2];
#pragma unroll
            for (int i = 0; i < kWarpColumns / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int k0 = 0; ok && k0 < blocks; k0 += kAhead) {
                ok = warp_wait(&sh.scale_full[group], group_full, abort_flag);
                if (!ok) break;
                float scale[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) scale[j] = sh.scale[group][j][row];
                __syncwarp();
                elect_arrive(&sh.scale_empty[group]);
                next_stage<kScaleSlots>(group, group_full);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (k0 + j >= blocks) break;
                    ok = ready || warp_wait(&sh.acc_full[buf], full, abort_flag);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t here = buf;
                    next_stage<kBuffers>(buf, full);
                    const uint32_t looks = look(&sh.acc_full[buf], full);
                    uint32_t r[2][32];
                    tmem_load32(from + here * kTileCols, r[0]);
                    tmem_load32(from + here * kTileCols + 32, r[1]);
                    tmem_wait_load(r[0]);
                    tmem_wait_load(r[1]);
                    tcgen05_fence_before();
                    __syncwarp();
                    elect_arrive_pair(freed + here * 8);
#pragma unroll
                    for (int i = 0; i < kWarpColumns / 2; ++i)
                        add_scaled(acc[i], r[i / 16][i % 16 * 2], r[i / 16][i % 16 * 2 + 1], scale[j]);
                    ready = saw(looks);
                }
            }
            if (!ok) break;
            const auto sum = [&](int i) { return i & 1 ? acc[i / 2].y : acc[i / 2].x; };
            const int top = (warp & 3) * 32, rows = w.rows - int(rank) * 128 - top;  // of this warp
            const int cols = g.out - w.col0 - c0;                                   // that are there
            O* p = static_cast<O*>(g.y) + (int64_t(w.row0) + rank * 128 + top) * g.out + w.col0 + c0;
            constexpr int kCols = 128 / int(sizeof(O));
#pragma unroll
            for (int c = 0; c < kWarpColumns; c += kCols)
                store_rows(turn + warp * kTurnBytes, p + c, g.out, rows, cols - c, g.vec,
                           [&](int i) { return sum(c + i); });
            __syncwarp();
        }
    }
    __syncwarp();
    if (*abort_flag) let_copies_land();
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves, or frees tensor memory, while the other still uses it
    tcgen05_fence_after();
    if (warp == kProductWarp) tmem_dealloc_pair(tmem, kTmemColumns);
}

constexpr size_t kMostSmem = 1024 + kStages * size_t(kStageBytes) + kAddWarps * kTurnBytes + (kMaxExperts + 1) * 4;

}  // namespace

uint32_t pipeline_timeouts_fp8() { return read_pipeline_timeouts(); }

cudaError_t launch_expert_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                     const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                     int64_t experts, int y_type, Scratch scratch, cudaStream_t stream) {
    Matrix mx = matrix_of(x, in, slots, 1, 1), mw = matrix_of(w, in, out, experts, 1);
    Matrix* ms[2] = {&mx, &mw};
    cudaError_t err;
    if (!make_readable(ms, {false, true}, offsets, slots, scratch, stream, &err))
        return launch_matmul_fp8_any(x, x_scale, w, w_scale, offsets, y, slots, in, out, experts, y_type, stream);
    if (err != cudaSuccess) return err;
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    Fp8Args g;
    if (!make_map(&g.w, type, mw, kBlock, 64, true) || !make_map(&g.x_small, type, mx, kBlock, 16, false))
        return cudaErrorInvalidValue;
    g.x = g.x_small;  // a CTA's rows round up to 64 only from 49 on
    if (slots > 48 && !make_map(&g.x, type, mx, kBlock, 64, false)) return cudaErrorInvalidValue;
    g.xs = x_scale;
    g.ws = w_scale;
    g.offsets = offsets;
    g.y = y;
    g.slots = int(slots);
    g.experts = int(experts);
    g.in = int(in);
    g.out = int(out);
    const int y_size = y_type == ROWOPS_F32 ? 4 : 2;
    g.vec = out * y_size % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
    g.scale_vec = (in + kBlock - 1) / kBlock % kAhead == 0 &&
                  (reinterpret_cast<uintptr_t>(x_scale) | reinterpret_cast<uintptr_t>(w_scale)) % 16 == 0;
    const int64_t tiles = most_row_tiles(slots, experts) * ((out + kTileCols - 1) / kTileCols);
    cudaError_t e = cudaErrorInvalidValue;
    if (tiles >= kMostTiles) return e;  // more than a device's memory holds
    with_type(y_type, [&](auto o) {
        e = launch_pairs<expert_product_fp8<decltype(o)>>(tiles, kThreads, kMostSmem, stream, g);
    });
    return e;
}

}  // namespace rowops
