// expert_fp8.cu - the experts' product on e4m3 operands with a scale for each
// block of 128 (tcgen05, clusters of two CTAs).
//
//   y[s][n] = sum_b xs[s][b] ws[e][n / 128][b] P_b,  P_b = sum_{k in block b} xq[s][k] wq[e][n][k]
//
// Tiles, copies and roles are those of expert_matmul.cu: 256 output columns by
// up to 256 rows of a group, and a stage of 128 bytes along the sum is one block.
// The tensor cores add up P_b alone; what they cannot do is the pair of scales,
// which differs from block to block.  So each block's products go to one of two
// tensor-memory buffers, and sixteen warps a CTA add scale * P_b to sums that stay
// in registers (64 a thread) while the next block's products run into the other.
//
// What bounds it: a block's 256 x 256 x 128 products take 512 clocks of the tensor
// cores; in that time a CTA reads 128 x 256 values from tensor memory (256 clocks)
// and adds them (128 clocks of two-wide fused multiply-adds), and the buffers
// change hands twice.  A lane holds one output column and a register one row, so
// the scale is a row's: warp 19 multiplies xs with ws once for all lanes, eight
// blocks ahead, and the adding warps read it from shared memory as a broadcast.
#include <cuda_fp8.h>

#include "groups.cuh"
#include "tensor_core.cuh"
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kBlock = 128;                  // values of the sum per scale, and per stage
constexpr int kStages = 6;
constexpr uint32_t kHalfBytes = 128 * 128;   // one operand's share of a CTA and stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr int kScaleSlots = 8;
constexpr int kAddWarps = 16;
constexpr int kWarpColumns = kMostRows / (kAddWarps / 4);  // rows of y that an adding warp holds
constexpr int kCopyWarpA = 16, kCopyWarpB = 17, kProductWarp = 18, kScaleWarp = 19;
constexpr int kThreads = 640;
constexpr uint32_t kTmemColumns = 512;

struct Fp8Args {
    CUtensorMap w;        // boxes of 128 output columns
    CUtensorMap x;        // boxes of 128 rows
    CUtensorMap x_small;  // boxes of 16 rows
    const float* xs;
    const float* ws;
    const int32_t* offsets;
    void* y;
    int slots, experts;
    int in, out;
};

struct Fp8Shared {
    float scale[kScaleSlots][kMostRows];
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    uint32_t tmem;
    int abort;
};

struct Fp8Tile {
    int expert, m0, n0, n, width;
};

__device__ __forceinline__ bool tile_at(const Fp8Args& g, const int* table, int64_t t, Fp8Tile& w) {
    const int tiles_m = (g.out + 255) / 256;
    const int64_t row = t / tiles_m;
    if (row >= table[g.experts]) return false;
    const RowTile r = row_tile(g.offsets, g.experts, g.slots, table, int(row));
    w.expert = uniform(r.expert);
    w.m0 = int(t % tiles_m) * 256;
    w.n0 = uniform(r.first);
    w.n = uniform(r.count);
    w.width = (w.n + 31) & ~31;
    return true;
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

// acc += s * p, two at a time.
__device__ __forceinline__ void add_scaled(float2& acc, uint32_t p0, uint32_t p1, float s0, float s1) {
    asm("{\n\t.reg .b64 a, p, s;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 a, p, s, a;\n\tmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(p0), "r"(p1), "f"(s0), "f"(s1));
}

template <typename O>
__global__ void __launch_bounds__(kThreads, 1) expert_product_fp8(const __grid_constant__ Fp8Args g) {
    extern __shared__ unsigned char raw[];
    unsigned char* stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    int* table = reinterpret_cast<int*>(stages + kStages * kStageBytes);
    __shared__ Fp8Shared sh;
    volatile int* abort_flag = &sh.abort;

    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);  // a copying warp per operand
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kAddWarps);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.scale_full[i], 1);
            mbar_init(&sh.scale_empty[i], kAddWarps);
        }
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarpA && lane == 0) {
        prefetch_map(&g.w);
        prefetch_map(&g.x);
        prefetch_map(&g.x_small);
    }
    if (warp == kProductWarp) tmem_alloc_pair(&sh.tmem, kTmemColumns);
    if (warp == 0) build_tile_table<kMostRows>(g.offsets, g.experts, g.slots, table);
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();
    tcgen05_fence_after();
    const uint32_t tmem = uniform(sh.tmem), stage0 = uniform(smem_addr(stages));

    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int blocks = (g.in + kBlock - 1) / kBlock;
    bool ok = true;
    if (warp == kCopyWarpA || warp == kCopyWarpB) {
        const bool is_a = warp == kCopyWarpA;
        const uint32_t to = stage0 + (is_a ? 0 : kHalfBytes);
        uint32_t it = 0;
        Fp8Tile w;
        for (int64_t t = first; ok && tile_at(g, table, t, w); t += step) {
            const int half = w.width / 2;
            const int m0 = w.m0 + int(rank) * 128, n0 = w.n0 + int(rank) * half;
            const uint32_t mine = is_a ? kHalfBytes : uint32_t(half) * 128;
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const uint32_t s = it % kStages;
                ok = warp_wait(&sh.empty[s], ((it / kStages) & 1) ^ 1, abort_flag);
                if (!ok) break;
                const uint32_t bar = map_to_rank(&sh.full[s], 0);
                if (rank == 0) elect_arrive_expect_tx(&sh.full[s], 2 * mine);
                const uint32_t dst = to + s * kStageBytes;
                if (is_a) {
                    tma_load_3d(dst, &g.w, kb * kBlock, m0, w.expert, bar);
                } else if (half == 128) {
                    tma_load_2d(dst, &g.x, kb * kBlock, n0, bar);
                } else {
                    for (int i = 0; i < half; i += 16)
                        tma_load_2d(dst + i * 128, &g.x_small, kb * kBlock, n0 + i, bar);
                }
            }
        }
        // every stage is released in this CTA too before it may leave
        for (uint32_t i = it > kStages ? it - kStages : 0; ok && i < it; ++i)
            ok = warp_wait(&sh.empty[i % kStages], (i / kStages) & 1, abort_flag);
    } else if (warp == kProductWarp) {
        if (rank == 0) {
            uint32_t it = 0;
            Fp8Tile w;
            for (int64_t t = first; ok && tile_at(g, table, t, w); t += step) {
                const uint32_t desc = with_n(instr_desc(0, false, false), w.width);  // 0: e4m3
                for (int kb = 0; kb < blocks; ++kb, ++it) {
                    const uint32_t s = it % kStages, d = tmem + (it & 1) * kMostRows;
                    ok = warp_wait(&sh.acc_empty[it & 1], ((it >> 1) & 1) ^ 1, abort_flag) &&
                         warp_wait(&sh.full[s], (it / kStages) & 1, abort_flag);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t a = stage0 + s * kStageBytes, b = a + kHalfBytes;
#pragma unroll
                    for (int i = 0; i < kBlock / 32; ++i)
                        mma_pair_8bit(d, operand_desc(a + i * 32, 16, 1024), operand_desc(b + i * 32, 16, 1024), desc,
                                      i > 0);
                    mma_commit_pair(&sh.acc_full[it & 1]);
                    mma_commit_pair(&sh.empty[s]);
                }
            }
        }
    } else if (warp == kScaleWarp) {
        uint32_t it = 0;
        const int out_blocks = (g.out + kBlock - 1) / kBlock;
        Fp8Tile w;
        for (int64_t t = first; ok && tile_at(g, table, t, w); t += step) {
            const int nb = w.m0 / kBlock + int(rank);
            const float* ws = g.ws + (int64_t(w.expert) * out_blocks + min(nb, out_blocks - 1)) * blocks;
            const float* xs = g.xs + int64_t(w.n0) * blocks;
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const uint32_t s = it % kScaleSlots;
                ok = warp_wait(&sh.scale_empty[s], ((it / kScaleSlots) & 1) ^ 1, abort_flag);
                if (!ok) break;
                const float wv = __ldg(ws + kb);
                float v[kMostRows / 32];
#pragma unroll
                for (int i = 0; i < kMostRows / 32; ++i) {
                    const int c = i * 32 + lane;
                    v[i] = c < w.n ? __ldg(xs + int64_t(c) * blocks + kb) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < kMostRows / 32; ++i) sh.scale[s][i * 32 + lane] = v[i] * wv;
                __syncwarp();
                elect_arrive(&sh.scale_full[s]);
            }
        }
    } else {
        const int c0 = warp / 4 * kWarpColumns, row = int(rank) * 128 + (warp & 3) * 32 + lane;
        const uint32_t from = tmem + (uint32_t(warp & 3) << 21) + uint32_t(c0);  // lane 32 * (warp % 4)
        const uint32_t free0 = map_to_rank(&sh.acc_empty[0], 0), free1 = map_to_rank(&sh.acc_empty[1], 0);
        uint32_t it = 0;
        Fp8Tile w;
        for (int64_t t = first; ok && tile_at(g, table, t, w); t += step) {
            float2 acc[kWarpColumns / 2];
#pragma unroll
            for (int i = 0; i < kWarpColumns / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const uint32_t s = it % kScaleSlots;
                ok = warp_wait(&sh.acc_full[it & 1], (it >> 1) & 1, abort_flag) &&
                     warp_wait(&sh.scale_full[s], (it / kScaleSlots) & 1, abort_flag);
                if (!ok) break;
                tcgen05_fence_after();
                const float4* scale = reinterpret_cast<const float4*>(&sh.scale[s][c0]);
#pragma unroll
                for (int q = 0; q < kWarpColumns / 16; ++q) {
                    if (c0 + q * 16 >= w.width) break;
                    uint32_t r[16];
                    tmem_load16(from + (it & 1) * kMostRows + q * 16, r);
                    tmem_wait_load16(r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = scale[q * 4 + i];
                        add_scaled(acc[q * 8 + i * 2], r[i * 4], r[i * 4 + 1], v.x, v.y);
                        add_scaled(acc[q * 8 + i * 2 + 1], r[i * 4 + 2], r[i * 4 + 3], v.z, v.w);
                    }
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(it & 1 ? free1 : free0);
                    mbar_arrive(&sh.scale_empty[s]);
                }
            }
            if (!ok) break;
            const int m = w.m0 + row;
            if (m < g.out) {
                O* p = static_cast<O*>(g.y) + int64_t(w.n0 + c0) * g.out + m;
#pragma unroll
                for (int i = 0; i < kWarpColumns; ++i)
                    if (c0 + i < w.n) p[int64_t(i) * g.out] = from_float<O>(i & 1 ? acc[i / 2].y : acc[i / 2].x);
            }
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

constexpr size_t kMostSmem = 1024 + kStages * size_t(kStageBytes) + (kMaxExperts + 1) * 4;

}  // namespace

uint32_t pipeline_timeouts_fp8() { return read_pipeline_timeouts(); }

cudaError_t launch_expert_matmul_fp8(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                     const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                     int64_t experts, int y_type, cudaStream_t stream) {
    const bool aligned = in % 16 == 0 && (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) % 16 == 0;
    if (!aligned)
        return launch_matmul_fp8_any(x, x_scale, w, w_scale, offsets, y, slots, in, out, experts, y_type, stream);
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    Fp8Args g;
    if (!make_map(&g.w, type, 1, w, in, out, experts, kBlock, 128, true) ||
        !make_map(&g.x, type, 1, x, in, slots, 1, kBlock, 128, false) ||
        !make_map(&g.x_small, type, 1, x, in, slots, 1, kBlock, 16, false))
        return cudaErrorInvalidValue;
    g.xs = x_scale;
    g.ws = w_scale;
    g.offsets = offsets;
    g.y = y;
    g.slots = int(slots);
    g.experts = int(experts);
    g.in = int(in);
    g.out = int(out);
    const int64_t tiles = most_row_tiles(slots, experts) * ((out + 255) / 256);
    cudaError_t e = cudaErrorInvalidValue;
    with_type(y_type, [&](auto o) {
        e = launch_pairs<expert_product_fp8<decltype(o)>>(tiles, kThreads, kMostSmem, stream, g);
    });
    return e;
}

}  // namespace rowops
