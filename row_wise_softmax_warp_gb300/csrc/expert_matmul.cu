// expert_matmul.cu - the experts' matrix products on tcgen05.
//
//   kRows     y[s][n]  = sum_k w[e][n][k] x[s][k]        rows s of expert e
//   kRowsT    y[s][n]  = sum_k w[e][k][n] x[s][k]
//   kWeights  dw[e][m][n] = sum_{s of e} dy[s][m] x[s][n]
//
// The first operand's side (M) is the weights' output width, or dw's rows; the
// second's (N) is tokens, or dw's columns.  Weights on the M side leave N free
// to follow the ragged groups: a group of n rows is cut into ceil(n / 256) even
// tiles of a multiple of 32 columns, so a group of 40 rows pays for 64 and not
// for the 256 of a fixed row tile.
//
// A cluster of two CTAs computes 256 x N (N <= 256): each holds its 128 rows of
// the first operand and half of the second in shared memory, 64 of the sum at a
// time, and its 128 x N accumulators in tensor memory, twice, so the epilogue
// of one tile runs beside the products of the next.  Both operands together
// take 64 bytes a clock from the L2 at the full rate of the tensor cores; one
// CTA alone with 128 x 256 would take 96.
// Warps 4 and 5 copy an operand each, warp 6 issues products (in CTA 0), warps
// 0..3 write results, and in kWeights warp 7 zeroes.
//
// Operands whose sum runs along rows in memory are K-major, the others
// MN-major: both sides of kWeights, the weights of kRowsT.  Sums past the end
// (k >= in) are zeros that TMA fills in.  The sum of kWeights ends inside a
// group's last 64 rows, where TMA would read the next group's: its products
// stop at a multiple of 16 rows, and the rows between are zeroed in shared
// memory before them (both sides: 0 times a NaN is no zero).
#include "groups.cuh"
#include "row_store.cuh"
#include "tensor_core.cuh"
#include "types.cuh"

namespace rowops {
namespace {

enum Form { kRows, kRowsT, kWeights };
template <Form F>
using FormOf = std::integral_constant<Form, F>;

constexpr int kTileN = kMostRows;              // most columns of a tile
constexpr int kStepK = 64;                     // of the sum per stage
constexpr int kStages = 6;
constexpr uint32_t kHalfBytes = 128 * 128;     // one operand's share of a CTA and stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr int kColumn = 64 * 128;              // bytes of a 64-value column of an MN-major operand
constexpr int kCopyWarpA = 4, kCopyWarpB = 5, kProductWarp = 6, kZeroWarp = 7;  // the last in kWeights only
constexpr uint32_t kTmemColumns = 512;

constexpr int threads_of(Form form) { return form == kWeights ? 256 : 224; }

struct ProductArgs {
    CUtensorMap a;        // first operand
    CUtensorMap b;        // second operand; kRows, kRowsT: boxes of 64 rows
    CUtensorMap b_small;  // kRows, kRowsT: boxes of 16 rows
    const int32_t* offsets;
    void* out;
    int slots, experts;
    int m, n, k;  // kRows*: m output width, k input width.  kWeights: dw is m x n
    uint32_t format;  // operand format code
    bool vec;         // kWeights: rows of dw allow 16-byte stores
};

struct Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t tail_full[kStages], tail_done[kStages];  // kWeights: a stage whose last rows are zeroed
    int warp_tiles[8];
    uint32_t tmem;
    uint32_t progress;  // stages whose copies are under way, for waits that span many
    int abort;
};

struct Tile {
    int expert = 0;
    int m0;       // first row of the pair's 256
    int n0;       // first column: a row of x and y, or a column of dw
    int n;        // columns to write
    int width;    // columns the products compute
    int sum0;     // kWeights: first row of the sum
    int sum;      // its length
};

// The number of tiles.
template <Form FORM>
__device__ __forceinline__ int tiles_in_all(const ProductArgs& g, const int* table) {
    const int tiles_m = (g.m + 255) / 256;
    if constexpr (FORM == kWeights) return (g.n + kTileN - 1) / kTileN * g.experts * tiles_m;  // the host has seen it
    else return all_tiles(table[g.experts], tiles_m);
}

// Tile t of `tiles`; false past the last.
template <Form FORM>
__device__ __forceinline__ bool tile_at(const ProductArgs& g, const int* table, int t, int tiles, Tile& w) {
    if (t >= tiles) return false;
    const int tiles_m = (g.m + 255) / 256;
    if constexpr (FORM == kWeights) {
        const int tiles_n = (g.n + kTileN - 1) / kTileN;
        const int row = t / tiles_m;
        w.expert = row / tiles_n;
        w.m0 = t % tiles_m * 256;
        w.n0 = row % tiles_n * kTileN;
        w.n = min(kTileN, g.n - w.n0);
        w.width = (w.n + 127) & ~127;
        const RowRange r = group_rows(g.offsets, w.expert, g.slots);
        w.sum0 = r.first;
        w.sum = r.count;
    } else {
        const int row = t / tiles_m;
        const RowTile r = row_tile(g.offsets, g.experts, g.slots, table, row, w.expert);
        w.expert = uniform(r.expert);
        w.m0 = t % tiles_m * 256;
        w.n0 = r.first;
        w.n = r.count;
        w.width = (w.n + 31) & ~31;
        w.sum0 = 0;
        w.sum = g.k;
    }
    return true;
}

// Rows of the last stage of a sum of kWeights that have to be zeroed, or 0.
__device__ __forceinline__ int ragged_rows(int sum) { return (16 - (sum & 15)) & 15; }

// Zeroes the ragged rows of one CTA's operands in a stage; the whole warp.
__device__ __forceinline__ void zero_ragged(unsigned char* stage, int sum, int width) {
    const int valid = (sum - 1) % kStepK + 1, rows = ragged_rows(sum);
    const int columns = 2 + width / 128;  // 64-value columns of both operands
    for (int i = threadIdx.x & 31; i < columns * rows * 8; i += 32) {
        const int c = i / (rows * 8), in = i % (rows * 8);
        unsigned char* column = stage + (c < 2 ? c * kColumn : int(kHalfBytes) + (c - 2) * kColumn);
        *reinterpret_cast<uint4*>(column + (valid + in / 8) * 128 + in % 8 * 16) = make_uint4(0, 0, 0, 0);
    }
}

// One warp's 32 rows of a tile in tensor memory, 32 columns at a time; after the
// last load the buffer is given back.
struct Source {
    uint32_t tmem, free_bar;
    bool zero;  // a sum of nothing: no buffer
    __device__ __forceinline__ void load(int c, int width, uint32_t (&r)[32]) const {
        if (zero) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
            return;
        }
        tmem_load32(tmem + uint32_t(c), r);
        tmem_wait_load(r);
        if (c + 32 >= width) {
            tcgen05_fence_before();
            __syncwarp();
            elect_arrive_pair(free_bar);
        }
    }
};

// kRows, kRowsT: a lane holds an output column and a register a row of y.  A step
// from row to row instead of a product a row, and no test where 32 rows are there:
// 8192 x 768 -> 2048, 30.0 -> 23.5 us.
template <typename O>
__device__ __forceinline__ void write_rows(const ProductArgs& g, const Tile& w, const Source& from, int m) {
    for (int c = 0; c < w.n; c += 32) {
        uint32_t r[32];
        from.load(c, w.n, r);
        if (m < g.m) {
            O* p = static_cast<O*>(g.out) + int64_t(w.n0 + c) * g.m + m;
            const int rows = w.n - c;
            if (rows >= 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i, p += g.m) *p = from_float<O>(__uint_as_float(r[i]));
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i, p += g.m)
                    if (i < rows) *p = from_float<O>(__uint_as_float(r[i]));
            }
        }
        __syncwarp();
    }
}

// kWeights: a lane holds a row of dw.  m: the warp's first row.
template <typename O>
__device__ __forceinline__ void write_weights(const ProductArgs& g, const Tile& w, const Source& from, int m,
                                              unsigned char* turn) {
    constexpr int kCols = 128 / int(sizeof(O));
    for (int c = 0; c < w.n; c += kCols) {
        uint32_t r[kCols / 32][32];
#pragma unroll
        for (int h = 0; h < kCols / 32; ++h)
            if (c + h * 32 < w.n) from.load(c + h * 32, w.n, r[h]);
        store_rows(turn, static_cast<O*>(g.out) + (int64_t(w.expert) * g.m + m) * g.n + w.n0 + c, g.n, g.m - m,
                   w.n - c, g.vec, [&](int i) { return __uint_as_float(r[i / 32][i % 32]); });
    }
}

template <typename O, Form FORM>  // the operands' type is g.format
__global__ void __launch_bounds__(threads_of(FORM), 1)
    expert_product(const __grid_constant__ ProductArgs g) {
    extern __shared__ unsigned char raw[];
    unsigned char* stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char* turn = stages + kStages * kStageBytes;  // kWeights
    int* table = reinterpret_cast<int*>(turn);              // the others
    __shared__ Shared sh;
    volatile int* abort_flag = &sh.abort;
    volatile uint32_t* progress = &sh.progress;

    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cluster_rank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);  // a copying lane per operand
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.tail_full[i], 2);
            mbar_init(&sh.tail_done[i], 2);  // the zeroing warps of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 8);  // the epilogue warps of both CTAs
        }
        sh.progress = 0;
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarpA && lane == 0) {
        prefetch_map(&g.a);
        prefetch_map(&g.b);
        if constexpr (FORM != kWeights) prefetch_map(&g.b_small);
    }
    if (warp == kProductWarp) tmem_alloc_pair(&sh.tmem, kTmemColumns);
    if constexpr (FORM != kWeights)
        build_tile_table<kMostRows, threads_of(FORM)>(g.offsets, g.experts, g.slots, table, sh.warp_tiles);
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();
    tcgen05_fence_after();
    const uint32_t tmem = uniform(sh.tmem), stage0 = uniform(smem_addr(stages));

    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = uniform(tiles_in_all<FORM>(g, table));
    bool ok = true;
    if (warp == kCopyWarpA || warp == kCopyWarpB) {
        const bool is_a = warp == kCopyWarpA;
        const uint32_t to = stage0 + (is_a ? 0 : kHalfBytes);
        const uint32_t full0 = map_to_rank(sh.full, 0), tail0 = map_to_rank(sh.tail_full, rank);
        uint32_t s = 0, phase = 1;  // the stage, and the parity of its release
        uint32_t stages_begun = 0;
        Tile w;
        for (int t = first; ok && tile_at<FORM>(g, table, t, tiles, w); t += step) {
            const int sum = uniform(w.sum), blocks = (sum + kStepK - 1) / kStepK;
            const int half = uniform(w.width) / 2, expert = uniform(w.expert), sum0 = uniform(w.sum0);
            const int m0 = uniform(w.m0) + int(rank) * 128, n0 = uniform(w.n0) + int(rank) * half;
            const uint32_t mine = is_a ? kHalfBytes : uint32_t(half) * 128;
            const bool ragged = FORM == kWeights && ragged_rows(sum) != 0;
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&sh.empty[s], phase, abort_flag);
                if (!ok) break;
                uint32_t bar = full0 + s * 8;
                if (ragged && kb == blocks - 1) {  // each CTA's zeroing warp waits for its own copies
                    if (rank == 0) elect_arrive(&sh.full[s]);
                    elect_arrive_expect_tx(&sh.tail_full[s], mine);
                    bar = tail0 + s * 8;
                } else if (rank == 0) {
                    elect_arrive_expect_tx(&sh.full[s], 2 * mine);
                }
                const uint32_t dst = to + s * kStageBytes;
                const int k0 = kb * kStepK;
                if (is_a) {
                    *progress = ++stages_begun;
                    if constexpr (FORM == kRows) {
                        tma_load_3d(dst, &g.a, k0, m0, expert, bar);
                    } else if constexpr (FORM == kRowsT) {
                        tma_load_3d(dst, &g.a, m0, k0, expert, bar);
                        tma_load_3d(dst + kColumn, &g.a, m0 + 64, k0, expert, bar);
                    } else {
                        tma_load_2d(dst, &g.a, m0, sum0 + k0, bar);
                        tma_load_2d(dst + kColumn, &g.a, m0 + 64, sum0 + k0, bar);
                    }
                } else if constexpr (FORM == kWeights) {
                    tma_load_2d(dst, &g.b, n0, sum0 + k0, bar);
                    if (half == 128) tma_load_2d(dst + kColumn, &g.b, n0 + 64, sum0 + k0, bar);
                } else {
                    load_rows(dst, &g.b, &g.b_small, k0, n0, half, bar);
                }
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
            uint32_t s = 0, phase = 0, acc = 0, tails = 0;  // tails: the phases of tail_done, a bit a stage
            const uint64_t a0 = FORM == kRows ? operand_desc(stage0, 16, 1024) : operand_desc(stage0, kColumn, 1024);
            const uint64_t b0 = FORM == kWeights ? operand_desc(stage0 + kHalfBytes, kColumn, 1024)
                                                 : operand_desc(stage0 + kHalfBytes, 16, 1024);
            constexpr uint32_t kNextA = (FORM == kRows ? 32 : 2048) >> 4, kNextB = (FORM == kWeights ? 2048 : 32) >> 4;
            Tile w;
            for (int t = first; ok && tile_at<FORM>(g, table, t, tiles, w); t += step) {
                const int sum = uniform(w.sum), blocks = (sum + kStepK - 1) / kStepK;
                if (blocks == 0) continue;
                const bool ragged = FORM == kWeights && ragged_rows(sum) != 0;
                const uint32_t d = tmem + (acc & 1) * kTileN;
                const uint32_t desc = uniform(with_n(instr_desc(g.format, FORM != kRows, FORM == kWeights), w.width));
                ok = warp_wait(&sh.acc_empty[acc & 1], ((acc >> 1) & 1) ^ 1, abort_flag);
                bool ready = false;  // the stage was seen full
                for (int kb = 0; ok && kb < blocks; ++kb) {
                    ok = ready || warp_wait(&sh.full[s], phase, abort_flag);
                    if (FORM == kWeights && ragged && kb == blocks - 1) {
                        ok = ok && warp_wait_cluster(&sh.tail_done[s], (tails >> s) & 1, abort_flag);
                        tails ^= 1u << s;
                    }
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t here = s, at = s * (kStageBytes >> 4);
                    // The look at the next stage overlaps with this one's products (weights'
                    // gradient of 32768 rows, 16 experts, 2048 x 4096: 334 -> 313 us).
                    next_stage<kStages>(s, phase);
                    const uint32_t looks = kb + 1 < blocks ? look(&sh.full[s], phase) : 0;
                    if (FORM == kWeights && kb == blocks - 1) {
                        const int steps = (sum - kb * kStepK + 15) / 16;
                        for (int i = 0; i < steps; ++i)
                            mma_pair_16bit(d, a0 + at + i * kNextA, b0 + at + i * kNextB, desc, kb > 0 || i > 0);
                    } else {  // past the end of a sum of kRows and kRowsT are zeros
                        mma_pair_16bit_4<kNextA, kNextB>(d, a0 + at, b0 + at, desc, kb > 0);
                    }
                    mma_commit_pair(&sh.empty[here]);
                    ready = saw(looks);
                }
                if (ok) mma_commit_pair(&sh.acc_full[acc & 1]);
                ++acc;
            }
        }
    } else if (FORM == kWeights && warp == kZeroWarp) {
        uint32_t it = 0, tails = 0;  // tails: the phases of tail_full
        Tile w;
        for (int t = first; tile_at<FORM>(g, table, t, tiles, w); t += step) {
            it += (w.sum + kStepK - 1) / kStepK;
            if (ragged_rows(w.sum) == 0) continue;
            const uint32_t s = (it - 1) % kStages;
            if (!warp_wait_stages(&sh.tail_full[s], (tails >> s) & 1, abort_flag, progress)) break;
            tails ^= 1u << s;
            zero_ragged(stages + s * kStageBytes, w.sum, w.width);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(&sh.tail_done[s], 0));
        }
    } else {
        uint32_t acc = 0;
        Tile w;
        for (int t = first; tile_at<FORM>(g, table, t, tiles, w); t += step) {
            const bool zero = uniform(w.sum) == 0;
            if (!zero && !warp_wait_stages(&sh.acc_full[acc & 1], (acc >> 1) & 1, abort_flag, progress)) break;
            tcgen05_fence_after();
            const Source from{tmem + (uint32_t(warp * 32) << 16) + (acc & 1) * kTileN,
                              map_to_rank(&sh.acc_empty[acc & 1], 0), zero};
            const int m = w.m0 + int(rank) * 128 + warp * 32;
            if constexpr (FORM == kWeights) write_weights<O>(g, w, from, m, turn + warp * kTurnBytes);
            else write_rows<O>(g, w, from, m + lane);
            if (!zero) ++acc;
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

constexpr size_t kMostSmem = 1024 + kStages * size_t(kStageBytes) + 4 * kTurnBytes;
static_assert(4 * kTurnBytes >= (kMaxExperts + 1) * 4, "the table of tiles lies where the others turn rows");

}  // namespace

uint32_t pipeline_timeouts_matmul() { return read_pipeline_timeouts(); }

cudaError_t launch_expert_matmul(const void* x, const void* w, const int32_t* offsets, void* y, int64_t slots,
                                 int64_t in, int64_t out, int64_t experts, bool transposed, int dtype,
                                 Scratch scratch, cudaStream_t stream) {
    Matrix mx = matrix_of(x, in, slots, 1, 2);
    Matrix mw = matrix_of(w, transposed ? out : in, transposed ? in : out, experts, 2);
    Matrix* ms[2] = {&mx, &mw};
    cudaError_t err;
    if (!make_readable(ms, {false, true}, offsets, slots, scratch, stream, &err))
        return launch_matmul_any(x, w, offsets, y, slots, in, out, experts, transposed, dtype, stream);
    if (err != cudaSuccess) return err;
    const CUtensorMapDataType type =
        dtype == ROWOPS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    ProductArgs g;
    if (!make_map(&g.a, type, mw, 64, transposed ? 64 : 128, true) || !make_map(&g.b_small, type, mx, 64, 16, false))
        return cudaErrorInvalidValue;
    g.b = g.b_small;  // half a tile is 64 rows or more only where a tile has more than 96
    if (slots > 96 && !make_map(&g.b, type, mx, 64, 64, false)) return cudaErrorInvalidValue;
    g.offsets = offsets;
    g.out = y;
    g.slots = int(slots);
    g.experts = int(experts);
    g.m = int(out);
    g.n = 0;
    g.k = int(in);
    g.format = dtype == ROWOPS_F16 ? 0 : 1;
    g.vec = false;
    const int64_t tiles = most_row_tiles(slots, experts) * ((out + 255) / 256);
    if (tiles >= kMostTiles) return cudaErrorInvalidValue;
    auto go = [&](auto t, auto form) {
        constexpr Form kForm = decltype(form)::value;
        return launch_pairs<expert_product<decltype(t), kForm>>(tiles, threads_of(kForm), kMostSmem, stream, g);
    };
    if (dtype == ROWOPS_F16) return transposed ? go(__half{}, FormOf<kRowsT>{}) : go(__half{}, FormOf<kRows>{});
    return transposed ? go(__nv_bfloat16{}, FormOf<kRowsT>{}) : go(__nv_bfloat16{}, FormOf<kRows>{});
}

cudaError_t launch_expert_matmul_wgrad(const void* dy, const void* x, const int32_t* offsets, void* dw,
                                       int64_t slots, int64_t in, int64_t out, int64_t experts, int dtype,
                                       int dw_type, Scratch scratch, cudaStream_t stream) {
    const int dw_size = dw_type == ROWOPS_F32 ? 4 : 2;
    if (slots == 0) return cudaMemsetAsync(dw, 0, size_t(experts) * out * in * dw_size, stream);
    Matrix mdy = matrix_of(dy, out, slots, 1, 2), mx = matrix_of(x, in, slots, 1, 2);
    Matrix* ms[2] = {&mdy, &mx};
    cudaError_t err;
    if (!make_readable(ms, {false, false}, offsets, slots, scratch, stream, &err))
        return launch_matmul_wgrad_any(dy, x, offsets, dw, slots, in, out, experts, dtype, dw_type, stream);
    if (err != cudaSuccess) return err;
    const CUtensorMapDataType type =
        dtype == ROWOPS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    ProductArgs g;
    if (!make_map(&g.a, type, mdy, 64, 64, false) || !make_map(&g.b, type, mx, 64, 64, false))
        return cudaErrorInvalidValue;
    g.b_small = g.b;
    g.offsets = offsets;
    g.out = dw;
    g.slots = int(slots);
    g.experts = int(experts);
    g.m = int(out);
    g.n = int(in);
    g.k = 0;
    g.format = dtype == ROWOPS_F16 ? 0 : 1;
    g.vec = in * dw_size % 16 == 0 && reinterpret_cast<uintptr_t>(dw) % 16 == 0;
    const int64_t tiles = experts * ((out + 255) / 256) * ((in + kTileN - 1) / kTileN);
    if (tiles >= kMostTiles) return cudaErrorInvalidValue;
    auto go = [&](auto o) {
        return launch_pairs<expert_product<decltype(o), kWeights>>(tiles, threads_of(kWeights), kMostSmem, stream, g);
    };
    if (dw_type == ROWOPS_F32) return go(float{});
    return dtype == ROWOPS_F16 ? go(__half{}) : go(__nv_bfloat16{});
}

}  // namespace rowops
