// expert_mx4.cu - the experts' product on microscaled 4-bit operands (tcgen05
// kind::mxf4, clusters of two CTAs).
//
//   y[s][n] = sum_k 2^(ws - 127) wq[e][n][k] * 2^(xs - 127) xq[s][k]     rows s of expert e
//
// Laid out as expert_matmul.cu: weights on the M side, 256 output columns of a pair of
// CTAs; tokens on the N side, up to 224 of a group; a stage of 128 bytes along the sum,
// which is 256 values in eight blocks.  The tensor cores multiply by the scales: they
// read them from tensor memory, where the 128 rows of an operand lie as 32 lanes of four
// columns, four blocks a column, the same in all four quarters.  Each CTA needs the
// scales of its own 128 output columns and those of all tokens.  Three warps a CTA read
// them as they lie in memory, write them to the stage in that order, and
// tcgen05.cp moves them, in order with the products that follow.
//
// Two accumulators of 224 columns and two stages' scales (24 columns each) fill 496 of
// the 512 columns of tensor memory; with 256 tokens a tile there would be no room for
// the scales, or for the second accumulator that hides the write-out.
//
// What bounds it: 16384 x 4096 -> 4096 takes 103 to 106 us (5200 to 5350 TFLOP/s; the bf16
// product 299).  Variants that leave work out, when all of it took 107: products alone 66 us,
// copies alone 73 (16 TB/s from the L2, 52 bytes a clock into an SM), both without scales 90,
// with scales that are written but not loaded 96.  So one part grows with K: what an SM takes
// in, operands, scales (9% of their bytes: a tile's 256 columns and, in both CTAs, its rows),
// and the hand-over of the latter.  The other is the write-out, some 0.8 us a round of tiles
// whatever K is, although the next tile's products run beside it: without its stores 16384 rows
// to 4096 columns take 20, 26, 48 and 92 us for K = 512, 1024, 2048 and 4096, with them 36, 39,
// 61 and 105, with half of them 27, 33, 57 and 100, with all but not turned 35, 39, 62 and 106.
// A single tile takes 5.5 us with its launch, 64 experts of 768 x 2048 with 8192 rows 21 us (16
// without stores) against 14 of HBM traffic, with 32 rows 8.9 against 3.2.  Four sets of scale
// warps, or fewer rows a tile and more stages, are no faster; two sets take 7% longer.
// Scales written stage by stage took 256 us: every hand-over to the other CTA has a fence
// that a thread's loads, stores and a cluster-wide release wait for, so one hand-over
// serves four stages, three sets of warps take turns, and loads follow it.
#include "bytes.cuh"
#include "groups.cuh"
#include "tensor_core.cuh"
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kTileRows = 224;                // most tokens of a tile
constexpr int kStepBytes = 128;               // of the sum per stage: eight blocks
constexpr int kStages = 5;
constexpr uint32_t kWBytes = 128 * 128, kXBytes = kTileRows / 2 * 128;  // a CTA's share of a stage
constexpr uint32_t kStageBytes = kWBytes + kXBytes;
static_assert(kStageBytes % 1024 == 0 && kXBytes % 1024 == 0, "operands start on whole swizzle atoms");
constexpr int kAhead = 4;                     // stages whose scales are written together
constexpr int kScaleSlots = 3;                // of such scales, each with a set of warps that writes it
constexpr uint32_t kAtom = 512;               // scales of 128 rows and four blocks
constexpr uint32_t kRoleBytes = kAhead * 2 * kAtom;  // of 128 rows in a slot
constexpr int kRoles = 3;                     // weights, tokens 0 .. 127, tokens 128 ..
constexpr uint32_t kSlotBytes = kRoles * kRoleBytes;
constexpr int kWriteWarps = 8;                // two for each 32 lanes of tensor memory, a block of 32 rows each in turn
constexpr int kCopyWarpW = kWriteWarps, kCopyWarpX = kCopyWarpW + 1, kProductWarp = kCopyWarpX + 1, kScaleWarp = kProductWarp + 1;
constexpr int kThreads = (kScaleWarp + kRoles * kScaleSlots) * 32;
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kScaleColumn = 2 * kTileRows, kScaleColumns = 24;

struct Mx4ProductArgs {
    CUtensorMap w;        // boxes of 128 output columns
    CUtensorMap x;        // boxes of 64 rows
    CUtensorMap x_small;  // boxes of 16 rows
    const uint8_t* xs;
    const uint8_t* ws;
    const int32_t* offsets;
    void* y;
    int slots, experts;
    int out, bytes;  // bytes of a row of an operand
    Divisor32 across;  // tiles of 256 output columns
    int blocks;      // scales of a row
    int scale_vec;   // bytes that a load of scales may take: 32, 16, 8 or 1
    bool vec;        // rows of y allow 16-byte stores
};

struct Mx4Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    uint64_t acc_full[2], acc_empty[2];
    int warp_tiles[kThreads / 32];
    uint32_t tmem;
    uint32_t progress;  // stages whose copies are under way, for waits that span many
    int abort;
};

struct Mx4Tile {
    int expert = 0;
    int m0;     // first output column of the pair's 256
    int n0, n;  // rows
    int width;  // rows the products compute
};

__device__ __forceinline__ bool tile_at(const Mx4ProductArgs& g, const int* table, const Group* groups, int t, int tiles,
                                        Mx4Tile& w) {
    if (t >= tiles) return false;
    const int row_tile = int(g.across.quotient(uint32_t(t)));
    const RowTile r = kept_row_tile(groups, g.experts, table, row_tile, w.expert);
    w.expert = uniform(r.expert);
    w.m0 = (t - row_tile * int(g.across.d)) * 256;
    w.n0 = uniform(r.first);
    w.n = uniform(r.count);
    w.width = (w.n + 31) & ~31;
    return true;
}

// Descriptor of an atom of scales: rows of 16 bytes, 8 of them in 128, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3fff) | (uint64_t(1) << 16) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}
// An atom to four columns of tensor memory of each CTA, from its own shared memory.
__device__ __forceinline__ void copy_scales(uint32_t to, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(to),
        "l"(desc)
        : "memory");
}

// Block-scaled instruction descriptor: e2m1 (code 1) both, power-of-two scales, M = 256,
// 64 values of the sum; `id`: the first of the two blocks' bytes within a column.
constexpr uint32_t mx4_desc(uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | (1u << 23) | ((256u >> 4) << 24) | (id << 29);
}
// A stage: four products of 64 values.  ws, xs: the stage's scales in tensor memory, four
// blocks in 4 and in 8 columns.
__device__ __forceinline__ void mma_pair_mx4_4(uint32_t d, uint64_t a, uint64_t b, uint32_t n_bits, uint32_t ws, uint32_t xs,
                                               bool add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t.reg .b32 i, j, u, v;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "or.b32 i, %3, %7;\n\tor.b32 j, %3, %8;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, i, [%4], [%5], p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, j, [%4], [%5], p;\n\t"
        "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\tadd.u32 u, %4, 4;\n\tadd.u32 v, %5, 8;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, i, [u], [v], p;\n\t"
        "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, j, [u], [v], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(n_bits), "r"(ws), "r"(xs), "r"(uint32_t(add)), "n"(mx4_desc(0)), "n"(mx4_desc(2))
        : "memory");
}

// What a scale warp reads: the scales of four stages of each of four rows a lane, which
// lie 32 apart.  The loads are not of the read-only kind: what wrote the scales may have
// ended after this kernel began.
struct ScaleRows {
    const uint8_t* p[4];  // their rows of scales; NULL: none
    const uint8_t* begin;
    const uint8_t* end;   // of all rows
    __device__ __forceinline__ void load(int block, int blocks, int vec, uint32_t (&r)[4][2 * kAhead]) const {
        const int left = blocks - block;  // at least 1
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < 2 * kAhead; ++i) r[j][i] = 0;
            if (p[j] == nullptr) continue;
            const uint8_t* at = p[j] + block;
            if (vec == 32) {  // blocks is a multiple of 32
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                             : "=r"(r[j][0]), "=r"(r[j][1]), "=r"(r[j][2]), "=r"(r[j][3]), "=r"(r[j][4]), "=r"(r[j][5]),
                               "=r"(r[j][6]), "=r"(r[j][7])
                             : "l"(at)
                             : "memory");
            } else if (vec == 16) {  // blocks is a multiple of 16
#pragma unroll
                for (int i = 0; i < kAhead / 2; ++i)
                    if (left > 16 * i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(at + 16 * i);
                        r[j][4 * i] = v.x, r[j][4 * i + 1] = v.y, r[j][4 * i + 2] = v.z, r[j][4 * i + 3] = v.w;
                    }
            } else if (vec == 8) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (left > 8 * i) {
                        const uint2 v = *reinterpret_cast<const uint2*>(at + 8 * i);
                        r[j][2 * i] = v.x, r[j][2 * i + 1] = v.y;
                    }
            } else {
                const int off = int(reinterpret_cast<uintptr_t>(at) & 3);
                uint32_t word[2 * kAhead + 1];
                words_at(at - off, begin, end, word);
#pragma unroll
                for (int i = 0; i < 2 * kAhead; ++i) {
                    const int there = left - 4 * i;  // the next row's scales are not this one's: 0 times NaN is NaN
                    const uint32_t v = __funnelshift_r(word[i], word[i + 1], 8 * off);
                    r[j][i] = there >= 4 ? v : there > 0 ? v & ((1u << (8 * there)) - 1) : 0;
                }
            }
        }
    }
};

// A block of 32 rows by a warp's 32 output columns: a lane holds a column, a register a
// row.  16-bit results are turned in shared memory, pairs of rows in a word, and written
// 16 bytes a lane: eight rows of 64 bytes a store, in place of one.
constexpr int kTurnPitch = 128 + 16;          // of a pair of rows; the step keeps a read's lanes in banks of their own
constexpr int kTurnBytes = 8 * kTurnPitch;
template <typename O>
__device__ __forceinline__ void write_block(unsigned char* turn, O* p, int64_t pitch, int rows, int cols, bool vec,
                                            const uint32_t (&r)[32]) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(O) == 2) {
        if (vec) {
            const int pair = lane / 4, col = lane % 4 * 8;  // a lane's two rows and eight columns
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // of the rows
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    Chunk<O, 2> c;
                    c.set(0, __uint_as_float(r[16 * half + 2 * i]));
                    c.set(1, __uint_as_float(r[16 * half + 2 * i + 1]));
                    *reinterpret_cast<uint32_t*>(turn + i * kTurnPitch + lane * 4) = c.raw;
                }
                __syncwarp();
                const uint4* from = reinterpret_cast<const uint4*>(turn + pair * kTurnPitch + col * 4);
                const uint4 a = from[0], b = from[1];
                __syncwarp();
                const uint4 low = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                             __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
                const uint4 high = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                              __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
                const int row = 16 * half + 2 * pair;
                O* at = p + row * pitch + col;
                if (col < cols) {  // cols is a multiple of 8
                    if (row < rows) *reinterpret_cast<uint4*>(at) = low;
                    if (row + 1 < rows) *reinterpret_cast<uint4*>(at + pitch) = high;
                }
            }
            return;
        }
    }
    if (lane < cols) {
        p += lane;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += pitch)
            if (i < rows) *p = from_float<O>(__uint_as_float(r[i]));
    }
    __syncwarp();
}

template <typename O>
__global__ void __launch_bounds__(kThreads, 1) expert_product_mx4(const __grid_constant__ Mx4ProductArgs g) {
    extern __shared__ unsigned char raw[];
    unsigned char* stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char* slots = stages + kStages * kStageBytes;
    unsigned char* turn = slots + kScaleSlots * kSlotBytes;
    Group* groups = reinterpret_cast<Group*>(turn + kWriteWarps * kTurnBytes);
    int* table = reinterpret_cast<int*>(groups + kMaxExperts);
    __shared__ Mx4Shared sh;
    volatile int* abort_flag = &sh.abort;
    volatile uint32_t* progress = &sh.progress;

    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(cluster_rank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);  // a copying lane per operand
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.scale_full[i], 2 * kRoles);  // both CTAs' scale warps
            mbar_init(&sh.scale_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kWriteWarps);  // of both CTAs
        }
        sh.progress = 0;
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kCopyWarpW && lane == 0) {
        prefetch_map(&g.w);
        prefetch_map(&g.x);
        prefetch_map(&g.x_small);
    }
    if (warp == kProductWarp) tmem_alloc_pair(&sh.tmem, kTmemColumns);
    // Each CTA's barriers and tensor memory are there; the other hears of it while the table is
    // built.  (An arrival with a release behind the table took 1500 clocks.)
    tcgen05_fence_before();
    cluster_arrive_relaxed();
    wait_for_earlier();  // what quantised the rows lets this kernel come this far
    build_tile_table<kTileRows, kThreads>(g.offsets, g.experts, g.slots, table, sh.warp_tiles, KeepGroups<kTileRows>{groups});
    __syncthreads();
    cluster_wait();
    tcgen05_fence_after();
    const uint32_t tmem = uniform(sh.tmem), stage0 = uniform(smem_addr(stages));

    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int tiles = uniform(all_tiles(table[g.experts], int(g.across.d)));
    const int steps = (g.bytes + kStepBytes - 1) / kStepBytes;  // stages of a sum
    bool ok = true;
    if (warp == kCopyWarpW || warp == kCopyWarpX) {
        const bool is_w = warp == kCopyWarpW;
        const uint32_t to = stage0 + (is_w ? 0 : kWBytes);
        const uint32_t full0 = map_to_rank(sh.full, 0);
        uint32_t s = 0, phase = 1, slot = 0, slot_phase = 1;  // the stage and the scales' slot, and their releases' parities
        uint32_t stages_begun = 0;
        Mx4Tile w;
        for (int t = first; ok && tile_at(g, table, groups, t, tiles, w); t += step) {
            const int half = w.width / 2;
            const int m0 = w.m0 + int(rank) * 128, n0 = w.n0 + int(rank) * half;
            const uint32_t mine = is_w ? kWBytes : uint32_t(half) * 128;
            for (int kb = 0; kb < steps; ++kb) {
                ok = warp_wait(&sh.empty[s], phase, abort_flag);
                if (!ok) break;
                const uint32_t bar = full0 + s * 8, dst = to + s * kStageBytes;
                if (rank == 0) elect_arrive_expect_tx(&sh.full[s], 2 * mine);
                if (is_w) {
                    *progress = ++stages_begun;
                    tma_load_3d(dst, &g.w, kb * kStepBytes, m0, w.expert, bar);
                } else {
                    load_rows(dst, &g.x, &g.x_small, kb * kStepBytes, n0, half, bar);
                }
                next_stage<kStages>(s, phase);
                if (kb % kAhead == 0) next_stage<kScaleSlots>(slot, slot_phase);
            }
        }
        // every stage and slot is released in this CTA too before it may leave
        for (int i = 0; ok && i < kStages; ++i) {
            ok = warp_wait(&sh.empty[s], phase, abort_flag);
            next_stage<kStages>(s, phase);
        }
        for (int i = 0; ok && i < kScaleSlots; ++i) {
            ok = warp_wait(&sh.scale_empty[slot], slot_phase, abort_flag);
            next_stage<kScaleSlots>(slot, slot_phase);
        }
    } else if (warp == kProductWarp) {
        if (rank == 0) {
            uint32_t s = 0, phase = 0, slot = 0, slot_phase = 0, acc = 0, turn = 0;  // turn: of the two places in tensor memory
            const uint64_t a0 = operand_desc(stage0, 16, 1024), b0 = operand_desc(stage0 + kWBytes, 16, 1024);
            const uint64_t s0 = scale_desc(uniform(smem_addr(slots)));
            Mx4Tile w, next;
            bool ready = false;  // the next stage was seen full, with its scales and its accumulator
            bool more = tile_at(g, table, groups, first, tiles, w);
            for (int t = first; ok && more; t += step, w = next) {
                next = w;
                more = tile_at(g, table, groups, t + step, tiles, next);
                const uint32_t d = tmem + (acc & 1) * kTileRows, n_bits = uint32_t(w.width >> 3) << 17;
                const bool two = w.width > 128;
                for (int kb = 0; kb < steps; ++kb) {
                    if (!ready) {
                        if (kb == 0) ok = warp_wait(&sh.acc_empty[acc & 1], ((acc >> 1) & 1) ^ 1, abort_flag);
                        if (kb % kAhead == 0) ok = ok && warp_wait<true>(&sh.scale_full[slot], slot_phase, abort_flag);
                        ok = ok && warp_wait(&sh.full[s], phase, abort_flag);
                        if (!ok) break;
                    }
                    tcgen05_fence_after();
                    const uint32_t here = s, at = s * (kStageBytes >> 4), scales = slot;
                    const bool last = kb == steps - 1, last_of_slot = kb % kAhead == kAhead - 1 || last;
                    next_stage<kStages>(s, phase);
                    if (last_of_slot) next_stage<kScaleSlots>(slot, slot_phase);
                    uint32_t looks = 0;
                    if (!last || more) {
                        looks = look(&sh.full[s], phase);
                        if (last_of_slot) looks &= look<true>(&sh.scale_full[slot], slot_phase);
                        if (last) looks &= look(&sh.acc_empty[(acc + 1) & 1], (((acc + 1) >> 1) & 1) ^ 1);
                    }
                    const uint32_t ws = tmem + kScaleColumn + turn * kScaleColumns, xs = ws + 8;
                    const uint64_t from = s0 + scales * (kSlotBytes >> 4) + (kb % kAhead) * 2 * (kAtom >> 4);
                    turn ^= 1;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        copy_scales(ws + q * 4, from + q * (kAtom >> 4));
                        copy_scales(xs + q * 8, from + (kRoleBytes + q * kAtom) / 16);
                        if (two) copy_scales(xs + q * 8 + 4, from + (2 * kRoleBytes + q * kAtom) / 16);
                    }
                    mma_pair_mx4_4(d, a0 + at, b0 + at, n_bits, ws, xs, kb > 0);
                    mma_commit_pair(&sh.empty[here]);
                    if (last_of_slot) mma_commit_pair(&sh.scale_empty[scales]);
                    if (last) mma_commit_pair(&sh.acc_full[acc & 1]);
                    ready = saw(looks);
                }
                ++acc;
            }
        }
    } else if (warp >= kScaleWarp) {
        // A set of a warp a role for each slot.  A fence waits for a thread's loads too, so a warp
        // asks for its next scales behind the hand-over of these: they come while it waits for
        // its slot.
        const int role = (warp - kScaleWarp) % kRoles, slot = (warp - kScaleWarp) / kRoles;
        const uint32_t full = map_to_rank(&sh.scale_full[slot], 0);
        unsigned char* to = slots + slot * kSlotBytes + role * kRoleBytes + lane * 16;
        const int parts = (steps + kAhead - 1) / kAhead;  // slots of a sum
        uint32_t phase = 1;
        int part = slot;
        Mx4Tile w;
        for (int t = first; ok && tile_at(g, table, groups, t, tiles, w); t += step, part -= parts) {
            if (part >= parts) continue;
            ScaleRows rows;
            rows.begin = role == 0 ? g.ws : g.xs;
            rows.end = rows.begin + (role == 0 ? int64_t(g.experts) * g.out : int64_t(g.slots)) * g.blocks;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = (role == 2 ? 128 : 0) + 32 * j + lane;
                if (role == 0) {
                    const int m = w.m0 + int(rank) * 128 + row;
                    rows.p[j] = m < g.out ? g.ws + (int64_t(w.expert) * g.out + m) * g.blocks : nullptr;
                } else {
                    rows.p[j] = row < w.n ? g.xs + int64_t(w.n0 + row) * g.blocks : nullptr;
                }
            }
            for (; part < parts; part += kScaleSlots) {
                uint32_t r[4][2 * kAhead];
                rows.load(part * 8 * kAhead, g.blocks, g.scale_vec, r);
                __syncwarp();
                ok = warp_wait(&sh.scale_empty[slot], phase, abort_flag);
                if (!ok) break;
                phase ^= 1;
#pragma unroll
                for (int q = 0; q < 2 * kAhead; ++q)
                    *reinterpret_cast<uint4*>(to + q * kAtom) = make_uint4(r[0][q], r[1][q], r[2][q], r[3][q]);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(full);
            }
        }
    } else {
        uint32_t acc = 0;
        Mx4Tile w;
        for (int t = first; tile_at(g, table, groups, t, tiles, w); t += step) {
            if (!warp_wait_stages(&sh.acc_full[acc & 1], (acc >> 1) & 1, abort_flag, progress)) break;
            tcgen05_fence_after();
            const uint32_t from = tmem + (uint32_t(warp & 3) << 21) + (acc & 1) * kTileRows;  // lane 32 * (warp % 4)
            const int m = w.m0 + int(rank) * 128 + (warp & 3) * 32;
            O* p = static_cast<O*>(g.y) + int64_t(w.n0) * g.out + m;
            constexpr int kStep = kWriteWarps / 4 * 32;
            // An arrival that nothing waits for could reach a CTA that has left.
            const bool again = t < tiles - 2 * step;
            int c = warp / 4 * 32;
            for (; c < w.n; c += kStep) {
                uint32_t r[32];
                tmem_load32(from + uint32_t(c), r);
                tmem_wait_load(r);
                if (c + kStep >= w.n && again) {
                    tcgen05_fence_before();
                    __syncwarp();
                    elect_arrive_pair(map_to_rank(&sh.acc_empty[acc & 1], 0));
                }
                write_block(turn + warp * kTurnBytes, p + int64_t(c) * g.out, g.out, w.n - c, g.out - m, g.vec, r);
            }
            if (warp / 4 * 32 >= w.n && again) {  // nothing here for the second warp
                __syncwarp();
                elect_arrive_pair(map_to_rank(&sh.acc_empty[acc & 1], 0));
            }
            ++acc;
        }
    }
    __syncwarp();
    if (*abort_flag) let_copies_land();
    tcgen05_fence_before();
    __syncthreads();
    if (*abort_flag) cluster_sync_all();
    else {
        cluster_arrive_relaxed();
        cluster_wait();
    }
    tcgen05_fence_after();
    if (warp == kProductWarp) tmem_dealloc_pair(tmem, kTmemColumns);
}

constexpr size_t kMostSmem = 1024 + kStages * size_t(kStageBytes) + kScaleSlots * kSlotBytes + kWriteWarps * kTurnBytes +
                             kMaxExperts * sizeof(Group) + (kMaxExperts + 1) * 4;
static_assert(kMostSmem <= kMaxDynSmem, "one CTA on an SM");

}  // namespace

uint32_t pipeline_timeouts_mx4() { return read_pipeline_timeouts(); }

cudaError_t launch_expert_matmul_mx4(const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                                     const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                     int64_t experts, int y_type, Scratch scratch, cudaStream_t stream) {
    Matrix mx = matrix_of(x, in / 2, slots, 1, 1), mw = matrix_of(w, in / 2, out, experts, 1);
    Matrix* ms[2] = {&mx, &mw};
    cudaError_t err;
    if (!make_readable(ms, {false, true}, offsets, slots, scratch, stream, &err, true))
        return launch_matmul_mx4_any(x, xs, w, ws, offsets, y, slots, in, out, experts, y_type, stream);
    if (err != cudaSuccess) return err;
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    Mx4ProductArgs g;
    if (!make_map(&g.w, type, mw, kStepBytes, 128, true) || !make_map(&g.x_small, type, mx, kStepBytes, 16, false))
        return cudaErrorInvalidValue;
    g.x = g.x_small;  // half a tile is 64 rows or more only where a tile has more than 96
    if (slots > 96 && !make_map(&g.x, type, mx, kStepBytes, 64, false)) return cudaErrorInvalidValue;
    g.xs = xs;
    g.ws = ws;
    g.offsets = offsets;
    g.y = y;
    g.slots = int(slots);
    g.experts = int(experts);
    g.out = int(out);
    g.across = Divisor32(uint32_t((out + 255) / 256));
    g.bytes = int(in / 2);
    g.blocks = int((in + 31) / 32);
    const uintptr_t at = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws) | uintptr_t(g.blocks);
    g.scale_vec = at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : at % 8 == 0 ? 8 : 1;
    const int y_size = y_type == ROWOPS_F32 ? 4 : 2;
    g.vec = out * y_size % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
    const int64_t tiles = most_row_tiles(slots, experts, kTileRows) * ((out + 255) / 256);
    cudaError_t e = cudaErrorInvalidValue;
    if (tiles >= kMostTiles) return e;  // more than a device's memory holds
    with_type(y_type, [&](auto o) {
        e = launch_pairs<expert_product_mx4<decltype(o)>>(tiles, kThreads, kMostSmem, stream, g, true);
    });
    return e;
}

}  // namespace rowops
