// tensor_core.cuh - tcgen05 and tiled TMA in clusters of two CTAs (sm_103a).
//
// The two CTAs of a cluster (SMs of one TPC) work on one 256-row tile: CTA r
// holds rows r * 128 .. of operand A, half the columns of operand B, and rows
// r * 128 .. of the accumulator in its tensor memory.  CTA 0 issues the
// matrix instructions for both.  Operand tiles lie in shared memory in rows of
// 128 bytes with the 128-byte swizzle, as TMA writes them.
#pragma once

#include <cuda.h>

#include <atomic>

#include "launch.h"
#include "pipeline.cuh"

namespace rowops {
namespace {

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(slot)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

// 32 columns of the warp's 32 lanes: lane i of the warp gets row i.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// The registers pass through the wait, so no use of them moves before it.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// ----------------------------------------------------------- matrix products

// Shared-memory operand descriptor, 128-byte swizzle.  K-major (rows of 64
// 16-bit or 128 8-bit values along the sum): `stride` is the distance of 8-row
// groups, `lead` unused.  MN-major (rows of 64 values along M or N): `stride`
// is the distance of groups of 8 along the sum, `lead` that of 64-value columns.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return uint64_t((addr >> 4) & 0x3fff) | (uint64_t((lead >> 4) & 0x3fff) << 16) |
           (uint64_t((stride >> 4) & 0x3fff) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: fp32 accumulators, operand format codes, M = 256.
constexpr uint32_t instr_desc(uint32_t format, bool a_mn, bool b_mn) {
    return (1u << 4) | (format << 7) | (format << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           ((256u >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_n(uint32_t desc, int n) { return desc | (uint32_t(n >> 3) << 17); }

// The products below are called by a whole warp, of which one lane issues them
// (the same each time).  The elected lane's predicate, and operands that the
// compiler sees to be alike in all lanes, keep descriptors in uniform registers;
// from a branch of one lane each product took about 95 clocks to issue, a stage
// of four 760 with its barriers, against 512 in which the tensor cores do them.
__device__ __forceinline__ void mma_pair_16bit(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(uint32_t(add))
        : "memory");
}
// Four in a row, whose operands lie NEXT_A and NEXT_B (in units of 16 bytes) apart;
// all but the first add.
#define ROWOPS_MMA_PAIR_4(KIND)                                                                              \
    asm volatile(                                                                                            \
        "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t" \
        "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], %1, %2, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"       \
        "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"                                                      \
        "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %3, p;\n\t"                                  \
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"                                                        \
        "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %3, p;\n\t"                                  \
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"                                                        \
        "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %3, p;\n}\n" ::"r"(d),                        \
        "l"(a), "l"(b), "r"(desc), "r"(uint32_t(add)), "n"(NEXT_A), "n"(NEXT_B)                              \
        : "memory")
template <int NEXT_A, int NEXT_B>
__device__ __forceinline__ void mma_pair_16bit_4(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    ROWOPS_MMA_PAIR_4("f16");
}
template <int NEXT_A, int NEXT_B>
__device__ __forceinline__ void mma_pair_8bit_4(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    ROWOPS_MMA_PAIR_4("f8f6f4");
}
#undef ROWOPS_MMA_PAIR_4
// Arrives on the barrier at this offset in both CTAs when every product issued so far is done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
            smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
}

// ---------------------------------------------------------- tiled TMA, barriers

// Polls of a wait: a poll takes 35 clocks on an idle SM and some 280 under the tensor
// cores' traffic, so a wait runs out after 0.07 to some 0.6 s.
constexpr uint32_t kQuickPolls = 1u << 22;

// Called by a whole warp; the elected lane acts.
__device__ __forceinline__ void elect_arrive(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void elect_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(smem_addr(bar)),
        "r"(bytes)
        : "memory");
}

// `bar`: shared::cluster address of a barrier of either CTA.  Called by a whole warp.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// `rows` (a multiple of 16) rows of 128 bytes, in as few copies as boxes of 64 and
// of 16 rows allow: a copy takes some 60 clocks to issue, seven of 16 rows nearly
// a stage's time.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* box64, const CUtensorMap* box16, int x, int y,
                                          int rows, uint32_t bar) {
    int i = 0;
    for (; i + 64 <= rows; i += 64) tma_load_2d(dst + i * 128, box64, x, y + i, bar);
    for (; i < rows; i += 16) tma_load_2d(dst + i * 128, box16, x, y + i, bar);
}
// The next place of a ring of N, and the parity there.
template <int N>
__device__ __forceinline__ void next_stage(uint32_t& s, uint32_t& phase) {
    if (++s == N) {
        s = 0;
        phase ^= 1;
    }
}
// A value that every lane of the warp holds, as lane 0 has it.  What decides a
// warp's role goes through it: in code that the compiler takes to be divergent, uniform
// registers are out of its reach, and a stage's copies and products took twice as
// long to issue (32768 rows, 16 experts, 2048 -> 4096 bf16: 326 -> 301 us; one tile of
// 4096: 21.5 -> 15.2 us).
template <typename T>
__device__ __forceinline__ T uniform(T v) {
    return __shfl_sync(kFullMask, v, 0);
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}
// Arrival on a barrier of either CTA that hands over tensor memory: the tcgen05
// fences around it order the accesses.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void elect_arrive_pair(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.shared::cluster.b64 _, [%0];\n}\n" ::"r"(bar)
        : "memory");
}
// Arrival that also releases this thread's shared-memory writes to the other CTA.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
}
// Orders this thread's shared-memory writes before later reads by TMA and tcgen05.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// Gives copies and products in flight time to land before an aborted kernel leaves (about a millisecond).
__device__ __forceinline__ void let_copies_land() {
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// Polls of a whole warp: one lane polls and a vote tells the others, so the compiler
// sees one answer for all.  No suspend hint: between two stages of products the wait's
// own latency is what counts.  The acquire is the CTA's: TMA's and tcgen05's
// arrivals order what they did.
//
// What this and look() rely on: the whole warp arrives converged (roles, tiles and
// answers of waits are the same in all lanes), so elect.sync with a full mask picks one
// lane; p is false before the elected lane's instruction, so the others read a value that
// was set; the barrier lies in this CTA's shared memory, on 8 bytes, and was initialised
// before the cluster's first synchronisation; the parity is 0 or 1; and the instructions
// take their documented operands alone.  A form with the suspend hint as a fourth operand
// under the elected lane's predicate ended in an illegal instruction and is not used.
enum class Polled { kDone, kAborted, kRanOut };
__device__ __forceinline__ Polled warp_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t polls) {
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (__any_sync(kFullMask, done)) {
            __syncwarp();
            return Polled::kDone;
        }
        if (__any_sync(kFullMask, *abort_flag)) return Polled::kAborted;
    }
    return Polled::kRanOut;
}
// Bounded wait of a whole warp; false (after raising the abort) on timeout or abort.
// For what comes after a stage's or a tile's writing at the latest.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const Polled p = warp_poll(bar, parity, abort_flag, kQuickPolls);
    if (p == Polled::kRanOut && (threadIdx.x & 31) == 0) raise_abort(abort_flag);
    return p == Polled::kDone;
}
// For what comes after a whole sum, or several, which may take seconds: the polls
// start again as long as `progress` moves, which a copying warp of the same CTA counts
// up a stage.  Bounded, as there are so many stages and no more.
__device__ __forceinline__ bool warp_wait_stages(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                 const volatile uint32_t* progress, uint32_t polls = kQuickPolls) {
    for (uint32_t seen = ~0u;;) {  // looked at only when the polls have run out
        const Polled p = warp_poll(bar, parity, abort_flag, polls);
        if (p != Polled::kRanOut) return p == Polled::kDone;
        const uint32_t now = uniform(*progress);
        if (now == seen) break;
        seen = now;
    }
    if ((threadIdx.x & 31) == 0) raise_abort(abort_flag);
    return false;
}
// A look at barriers without waiting: under the tensor cores' traffic one takes some
// 280 clocks (55 on an idle SM), so a loop looks at the next stage's before it
// works on this one's and asks for the answer, saw(), afterwards.  The whole warp.
__device__ __forceinline__ uint32_t look(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done;
}
__device__ __forceinline__ bool saw(uint32_t looks) {
    const bool all = __any_sync(kFullMask, looks);
    __syncwarp();
    return all;
}
// With a cluster-wide acquire, for what the other CTA wrote by itself.
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const bool ok = __all_sync(kFullMask, mbar_wait_cluster(bar, parity, abort_flag));
    if (!ok && (threadIdx.x & 31) == 0) raise_abort(abort_flag);
    return ok;
}

// ------------------------------------------------------------------ host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled tensor_map_encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(p) : nullptr;
    }();
    return fn;
}

// An operand that TMA can read: rows of `width` values of `size` bytes, `pitch`
// bytes apart, `height` of them, `depth` times.
struct Matrix {
    const void* base;
    int64_t width, height, depth, pitch;
    int size;
};
inline Matrix matrix_of(const void* base, int64_t width, int64_t height, int64_t depth, int size) {
    return {base, width, height, depth, width * size, size};
}
inline bool tma_reads(const Matrix& m) { return m.pitch % 16 == 0 && reinterpret_cast<uintptr_t>(m.base) % 16 == 0; }

// Copies the operands that TMA cannot read into scratch memory and points them
// there; false where there is too little of it.  by_expert: the operand holds a
// matrix an expert.
inline bool make_readable(Matrix* (&ms)[2], const bool (&by_expert)[2], const int32_t* offsets, int64_t slots,
                          Scratch scratch, cudaStream_t stream, cudaError_t* err) {
    RepackJob jobs[2];
    int n = 0;
    *err = cudaSuccess;
    for (int i = 0; i < 2; ++i) {
        Matrix& m = *ms[i];
        if (tma_reads(m)) continue;
        const int64_t rows = m.height * m.depth, bytes = m.width * m.size;
        void* dst = scratch.take(repack_bytes(rows, bytes));
        if (dst == nullptr) return false;
        jobs[n++] = {m.base, dst, rows, bytes, by_expert[i] ? m.height : 0};
        m.base = dst;
        m.pitch = repack_pitch(bytes);
    }
    if (n > 0) *err = launch_repack(jobs, n, offsets, slots, stream);
    return true;
}

// A tensor map over m (3D where it has a depth), read in boxes of box_x x box_y
// values with the 128-byte swizzle; values outside read as 0.
inline bool make_map(CUtensorMap* map, CUtensorMapDataType type, const Matrix& m, int box_x, int box_y, bool three) {
    const EncodeTiled encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[3] = {cuuint64_t(m.width), cuuint64_t(m.height), cuuint64_t(m.depth)};
    const cuuint64_t strides[2] = {cuuint64_t(m.pitch), cuuint64_t(m.pitch * m.height)};
    const cuuint32_t box[3] = {cuuint32_t(box_x), cuuint32_t(box_y), 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return encode(map, type, three ? 3 : 2, const_cast<void*>(m.base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of two of `kernel` that the current device runs at once (0 if
// unknown); the first call on a device also allows the kernel its shared memory.
template <auto kernel>
int resident_pairs(int threads, size_t smem) {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64)
        if (const int c = cached[dev].load(std::memory_order_relaxed)) return c;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <auto kernel, typename A>
cudaError_t launch_pairs(int64_t pairs, int threads, size_t smem, cudaStream_t stream, const A& args) {
    const int resident = resident_pairs<kernel>(threads, smem);
    if (resident <= 0) {
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? cudaErrorInvalidConfiguration : e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.gridDim = dim3(2 * unsigned(pairs < resident ? pairs : resident));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    note_launches(1);
    return e;
}

}  // namespace
}  // namespace rowops
