// repack.cu - rows that start on any byte copied to rows that start on 16-byte
// boundaries, so that TMA can read them (an in-width of 773 values of 2 bytes, say).
//
// A warp takes a row; a lane makes 16 bytes of the copy from five aligned 4-byte
// words, shifted together.  Bound by HBM: every byte is read and written once (8 experts of 2003 x
// 1001 fp16 and 8192 rows of 1001: 97 MB in about 23 us with its launch).  What lies between a
// row's end and the next boundary is whatever the source holds there; the tensor
// map over the copy ends at the row's true width.
#include "groups.cuh"
#include "launch.h"

namespace rowops {
namespace {

constexpr int kRepackThreads = 256;

// Rows of a warp, one after another: four where there are many (a warp whose rows
// no expert needs costs little then), one where each is a wait of its own.  The product
// with its copies, four against one row a warp: 3606 rows 17.8 and 15.8 us, 24216 56.5 and
// 55.8, 41280 53.3 and 54.1; 2 rows of x and 64 experts, 33090 16.5 and 20.6, 128194 27.1 and 56.0.
constexpr int kRepackRows = 4;
constexpr int64_t kManyRows = 32768;

struct RepackArgs {
    RepackJob job[2];
    const int32_t* offsets;
    int slots;
    int each;  // rows of a warp
};

// The aligned word at `at`, of whose bytes those in [begin, end) are there.
__device__ __forceinline__ uint32_t word_at(const uint8_t* at, const uint8_t* begin, const uint8_t* end) {
    if (at >= begin && at + 4 <= end) return __ldg(reinterpret_cast<const uint32_t*>(at));
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i)
        if (at + i >= begin && at + i < end) w |= uint32_t(at[i]) << (8 * i);
    return w;
}

__global__ void __launch_bounds__(kRepackThreads) repack(const RepackArgs g) {
    const int lane = threadIdx.x & 31;
    const int64_t first = (int64_t(blockIdx.x) * (kRepackThreads / 32) + (threadIdx.x >> 5)) * g.each;
    for (int64_t r = first; r < first + g.each; ++r) {
        const bool second = r >= g.job[0].rows;
        const RepackJob& j = g.job[second];
        const int64_t row = second ? r - g.job[0].rows : r;
        if (row >= j.rows) return;
        // a matrix of weights whose expert has no rows is not read later either
        if (j.rows_per_expert > 0 && g.offsets != nullptr &&
            group_rows(g.offsets, int(row / j.rows_per_expert), g.slots).count == 0)
            continue;
        const uint8_t* begin = static_cast<const uint8_t*>(j.src);
        const uint8_t* end = begin + j.rows * j.row_bytes;
        const uint8_t* from = begin + row * j.row_bytes;
        const int off = int(reinterpret_cast<uintptr_t>(from) & 3);
        from -= off;
        uint8_t* to = static_cast<uint8_t*>(j.dst) + row * repack_pitch(j.row_bytes);
        constexpr int U = 4;
        for (int64_t c0 = lane * 16; c0 < j.row_bytes; c0 += U * 512) {
            uint32_t w[U][5];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 512 < j.row_bytes)
#pragma unroll
                    for (int i = 0; i < 5; ++i) w[u][i] = word_at(from + c0 + u * 512 + 4 * i, begin, end);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * 512 >= j.row_bytes) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[u][i] = __funnelshift_r(w[u][i], w[u][i + 1], 8 * off);
                *reinterpret_cast<uint4*>(to + c0 + u * 512) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_repack(const RepackJob* jobs, int n, const int32_t* offsets, int64_t slots, cudaStream_t stream) {
    RepackArgs g = {};
    int64_t rows = 0;
    for (int i = 0; i < n; ++i) {
        g.job[i] = jobs[i];
        rows += jobs[i].rows;
    }
    g.offsets = offsets;
    g.slots = int(slots);
    g.each = rows >= kManyRows ? kRepackRows : 1;
    const int64_t per = kRepackThreads / 32 * g.each;
    repack<<<unsigned((rows + per - 1) / per), kRepackThreads, 0, stream>>>(g);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
