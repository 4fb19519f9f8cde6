// repack.cu - rows that start on any byte copied to rows that start on 16-byte
// boundaries, so that TMA can read them (an in-width of 773 values of 2 bytes, say).
//
// A warp takes a row; a lane makes 16 bytes of the copy from five aligned 4-byte
// words, shifted together.  Bound by HBM: every byte is read and written once (8 experts of
// 2003 x 1001 fp16 and 8192 rows of 1001, 97 MB: some 16 us of the product's 50).  What lies
// between a row's end and the next boundary is whatever the source holds there; the tensor
// map over the copy ends at the row's true width.
#include "bytes.cuh"
#include "groups.cuh"
#include "launch.h"

namespace rowops {
namespace {

constexpr int kRepackThreads = 256;

// Rows of a warp, one after another: four where there are many (a warp whose rows
// no expert needs costs little then), one where each is a wait of its own.  The product
// with its copies, four against one row a warp: 3606 rows 17.8 and 15.8 us, 24216 56.5 and
// 55.8, 41280 53.3 and 54.1; 2 rows of x and 64 experts, 33090 16.5 and 20.6, 128194 27.1 and 56.0.
// Of rows of one piece of 512 bytes two are on their way together (4-bit products of 65536 x
// 514, with two 61, one or four 65 us; 64 experts of 770 -> 2048 with 8192 rows 56 and 67).
// Rows of 256 bytes or fewer share a warp (840 rows of 87 experts, 118 -> 3088: 69 -> 32 us; 8192
// rows of 64 experts, 200 -> 2048 47 -> 30).
constexpr int kRepackRows = 4;
constexpr int64_t kManyRows = 32768;

struct RepackArgs {
    RepackJob job[2];
    const int32_t* offsets;
    int slots;
    int each;   // passes of a warp
    int lanes;  // of a row: a power of two; short rows share a warp
};

// A pass takes a row, of SHORT ones 32 / lanes, R passes at a time; U pieces of 512 bytes of
// a row that has more are on their way together.
template <int R, int U, bool SHORT = false>
__global__ void __launch_bounds__(kRepackThreads) repack(const RepackArgs g) {
    static_assert(R == 1 || U == 1, "rows of several pieces are taken one at a time");
    let_next_start();
    wait_for_earlier();
    const int lane = threadIdx.x & 31;
    const int per = SHORT ? 32 / g.lanes : 1;
    const int64_t first = (int64_t(blockIdx.x) * (kRepackThreads / 32) + (threadIdx.x >> 5)) * g.each * per + (SHORT ? lane / g.lanes : 0);
    for (int64_t r = first; r < first + g.each * per; r += R * per) {
        const uint8_t *from[R], *begin[R], *end[R];
        uint8_t* to[R];
        int off[R];
        int64_t bytes[R];  // 0: no such row, or not wanted
#pragma unroll
        for (int n = 0; n < R; ++n) {
            const int64_t at = r + n * per;
            const bool second = at >= g.job[0].rows;
            const RepackJob j = second ? g.job[1] : g.job[0];
            const int64_t row = second ? at - g.job[0].rows : at;
            bytes[n] = row < j.rows ? j.row_bytes : 0;
            // a matrix of weights whose expert has no rows is not read later either
            if (bytes[n] != 0 && j.rows_per_expert > 0 && g.offsets != nullptr) {
                const int e = row <= UINT32_MAX ? int(uint32_t(row) / uint32_t(j.rows_per_expert)) : int(row / j.rows_per_expert);
                if (group_rows(g.offsets, e, g.slots).count == 0) bytes[n] = 0;
            }
            begin[n] = static_cast<const uint8_t*>(j.src);
            end[n] = begin[n] + j.rows * j.row_bytes;
            from[n] = begin[n] + row * j.row_bytes;
            off[n] = int(reinterpret_cast<uintptr_t>(from[n]) & 3);
            to[n] = static_cast<uint8_t*>(j.dst) + row * repack_pitch(j.row_bytes);
        }
        for (int64_t c0 = (SHORT ? lane % g.lanes : lane) * 16; c0 < (R == 1 ? bytes[0] : 512); c0 += U * 512) {
            uint32_t w[R][U][5];
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * 512 < bytes[n]) words_at(from[n] - off[n] + c0 + u * 512, begin[n], end[n], w[n][u]);
#pragma unroll
            for (int n = 0; n < R; ++n)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c0 + u * 512 >= bytes[n]) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[n][u][i] = __funnelshift_r(w[n][u][i], w[n][u][i + 1], 8 * off[n]);
                    *reinterpret_cast<uint4*>(to[n] + c0 + u * 512) =
                        make_uint4(w[n][u][0], w[n][u][1], w[n][u][2], w[n][u][3]);
                }
        }
    }
}

}  // namespace

cudaError_t launch_repack(const RepackJob* jobs, int n, const int32_t* offsets, int64_t slots, cudaStream_t stream,
                          bool early) {
    RepackArgs g = {};
    int64_t rows = 0;
    for (int i = 0; i < n; ++i) {
        g.job[i] = jobs[i];
        rows += jobs[i].rows;
    }
    g.offsets = offsets;
    g.slots = int(slots);
    const int64_t widest = jobs[0].row_bytes > jobs[n - 1].row_bytes ? jobs[0].row_bytes : jobs[n - 1].row_bytes;
    g.lanes = 32;
    while (g.lanes > 1 && widest <= g.lanes / 2 * 16) g.lanes /= 2;
    const int64_t passes = (rows + 32 / g.lanes - 1) / (32 / g.lanes);
    g.each = passes >= kManyRows ? kRepackRows : 1;
    const int64_t per = kRepackThreads / 32 * g.each;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(unsigned((passes + per - 1) / per));
    cfg.blockDim = dim3(kRepackThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    cudaError_t e;
    if (widest > 512) e = cudaLaunchKernelEx(&cfg, repack<1, 4>, g);
    else if (g.lanes == 32) e = g.each == 1 ? cudaLaunchKernelEx(&cfg, repack<1, 1>, g) : cudaLaunchKernelEx(&cfg, repack<2, 1>, g);
    else e = g.each == 1 ? cudaLaunchKernelEx(&cfg, repack<1, 1, true>, g) : cudaLaunchKernelEx(&cfg, repack<2, 1, true>, g);
    note_launches(1);
    return e;
}

}  // namespace rowops
