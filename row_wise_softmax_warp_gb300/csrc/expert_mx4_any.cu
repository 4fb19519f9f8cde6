// expert_mx4_any.cu - the experts' product on microscaled 4-bit operands, for every
// alignment.
//
//   y[s][n] = sum_b 2^(xs[s][b] + ws[e][n][b] - 254) sum_{k in block b} xq[s][k] wq[e][n][k]
//
// A block computes 64 x 64 values, a block of 32 of the sum at a time: its bytes are
// widened to fp16, which holds e2m1 exactly, in shared memory; four warps of 32 x 32 use
// mma.sync, and each value's 32 products are multiplied by their power of two in fp32
// before they join its sum.
#include "groups.cuh"
#include "mma_sync.cuh"
#include "quant.cuh"
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kTile = 64;
constexpr int kBlock = 32;         // of the sum, and of a scale
constexpr int kPitch = kBlock + 8;
constexpr int kAnyThreads = 128;   // two for each row of a tile

struct Mx4AnyArgs {
    const uint8_t* x;
    const uint8_t* xs;
    const uint8_t* w;
    const uint8_t* ws;
    const int32_t* offsets;
    void* y;
    int64_t slots, bytes, out;  // bytes: of a row, half its values
    int experts;
};

// Half a row's block: eight bytes of row `row` from `at`; 0 where there are none.
__device__ __forceinline__ void fetch(const uint8_t* p, bool there, int64_t at, int64_t bytes, uint8_t (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = there && at + i < bytes ? __ldg(p + at + i) : uint8_t(0);
}
__device__ __forceinline__ void put(uint16_t* to, const uint8_t (&r)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(r[i], __NV_E2M1);
        *reinterpret_cast<uint32_t*>(to + 2 * i) = uint32_t(h.x) | (uint32_t(h.y) << 16);
    }
}

template <typename O>
__global__ void __launch_bounds__(kAnyThreads) matmul_mx4_any(const Mx4AnyArgs g) {
    __shared__ __align__(16) uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
    __shared__ uint8_t scale[2][kTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wm = (warp >> 1) * 32, wn = (warp & 1) * 32;
    const int gr = lane >> 2, gc = (lane & 3) * 2;
    const int mine = threadIdx.x >> 1, half = threadIdx.x & 1;  // the row and the half that this thread fetches
    const int64_t tiles_n = (g.out + kTile - 1) / kTile, blocks = (g.bytes + 15) / 16;

    for (int64_t t = blockIdx.x;; t += gridDim.x) {
        const int64_t n0 = t % tiles_n * kTile;
        int e, first, count;
        if (!find_row_tile<kTile>(g.offsets, g.experts, int(g.slots), t / tiles_n, e, first, count)) break;
        const bool has_a = mine < count, has_b = n0 + mine < g.out;
        const int64_t a_row = first + mine, b_row = int64_t(e) * g.out + n0 + mine;
        float acc[2][4][4] = {};
        for (int64_t b = 0; b < blocks; ++b) {
            uint8_t ra[8], rb[8];
            fetch(g.x + a_row * g.bytes, has_a, b * 16 + half * 8, g.bytes, ra);
            fetch(g.w + b_row * g.bytes, has_b, b * 16 + half * 8, g.bytes, rb);
            __syncthreads();
            put(&sa[mine][half * 16], ra);
            put(&sb[mine][half * 16], rb);
            if (half == 0) scale[0][mine] = has_a ? g.xs[a_row * blocks + b] : uint8_t(127);
            else scale[1][mine] = has_b ? g.ws[b_row * blocks + b] : uint8_t(127);
            __syncthreads();
            float part[2][4][4] = {};
#pragma unroll
            for (int kk = 0; kk < kBlock; kk += 16) {
                uint32_t fa[2][4], fb[4][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = wm + i * 16 + gr;
                    fa[i][0] = *reinterpret_cast<const uint32_t*>(&sa[r][kk + gc]);
                    fa[i][1] = *reinterpret_cast<const uint32_t*>(&sa[r + 8][kk + gc]);
                    fa[i][2] = *reinterpret_cast<const uint32_t*>(&sa[r][kk + gc + 8]);
                    fa[i][3] = *reinterpret_cast<const uint32_t*>(&sa[r + 8][kk + gc + 8]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = wn + j * 8 + gr;
                    fb[j][0] = *reinterpret_cast<const uint32_t*>(&sb[r][kk + gc]);
                    fb[j][1] = *reinterpret_cast<const uint32_t*>(&sb[r][kk + gc + 8]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816<false>(part[i][j], fa[i], fb[j]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int xc = scale[0][wm + i * 16 + gr + (v >> 1) * 8], wc = scale[1][wn + j * 8 + gc + (v & 1)];
                        const float p = xc == 255 || wc == 255 ? __int_as_float(0x7fffffff) : ldexpf(part[i][j][v], xc + wc - 254);
                        acc[i][j][v] += p;
                    }
        }
        O* y = static_cast<O*>(g.y);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int r = wm + i * 16 + gr + (v >> 1) * 8;
                    const int64_t col = n0 + wn + j * 8 + gc + (v & 1);
                    if (r < count && col < g.out) y[int64_t(first + r) * g.out + col] = from_float<O>(acc[i][j][v]);
                }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_matmul_mx4_any(const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                                  const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                  int64_t experts, int y_type, cudaStream_t stream) {
    const Mx4AnyArgs g{x, xs, w, ws, offsets, y, slots, in / 2, out, int(experts)};
    const int64_t tiles = (slots / kTile + experts) * ((out + kTile - 1) / kTile);  // at most
    with_type(y_type, [&](auto o) {
        matmul_mx4_any<decltype(o)>
            <<<unsigned(tiles < (1 << 20) ? tiles : (1 << 20)), kAnyThreads, 0, stream>>>(g);
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
