// expert_matmul_any.cu - the experts' matrix products for every alignment.
//
// The tcgen05 kernels (expert_matmul.cu, expert_fp8.cu) read rows that start on
// 16-byte boundaries; others (of 773 values of 2 bytes, say) are copied to such
// boundaries in the caller's workspace first (repack.cu).  This kernel takes them as
// they are where that workspace is missing or too small: 8192 rows of 8 experts, 1001 ->
// 2003: 395 us, against 56 with the copies.
//
//   kRows        y[s][n]  = sum_k x[s][k] w[e][n][k]      rows s of expert e
//   kRowsT       y[s][n]  = sum_k x[s][k] w[e][k][n]
//   kWeights     dw[e][m][n] = sum_{s of e} dy[s][m] x[s][n]
//
// A block computes 64 x 64 values from steps of 32 along the sum, staged in
// shared memory with the next step's values already in registers; four warps
// of 32 x 32 use mma.sync (m16n8k16, fp32 accumulators).  e4m3 operands are
// widened to fp16, which holds them exactly, and each 128 of the sum are
// multiplied by their scales in fp32 before they join the total.
#include <cuda_fp8.h>

#include "groups.cuh"
#include "types.cuh"

namespace rowops {
namespace {

enum Form { kRows, kRowsT, kWeights };

constexpr int kTile = 64;
constexpr int kStep = 32;
constexpr int kPitch = kStep + 8;
constexpr int kAnyThreads = 128;
constexpr int kPerThread = kTile * kStep / kAnyThreads;

// A matrix operand as (row, k) -> element with two strides, one of which is 1.
template <typename S>
struct Operand {
    const S* p;
    int64_t row_stride, k_stride;
    int64_t rows, ks;  // what is there; the rest reads as 0
};

__device__ __forceinline__ uint16_t bits_of(__half v) { return __half_as_ushort(v); }
__device__ __forceinline__ uint16_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint16_t bits_of(__nv_fp8_e4m3 v) {
    return __half_as_ushort(__half(__nv_cvt_fp8_to_halfraw(v.__x, __NV_E4M3)));
}

template <typename S>
__device__ __forceinline__ void place(int i, bool k_first, int& row, int& k) {
    const int at = threadIdx.x + i * kAnyThreads;
    if (k_first) {
        k = at % kStep;
        row = at / kStep;
    } else {
        row = at % kTile;
        k = at / kTile;
    }
}

template <typename S>
__device__ __forceinline__ void fetch(const Operand<S>& o, int64_t k0, uint16_t (&r)[kPerThread]) {
    const bool k_first = o.k_stride == 1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        int row, k;
        place<S>(i, k_first, row, k);
        r[i] = row < o.rows && k0 + k < o.ks ? bits_of(o.p[row * o.row_stride + (k0 + k) * o.k_stride]) : uint16_t(0);
    }
}

template <typename S>
__device__ __forceinline__ void put(const Operand<S>& o, uint16_t (*sh)[kPitch], const uint16_t (&r)[kPerThread]) {
    const bool k_first = o.k_stride == 1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        int row, k;
        place<S>(i, k_first, row, k);
        sh[row][k] = r[i];
    }
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

struct AnyArgs {
    const void* a;           // x, or dy (kWeights)
    const void* b;           // w, or x (kWeights)
    const float* a_scale;    // e4m3 only: [slots][ceil(in / 128)]
    const float* b_scale;    //            [experts][ceil(out / 128)][ceil(in / 128)]
    const int32_t* offsets;
    void* c;
    int64_t slots, in, out;  // kWeights: dw is out x in
    int experts;
};

// S: operand type, O: output type.
template <typename S, typename O, Form FORM>
__global__ void __launch_bounds__(kAnyThreads) matmul_any(const AnyArgs g) {
    constexpr bool kFp8 = sizeof(S) == 1;
    constexpr bool kBf16 = std::is_same<S, __nv_bfloat16>::value;
    __shared__ __align__(16) uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wm = (warp >> 1) * 32, wn = (warp & 1) * 32;
    const int gr = lane >> 2, gc = (lane & 3) * 2;
    const int64_t ncols = FORM == kWeights ? g.in : g.out;  // columns of c
    const int64_t tiles_n = (ncols + kTile - 1) / kTile;
    const int64_t tiles_m = FORM == kWeights ? (g.out + kTile - 1) / kTile : 0;

    for (int64_t t = blockIdx.x;; t += gridDim.x) {
        const int64_t n0 = t % tiles_n * kTile;
        int e, first, count;
        int64_t m0;
        if constexpr (FORM == kWeights) {
            const int64_t row = t / tiles_n;
            e = int(row / tiles_m);
            if (e >= g.experts) break;
            m0 = row % tiles_m * kTile;
            const RowRange r = group_rows(g.offsets, e, int(g.slots));
            first = r.first;
            count = r.count;
        } else {
            if (!find_row_tile<kTile>(g.offsets, g.experts, int(g.slots), t / tiles_n, e, first, count)) break;
            m0 = first;
        }
        Operand<S> a, b;
        int64_t sum;  // length of the sum
        int64_t rows;  // rows of c in this tile
        if constexpr (FORM == kWeights) {
            sum = count;
            rows = min(int64_t(kTile), g.out - m0);
            a = {static_cast<const S*>(g.a) + int64_t(first) * g.out + m0, 1, g.out, rows, sum};
            b = {static_cast<const S*>(g.b) + int64_t(first) * g.in + n0, 1, g.in, g.in - n0, sum};
        } else {
            sum = g.in;
            rows = count;
            a = {static_cast<const S*>(g.a) + m0 * g.in, g.in, 1, rows, sum};
            const S* w = static_cast<const S*>(g.b) + int64_t(e) * g.in * g.out;
            if constexpr (FORM == kRows) b = {w + n0 * g.in, g.in, 1, g.out - n0, sum};
            else b = {w + n0, 1, g.out, g.out - n0, sum};
        }

        float acc[2][4][4] = {}, part[2][4][4] = {};
        uint16_t ra[kPerThread], rb[kPerThread];
        fetch(a, 0, ra);
        fetch(b, 0, rb);
        for (int64_t k0 = 0; k0 < sum; k0 += kStep) {
            __syncthreads();
            put(a, sa, ra);
            put(b, sb, rb);
            __syncthreads();
            if (k0 + kStep < sum) {
                fetch(a, k0 + kStep, ra);
                fetch(b, k0 + kStep, rb);
            }
#pragma unroll
            for (int kk = 0; kk < kStep; kk += 16) {
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
                    for (int j = 0; j < 4; ++j) mma16816<kBf16>(kFp8 ? part[i][j] : acc[i][j], fa[i], fb[j]);
            }
            if constexpr (kFp8) {
                if ((k0 + kStep) % 128 != 0 && k0 + kStep < sum) continue;
                const int64_t kb = k0 / 128, kbs = (g.in + 127) / 128;
                const float ws = g.b_scale[(e * ((g.out + 127) / 128) + n0 / 128) * kbs + kb];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = wm + i * 16 + gr + h * 8;
                        const float s = r < rows ? g.a_scale[(m0 + r) * kbs + kb] * ws : 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                acc[i][j][h * 2 + v] = fmaf(part[i][j][h * 2 + v], s, acc[i][j][h * 2 + v]);
                                part[i][j][h * 2 + v] = 0.f;
                            }
                    }
            }
        }
        const int64_t c_row0 = FORM == kWeights ? int64_t(e) * g.out + m0 : m0;
        O* c = static_cast<O*>(g.c);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int r = wm + i * 16 + gr + (v >> 1) * 8;
                    const int64_t col = n0 + wn + j * 8 + gc + (v & 1);
                    if (r < rows && col < ncols) c[(c_row0 + r) * ncols + col] = from_float<O>(acc[i][j][v]);
                }
        __syncthreads();
    }
}

template <typename S, typename O, Form FORM>
cudaError_t go(const AnyArgs& g, cudaStream_t stream) {
    const int64_t ncols = FORM == kWeights ? g.in : g.out;
    const int64_t row_tiles = FORM == kWeights ? int64_t(g.experts) * ((g.out + kTile - 1) / kTile)
                                               : g.slots / kTile + g.experts;  // at most
    const int64_t tiles = row_tiles * ((ncols + kTile - 1) / kTile);
    matmul_any<S, O, FORM><<<unsigned(tiles < (1 << 20) ? tiles : (1 << 20)), kAnyThreads, 0, stream>>>(g);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_matmul_any(const void* x, const void* w, const int32_t* offsets, void* y, int64_t slots,
                              int64_t in, int64_t out, int64_t experts, bool transposed, int dtype,
                              cudaStream_t stream) {
    const AnyArgs g{x, w, nullptr, nullptr, offsets, y, slots, in, out, int(experts)};
    if (dtype == ROWOPS_F16)
        return transposed ? go<__half, __half, kRowsT>(g, stream) : go<__half, __half, kRows>(g, stream);
    return transposed ? go<__nv_bfloat16, __nv_bfloat16, kRowsT>(g, stream)
                      : go<__nv_bfloat16, __nv_bfloat16, kRows>(g, stream);
}

cudaError_t launch_matmul_wgrad_any(const void* dy, const void* x, const int32_t* offsets, void* dw, int64_t slots,
                                    int64_t in, int64_t out, int64_t experts, int dtype, int dw_type,
                                    cudaStream_t stream) {
    const AnyArgs g{dy, x, nullptr, nullptr, offsets, dw, slots, in, out, int(experts)};
    if (dtype == ROWOPS_F16)
        return dw_type == ROWOPS_F32 ? go<__half, float, kWeights>(g, stream) : go<__half, __half, kWeights>(g, stream);
    return dw_type == ROWOPS_F32 ? go<__nv_bfloat16, float, kWeights>(g, stream)
                                 : go<__nv_bfloat16, __nv_bfloat16, kWeights>(g, stream);
}

cudaError_t launch_matmul_fp8_any(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                                  const int32_t* offsets, void* y, int64_t slots, int64_t in, int64_t out,
                                  int64_t experts, int y_type, cudaStream_t stream) {
    const AnyArgs g{x, w, x_scale, w_scale, offsets, y, slots, in, out, int(experts)};
    cudaError_t e = cudaErrorInvalidValue;
    with_type(y_type, [&](auto o) { e = go<__nv_fp8_e4m3, decltype(o), kRows>(g, stream); });
    return e;
}

}  // namespace rowops
