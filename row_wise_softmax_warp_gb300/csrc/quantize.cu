// quantize.cu - e4m3 values and one fp32 scale for each block of 128 columns
// of a row (block_rows = 1) or of a 128 x 128 tile (block_rows = 128).
//
//   a = max(max_{finite x in block} |x|, 2^-100),  scale = a / 448,
//   q = e4m3(448 x / a)     (round to nearest even; 448 is the largest e4m3)
//
// The quotient is correctly rounded: for 16-bit x, 448 x is exact in fp32, so a
// value that lies half-way between two e4m3 values is seen as such.  An
// infinite or NaN x becomes e4m3 NaN and does not enter the scale.  2^-100
// keeps the scale of a block of zeros a normal number.
//
// Bound by HBM: reads the input once into registers, writes a byte a value.
// Sixteen lanes hold a row's 128 columns, 8 values each.
#include <cuda_fp8.h>

#include "types.cuh"

namespace rowops {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantGroups = kQuantThreads / 16;
constexpr float kLargest = 448.0f;        // of e4m3
constexpr float kSmallestMax = 0x1p-100f;

// 8 consecutive values, of which `n` are there (the others are 0).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    if constexpr (VEC) {  // n is 0 or 8
        constexpr int V = 16 / int(sizeof(T));
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            Chunk<T, V> c;
            if (n > 0) c.load(p + h * V);
#pragma unroll
            for (int i = 0; i < V; ++i) v[h * V + i] = c.get(i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_float(p[i]) : 0.f;
    }
}

__device__ __forceinline__ float finite_max(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(v[i]);
        if (a < INFINITY) m = fmaxf(m, a);
    }
    return m;
}

// a: the block's maximum.  Values and a are divided by 2^32 where 448 x could overflow.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float a) {
    const float s = a > 0x1p100f ? 0x1p-32f : 1.0f;
    const float d = a * s;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        f.x = fabsf(v[2 * i]) < INFINITY ? __fdiv_rn(kLargest * (v[2 * i] * s), d) : NAN;
        f.y = fabsf(v[2 * i + 1]) < INFINITY ? __fdiv_rn(kLargest * (v[2 * i + 1] * s), d) : NAN;
        w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, int n, uint2 w) {
    if constexpr (VEC) {
        if (n > 0) *reinterpret_cast<uint2*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = uint8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
}

// Sixteen lanes per (row, block of 128 columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows(const T* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, int64_t items,
                  int blocks, int64_t cols) {
    const int64_t item = int64_t(blockIdx.x) * kQuantGroups + (threadIdx.x >> 4);
    const bool there = item < items;  // every lane stays for the shuffles
    const int64_t row = there ? item / blocks : 0;
    const int64_t c = (there ? item % blocks : 0) * 128 + (threadIdx.x & 15) * 8;
    const int n = there ? int(max(int64_t(0), min(int64_t(8), cols - c))) : 0;
    float v[8];
    load8<T, VEC>(x + row * cols + c, n, v);
    const float a = fmaxf(group_max<16>(finite_max(v)), kSmallestMax);
    store8<VEC>(q + row * cols + c, n, quantize8(v, a));
    if (there && (threadIdx.x & 15) == 0) scale[item] = __fdiv_rn(a, kLargest);
}

// One block per 128 x 128 tile; each group of sixteen lanes holds 8 rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_tiles(const T* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, int64_t rows,
                   int64_t cols, int row_blocks, int col_blocks) {
    __shared__ float scratch[kQuantThreads / 32];
    const int64_t tile = blockIdx.x;
    const int64_t batch = tile / (int64_t(row_blocks) * col_blocks);
    const int64_t in = tile % (int64_t(row_blocks) * col_blocks);
    const int64_t r0 = in / col_blocks * 128 + (threadIdx.x >> 4), c = in % col_blocks * 128 + (threadIdx.x & 15) * 8;
    const int nc = int(max(int64_t(0), min(int64_t(8), cols - c)));
    float v[8][8];
    float a = kSmallestMax;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * kQuantGroups;
        load8<T, VEC>(x + (batch * rows + r) * cols + c, r < rows ? nc : 0, v[i]);
        a = fmaxf(a, finite_max(v[i]));
    }
    a = block_max<kQuantThreads>(a, scratch);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * kQuantGroups;
        store8<VEC>(q + (batch * rows + r) * cols + c, r < rows ? nc : 0, quantize8(v[i], a));
    }
    if (threadIdx.x == 0) scale[tile] = __fdiv_rn(a, kLargest);
}

}  // namespace

cudaError_t launch_quantize_blocks(const void* x, uint8_t* q, float* scale, int64_t batches, int64_t rows,
                                   int64_t cols, int64_t block_rows, int x_type, cudaStream_t stream) {
    const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 8 == 0;
    const int blocks = int((cols + 127) / 128);
    with_type(x_type, [&](auto ti) {
        using T = decltype(ti);
        const T* xp = static_cast<const T*>(x);
        if (block_rows == 1) {
            const int64_t items = batches * rows * blocks;
            const unsigned grid = unsigned((items + kQuantGroups - 1) / kQuantGroups);
            if (vec) quantize_rows<T, true><<<grid, kQuantThreads, 0, stream>>>(xp, q, scale, items, blocks, cols);
            else quantize_rows<T, false><<<grid, kQuantThreads, 0, stream>>>(xp, q, scale, items, blocks, cols);
        } else {
            const int row_blocks = int((rows + 127) / 128);
            const unsigned grid = unsigned(batches * row_blocks * blocks);
            if (vec)
                quantize_tiles<T, true>
                    <<<grid, kQuantThreads, 0, stream>>>(xp, q, scale, rows, cols, row_blocks, blocks);
            else
                quantize_tiles<T, false>
                    <<<grid, kQuantThreads, 0, stream>>>(xp, q, scale, rows, cols, row_blocks, blocks);
        }
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
