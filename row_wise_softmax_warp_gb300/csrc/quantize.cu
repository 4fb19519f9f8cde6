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
// Sixteen lanes hold a row's 128 columns, 8 values each; a thread has several
// such loads on their way at once.  At 6.8 TB/s a bf16 value (3 bytes with the one
// written) may take an SM's lanes some 17 instructions, so the quotients come from one
// reciprocal a block.  16384 x 4096 bf16: 35 us by rows; 4096 x 4096 by tiles: 14.2 us,
// whose loads, maximum and stores follow one another in each block of threads.  Rows
// that are no multiple of 8 values are read value by value (8192 x 1001: 10.5 us, x 1000: 6.4).
#include "quant.cuh"
#include "types.cuh"

namespace rowops {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantGroups = kQuantThreads / 16;

// 8 consecutive values, of which `n` are there (the others are 0), as loaded:
// widened to fp32 only when they are used, so loads on their way take few registers.
template <typename T, bool VEC>
struct Eight;
template <typename T>
struct Eight<T, true> {  // n is 0 or 8
    static constexpr int V = 16 / int(sizeof(T));
    Chunk<T, V> c[8 / V];
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n > 0)
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) c[h].load(p + h * V);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c[i / V].get(i % V);
    }
};
template <typename T>
struct Eight<T, false> {
    float f[8];
    __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? to_float(p[i]) : 0.f;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
};

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

// Sixteen lanes per (row, block of 128 columns); a block of threads takes
// kQuantGroups * ITEMS of them in a run, its groups side by side.
// FULL: rows are whole blocks, so a block's number gives its place.
template <typename T, bool VEC, bool FULL, int ITEMS>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows(const T* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, uint32_t items,
                  uint32_t blocks, uint32_t cols) {
    const uint32_t first = blockIdx.x * (kQuantGroups * ITEMS) + (threadIdx.x >> 4);
    Eight<T, VEC> in[ITEMS];
    int64_t at[ITEMS];
    int n[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {  // every lane stays for the shuffles
        const uint32_t item = first + j * kQuantGroups, c0 = (threadIdx.x & 15) * 8;
        if constexpr (FULL) {
            at[j] = int64_t(item) * 128 + c0;
            n[j] = item < items ? 8 : 0;
        } else {
            const uint32_t row = item / blocks, c = (item - row * blocks) * 128 + c0;
            at[j] = int64_t(row) * cols + c;
            n[j] = item < items && c < cols ? int(min(cols - c, 8u)) : 0;
        }
        in[j].load(x + at[j], n[j]);
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        float v[8];
        in[j].get(v);
        float a = group_max<16>(largest(v));
        if (__any_sync(kFullMask, a == INFINITY)) a = group_max<16>(largest_finite(v));
        a = fmaxf(a, kSmallestMax);
        store8<VEC>(q + at[j], n[j], quantize8(v, Divisor(a)));
        const uint32_t item = first + j * kQuantGroups;
        if (item < items && (threadIdx.x & 15) == 0) scale[item] = scale_of(a);
    }
}

// One block per 128 x 128 tile; each group of sixteen lanes holds kTileRows rows.
constexpr int kTileThreads = 256;
constexpr int kTileRows = 128 * 16 / kTileThreads;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads)
    quantize_tiles(const T* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, int64_t rows,
                   int64_t cols, int row_blocks, int col_blocks) {
    __shared__ float scratch[kTileThreads / 32];
    const int64_t tile = blockIdx.x;
    const int64_t batch = tile / (int64_t(row_blocks) * col_blocks);
    const int64_t place = tile % (int64_t(row_blocks) * col_blocks);
    const int64_t r0 = place / col_blocks * 128 + (threadIdx.x >> 4), c = place % col_blocks * 128 + (threadIdx.x & 15) * 8;
    const int nc = int(max(int64_t(0), min(int64_t(8), cols - c)));
    Eight<T, VEC> in[kTileRows];
    float a = 0.f, v[8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const int64_t r = r0 + i * (kTileThreads / 16);
        in[i].load(x + (batch * rows + r) * cols + c, r < rows ? nc : 0);
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        in[i].get(v);
        a = fmaxf(a, largest(v));
    }
    a = block_max<kTileThreads>(a, scratch);
    if (a == INFINITY) {  // the same for every thread
        a = 0.f;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            in[i].get(v);
            a = fmaxf(a, largest_finite(v));
        }
        a = block_max<kTileThreads>(a, scratch);
    }
    a = fmaxf(a, kSmallestMax);
    const Divisor over(a);
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const int64_t r = r0 + i * (kTileThreads / 16);
        in[i].get(v);
        store8<VEC>(q + (batch * rows + r) * cols + c, r < rows ? nc : 0, quantize8(v, over));
    }
    if (threadIdx.x == 0) scale[tile] = scale_of(a);
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
            auto go = [&](auto kernel, int each) {
                const int64_t per = int64_t(kQuantGroups) * each;
                kernel<<<unsigned((items + per - 1) / per), kQuantThreads, 0, stream>>>(
                    xp, q, scale, uint32_t(items), uint32_t(blocks), uint32_t(cols));
            };
            // Blocks of threads of one item a group fill more SMs where there are few (one
            // against four items, bf16 of 768 and 4096 columns: 1536 items 1.62 and 2.07 us, 9600
            // 2.07 and 2.47); many are alike or slightly faster with four loads on their way
            // (49152: 6.03 and 6.08 us, 76800: 8.10 and 7.91).
            const bool few = items < 64 * int64_t(sm_count()) * kQuantGroups / 16;
            if (vec && few) go(quantize_rows<T, true, false, 1>, 1);
            else if (vec && cols % 128 == 0) go(quantize_rows<T, true, true, 4>, 4);
            else if (vec) go(quantize_rows<T, true, false, 4>, 4);
            else go(quantize_rows<T, false, false, 1>, 1);
        } else {
            const int row_blocks = int((rows + 127) / 128);
            const unsigned grid = unsigned(batches * row_blocks * blocks);
            if (vec)
                quantize_tiles<T, true>
                    <<<grid, kTileThreads, 0, stream>>>(xp, q, scale, rows, cols, row_blocks, blocks);
            else
                quantize_tiles<T, false>
                    <<<grid, kTileThreads, 0, stream>>>(xp, q, scale, rows, cols, row_blocks, blocks);
        }
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
