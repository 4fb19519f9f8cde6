// quantize_mx4.cu - microscaled 4-bit values (e2m1) with a power of two for each
// block of 32 columns of a row (quant.cuh).
//
// Bound by HBM: reads the input once, writes 17 bytes for 32 values.  Four lanes hold
// a block.  Where rows are whole blocks the matrix is one run of chunks of eight values,
// of which a thread has four on their way (16384 x 4096 bf16: 27 us, 6.2 TB/s; one at a
// time 49, eight 36), and the maximum of 16-bit values is taken on their bits, two at a
// time.  Rows of other lengths are read value by value where they are no multiple of 8
// (16384 x 1001: 24 us, x 1000: 15).
#include "eight.cuh"
#include "quant.cuh"

namespace rowops {
namespace {

// The largest magnitude of eight values as fp32 bits; 16-bit values are compared as they
// are, two at a time.
template <typename T>
__device__ __forceinline__ uint32_t most_of(const Held<T, 32, true>& x) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            m = max(max(m, max(x.c[h].x & 0x7fffffffu, x.c[h].y & 0x7fffffffu)),
                    max(x.c[h].z & 0x7fffffffu, x.c[h].w & 0x7fffffffu));
        return group_max_bits<4>(m);
    } else {
        const uint4 w = x.c[0];
        uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                              __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, o));
        return __float_as_uint(unpack2<T>(max(m & 0xffffu, m >> 16)).x);
    }
}

// Rows that are whole blocks: the matrix as one run of chunks of eight values, ITEMS of
// them a thread.
template <typename T, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    quantize_mx4_run(const T* x, uint32_t* __restrict__ q, uint8_t* __restrict__ scale, int64_t chunks) {
    let_next_start();
    const int64_t first = int64_t(blockIdx.x) * (THREADS * ITEMS) + threadIdx.x;
    Held<T, 32, true> in[ITEMS];
#pragma unroll
    for (int n = 0; n < ITEMS; ++n)
        in[n].load(x, Place<32, true>(first + n * THREADS, 8, 0, 0, first + n * THREADS < chunks ? 8 : 0));
#pragma unroll
    for (int n = 0; n < ITEMS; ++n) {
        const int64_t at = first + n * THREADS;
        const uint32_t code = mx4_code(most_of<T>(in[n]));
        float2 v[4];
        in[n].get(v);
        if (at < chunks) {
            q[at] = mx4_eight(v, code);
            if ((threadIdx.x & 3) == 0) scale[at / 4] = uint8_t(code);
        }
    }
}

constexpr int kMxThreads = 256;

struct Mx4Args {
    const void* x;
    uint8_t* q;
    uint8_t* scale;
    int64_t rows;
    int cols, units;
    int64_t items;  // units of all rows
};

// Other rows, a warp 256 columns.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads) quantize_mx4_rows(const Mx4Args a) {
    let_next_start();
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * (kMxThreads / 32);
    for (int64_t item = int64_t(blockIdx.x) * (kMxThreads / 32) + (threadIdx.x >> 5); item < a.items; item += step) {
        const int64_t row = item / a.units;
        const int base = int(item - row * a.units) * 256;
        Held<T, 32, VEC> x;
        x.load(static_cast<const T*>(a.x), Place<32, VEC>(row, a.cols, base, lane, a.cols));
        float2 v[4];
        x.get(v);
        store_mx4<32, VEC>(a.q + row * ((a.cols + 1) / 2), a.scale + row * ((a.cols + 31) / 32), base, lane, a.cols, v);
    }
}

}  // namespace

cudaError_t launch_quantize_mx4(const void* x, uint8_t* q, uint8_t* scale, int64_t rows, int64_t cols, int x_type,
                                cudaStream_t stream) {
    const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0;
    with_type(x_type, [&](auto t) {
        using T = decltype(t);
        if (vec && cols % 32 == 0) {
            const int64_t chunks = rows * cols / 8;
            auto go = [&](auto kernel, int per, int threads) {
                kernel<<<unsigned((chunks + per - 1) / per), threads, 0, stream>>>(
                    static_cast<const T*>(x), reinterpret_cast<uint32_t*>(q), scale, chunks);
            };
            const bool few = chunks < 2048 * int64_t(sm_count());
            if (few) go(quantize_mx4_run<T, 1, 128>, 128, 128);
            else go(quantize_mx4_run<T, 4, 256>, 4 * 256, 256);
        } else {
            Mx4Args a{x, q, scale, rows, int(cols), int((cols + 255) / 256), 0};
            a.items = rows * a.units;
            const int64_t blocks = (a.items + kMxThreads / 32 - 1) / (kMxThreads / 32), most = int64_t(1) << 20;
            const unsigned grid = unsigned(blocks < most ? blocks : most);
            if (vec) quantize_mx4_rows<T, true><<<grid, kMxThreads, 0, stream>>>(a);
            else quantize_mx4_rows<T, false><<<grid, kMxThreads, 0, stream>>>(a);
        }
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
