// quantize_mx4.cu - microscaled 4-bit values (e2m1) with a power of two for each
// block of 32 columns of a row (quant.cuh).
//
// Bound by HBM: reads the input once, writes 17 bytes for 32 values.  Four lanes hold
// a block, a warp 256 columns.  Where rows are whole blocks the matrix is one run of
// them, and a warp's eight scales go out as one store.
#include "eight.cuh"
#include "quant.cuh"

namespace rowops {
namespace {

constexpr int kMxThreads = 256;

struct Mx4Args {
    const void* x;
    uint8_t* q;
    uint8_t* scale;
    int64_t rows;
    int cols, units;
    int64_t items;  // of 256 values: of the matrix (FLAT), or units of its rows
};

template <typename T, bool VEC, bool FLAT, int ITEMS>
__global__ void __launch_bounds__(kMxThreads) quantize_mx4_rows(const Mx4Args a) {
    const int lane = threadIdx.x & 31;
    const int64_t first = (int64_t(blockIdx.x) * (kMxThreads / 32) + (threadIdx.x >> 5)) * ITEMS;
    const int64_t step = int64_t(gridDim.x) * (kMxThreads / 32) * ITEMS;
    for (int64_t item0 = first; item0 < a.items; item0 += step) {
        Held<T, 32, VEC> x[ITEMS];
        int64_t row[ITEMS];
        int base[ITEMS], cols[ITEMS];
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int64_t item = item0 + n;
            if constexpr (FLAT) {  // the matrix as rows of 256
                row[n] = item;
                base[n] = 0;
                const int64_t left = a.rows * int64_t(a.cols) - item * 256;
                cols[n] = left < 256 ? int(max(left, int64_t(0))) : 256;
            } else {
                row[n] = item / a.units;
                base[n] = int(item - row[n] * a.units) * 256;
                cols[n] = item < a.items ? a.cols : 0;
            }
            x[n].load(static_cast<const T*>(a.x) + row[n] * (FLAT ? 256 : a.cols), base[n], lane, cols[n]);
        }
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x[n].get(i);
            if constexpr (FLAT) {
                store_mx4<32, VEC>(a.q + row[n] * 128, a.scale + row[n] * 8, 0, lane, cols[n], v);
            } else {
                store_mx4<32, VEC>(a.q + row[n] * ((a.cols + 1) / 2), a.scale + row[n] * ((a.cols + 31) / 32), base[n],
                                   lane, cols[n], v);
            }
        }
    }
}

}  // namespace

cudaError_t launch_quantize_mx4(const void* x, uint8_t* q, uint8_t* scale, int64_t rows, int64_t cols, int x_type,
                                cudaStream_t stream) {
    Mx4Args a{x, q, scale, rows, int(cols), int((cols + 255) / 256), 0};
    const bool vec = cols % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0;
    const bool flat = vec && cols % 32 == 0;
    a.items = flat ? (rows * cols + 255) / 256 : rows * a.units;
    auto go = [&](auto kernel, int each) {
        const int64_t per = int64_t(kMxThreads / 32) * each;
        const int64_t blocks = (a.items + per - 1) / per, most = int64_t(1) << 20;
        kernel<<<unsigned(blocks < most ? blocks : most), kMxThreads, 0, stream>>>(a);
    };
    with_type(x_type, [&](auto t) {
        using T = decltype(t);
        if (flat) go(quantize_mx4_rows<T, true, true, 1>, 1);
        else if (vec) go(quantize_mx4_rows<T, true, false, 1>, 1);
        else go(quantize_mx4_rows<T, false, false, 1>, 1);
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
