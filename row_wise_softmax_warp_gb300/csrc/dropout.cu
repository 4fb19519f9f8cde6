// dropout.cu - dropout from a counter-based generator, with a residual's addition.
//
//   y = residual + [u >= t] * x * 65536 / (65536 - t),   t = round(65536 p)
//
// u: 16 bits for each value (philox.cuh).  On a gradient, without a residual, the same
// call is the backward pass.  Bound by HBM where a value takes 6 bytes or more, by
// the generator's products below.
#include "eight.cuh"

namespace rowops {
namespace {

constexpr int kDropThreads = 256;

struct DropoutArgs {
    const void* x;
    const void* residual;  // may be NULL
    void* y;
    Dropout drop;
    int64_t rows;
    int cols, units;  // units: groups of 256 columns in a row
    int64_t items;    // rows * units; VEC: groups of 256 values of the whole matrix
};

// A warp takes 256 values at a time.  VEC: rows are whole blocks of 8, so the matrix is
// one run of them.
template <typename T, typename R, bool VEC, int ITEMS>
__global__ void __launch_bounds__(kDropThreads) dropout_rows(const DropoutArgs g) {
    const int lane = threadIdx.x & 31;
    const Masker masker(g.drop);
    const int64_t first = (int64_t(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5)) * ITEMS;
    const int64_t step = int64_t(gridDim.x) * (kDropThreads / 32) * ITEMS;
    for (int64_t item0 = first; item0 < g.items; item0 += step) {
        Held<T, 32, VEC> x[ITEMS];
        Held<R, 32, VEC> residual[ITEMS];
        int64_t row[ITEMS], at[ITEMS];
        int base[ITEMS], cols[ITEMS];
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int64_t item = item0 + n;
            if constexpr (VEC) {  // the matrix as rows of 256
                row[n] = item;
                base[n] = 0;
                at[n] = item * 256;
                const int64_t left = g.rows * int64_t(g.cols) - at[n];
                cols[n] = left < 256 ? int(max(left, int64_t(0))) : 256;
            } else {
                row[n] = item / g.units;
                base[n] = int(item - row[n] * g.units) * 256;
                at[n] = row[n] * g.cols;
                cols[n] = item < g.items ? g.cols : 0;
            }
            x[n].load(static_cast<const T*>(g.x) + at[n], base[n], lane, cols[n]);
            if (g.residual) residual[n].load(static_cast<const R*>(g.residual) + at[n], base[n], lane, cols[n]);
        }
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x[n].get(i);
            drop_eight<32, VEC>(v, g.drop, masker, row[n], VEC ? 32 : (g.cols + 7) / 8, base[n], lane);
            if (g.residual)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += residual[n].get(i);
            store_eight<32, VEC>(static_cast<R*>(g.y) + at[n], base[n], lane, cols[n], v);
        }
    }
}

}  // namespace

cudaError_t launch_dropout(const void* x, const void* residual, const uint64_t* rng, void* y, int64_t rows,
                           int64_t cols, float p, int x_type, int y_type, cudaStream_t stream) {
    DropoutArgs g{x, residual, y, dropout_of(rng, p), rows, int(cols), int((cols + 255) / 256), 0};
    const bool vec = cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                                        reinterpret_cast<uintptr_t>(y)) & 15) == 0;
    g.items = vec ? (rows * cols + 255) / 256 : rows * g.units;
    auto go = [&](auto kernel, int each) {
        const int64_t per = int64_t(kDropThreads / 32) * each;
        const int64_t blocks = (g.items + per - 1) / per, most = int64_t(1) << 20;
        kernel<<<unsigned(blocks < most ? blocks : most), kDropThreads, 0, stream>>>(g);
    };
    with_type(x_type, [&](auto t) {
        with_type(y_type, [&](auto r) {
            using T = decltype(t);
            using R = decltype(r);
            if (vec) go(dropout_rows<T, R, true, 1>, 1);
            else go(dropout_rows<T, R, false, 1>, 1);
        });
    });
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace rowops
