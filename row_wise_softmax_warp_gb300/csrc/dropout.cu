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
        int64_t row[ITEMS];
        int base[ITEMS], cols[ITEMS];
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int64_t item = item0 + n;
            if constexpr (VEC) {  // the matrix as rows of 256
                row[n] = item;
                base[n] = 0;
                cols[n] = int(max(int64_t(0), min(int64_t(256), g.rows * int64_t(g.cols) - item * 256)));
            } else {
                row[n] = item / g.units;
                base[n] = int(item - row[n] * g.units) * 256;
                cols[n] = item < g.items ? g.cols : 0;
            }
            const Place<32, VEC> o(row[n], VEC ? 256 : g.cols, base[n], lane, cols[n]);
            x[n].load(static_cast<const T*>(g.x), o);
            if (g.residual) residual[n].load(static_cast<const R*>(g.residual), o);
        }
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const Place<32, VEC> o(row[n], VEC ? 256 : g.cols, base[n], lane, cols[n]);
            float2 v[4];
            x[n].get(v);
            drop_eight<32, VEC>(v, g.drop, masker, row[n], VEC ? 32 : (g.cols + 7) / 8, base[n], lane);
            if (g.residual) {
                float2 r[4];
                residual[n].get(r);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = add2(v[i], r[i]);
            }
            store_eight<32, VEC>(static_cast<R*>(g.y), o, v);
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
